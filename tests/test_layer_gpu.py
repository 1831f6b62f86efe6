"""The operators around the products as a decoder layer uses them together: the norm with residual, projections with adapters, the
norm again, the router's rule and the experts, the last norm in 8 bits.

Every step is compared with its oracle on the inputs that it had on the device, with the tolerances of the operator's own
tests; a captured run of all of them has the same bits as one step after another."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import layer as ol
from tests.gpu_util import qlib, to_f64
from tests.test_lora_gpu import adapters, check as check_lora, ids_of
from tests.test_norm_gpu import check_codes, check_y, matrix

pytestmark = pytest.mark.gpu

HIDDEN, INNER, EXPERTS, TOPK = 256, 640, 16, 4


class Layer:
    def __init__(self, q, m):
        self.q, self.m = q, m
        self.w_in, self.w_out = wl.weight(wl.NVFP4, INNER, HIDDEN, seed=1), wl.weight(wl.NVFP4, HIDDEN, INNER, seed=2)
        self.p_in, self.p_out = q.PackedWeight.from_logical(self.w_in), q.PackedWeight.from_logical(self.w_out)
        self.ad_in = adapters(q, 5, 16, HIDDEN, INNER, 3, ranks=[16, 8, 0, 5, 12])
        self.ad_out = adapters(q, 5, 32, INNER, HIDDEN, 4)
        self.norms = [matrix(1, HIDDEN, s)[0] for s in (5, 6, 7)]
        self.logical = wl.moe_layer(wl.MXFP4, EXPERTS, HIDDEN, 128, seed=8, shared=True)
        self.moe = q.PackedMoE(self.logical)
        self.router = torch.randn(HIDDEN, EXPERTS, generator=torch.Generator().manual_seed(9)).cuda() * HIDDEN ** -0.5
        self.kw = dict(score="sigmoid", groups=4, topk_groups=2, scale=2.5)
        self.bias = 0.3 * np.random.default_rng(10).standard_normal(EXPERTS).astype(np.float32)
        self.rule = q.RouteRule(bias=torch.from_numpy(self.bias).cuda(), **self.kw)
        lora = max(q.lora_workspace_size(self.ad_in, m), q.lora_workspace_size(self.ad_out, m))
        self.ws = [q.Workspace(b) for b in (
            q.qg_gemm_workspace_size(self.p_in.fmt, INNER, HIDDEN, m), lora, q.qg_gemm_workspace_size(self.p_out.fmt, HIDDEN, INNER, m),
            q.qmoe_route_workspace_size(m, EXPERTS, TOPK), q.qmoe_workspace_size(self.moe.desc, m, TOPK))]

    def __call__(self, x, residual, ids):
        q, ws = self.q, self.ws
        h1, s1 = q.rms_norm(x, self.norms[0], residual)
        plain_in = q.gemm(self.p_in, h1, workspace=ws[0])
        inner = q.lora(self.ad_in, ids, h1, plain_in, out=torch.empty_like(plain_in), workspace=ws[1])
        plain_out = q.gemm(self.p_out, inner, workspace=ws[2])
        back = q.lora(self.ad_out, ids, inner, plain_out.clone(), workspace=ws[1])  # in place; the same workspace after other sizes
        h2, s2 = q.rms_norm(back, self.norms[1], s1)
        logits = h2.float() @ self.router
        mixed, experts, weights, _ = q.moe_forward(self.moe, h2, logits, TOPK, workspace=ws[4], route_ws=ws[3], rule=self.rule)
        codes, scales, s3 = q.rms_norm_fp8(mixed, self.norms[2], s2, group=128)
        return dict(h1=h1, s1=s1, plain_in=plain_in, inner=inner, plain_out=plain_out, back=back, h2=h2, s2=s2, logits=logits,
                    mixed=mixed, experts=experts, weights=weights, codes=codes, scales=scales, s3=s3)


def check_gemm(w, x, got):
    bits = x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    ref, _ = oracle.gemv(w, bits)
    assert np.all(np.abs(to_f64(got) - ref) <= oracle.tolerance(w, bits, ref=ref))


def check_norm(x, residual, weight, y, s):
    want_s, want = ol.rms_norm(to_f64(x), to_f64(residual), to_f64(weight), 1e-6, 0.0)
    assert np.array_equal(to_f64(s), want_s)
    if y is not None:
        check_y(y, want)
    return want


def inputs(m, seed):
    ids = torch.tensor(ids_of("mixed", m, 5, seed), dtype=torch.int32, device="cuda")
    return matrix(m, HIDDEN, seed), matrix(m, HIDDEN, seed + 1, 2.0), ids


@pytest.mark.parametrize("m", [1, 4, 40, 300])
def test_layer_step_by_step_and_captured(m):
    q = qlib()
    layer = Layer(q, m)
    x, residual, ids = inputs(m, m)
    r = layer(x, residual, ids)
    check_norm(x, residual, layer.norms[0], r["h1"], r["s1"])
    check_gemm(layer.w_in, r["h1"], r["plain_in"])
    check_lora(layer.ad_in, ids.tolist(), r["h1"], r["plain_in"], r["inner"])
    check_gemm(layer.w_out, r["inner"], r["plain_out"])
    check_lora(layer.ad_out, ids.tolist(), r["inner"], r["plain_out"], r["back"])
    check_norm(r["back"], r["s1"], layer.norms[1], r["h2"], r["s2"])
    want_ids, p = ol.route_by(r["logits"].cpu().numpy(), TOPK, bias=layer.bias, **layer.kw)
    assert np.array_equal(r["experts"].cpu().numpy(), want_ids)
    spread = float(r["logits"].max() - r["logits"].min())
    assert np.all(np.abs(r["weights"].cpu().numpy() - p) <= (64 + spread) * 2.0 ** -24 * p)
    xv, lo, mixed = to_f64(r["h2"]), layer.logical, to_f64(r["mixed"])
    for i in {0, m // 2, m - 1}:  # a few tokens' experts
        ref, tol = np.zeros(HIDDEN), np.zeros(HIDDEN)
        for e, pe in [*zip(want_ids[i], p[i]), (-1, 1.0)]:
            gu, dn = (lo.shared_gate_up, lo.shared_down) if e < 0 else (lo.gate_up[e], lo.down[e])
            _, _, h, d = oracle.expert_ffn(oracle.dequant(gu), oracle.dequant(dn), xv[i:i + 1])
            ref += pe * d[0]
            tol += pe * ((2e-3 + 2.0 ** -8) * np.linalg.norm(h) * float(np.max(oracle.row_norms(dn))) + 2.0 ** -8 * np.abs(d[0]))
        assert np.all(np.abs(mixed[i] - ref) <= tol + 2.0 ** -7 * np.abs(ref))
    check_codes(r["codes"], r["scales"], check_norm(r["mixed"], r["s2"], layer.norms[2], None, r["s3"]), 128)
    assert all(layer.ws[i].status() == 0 for i in (0, 1, 2, 4))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(x, residual, ids)
    for a, b in zip((x, residual, ids), inputs(m, m + 50)):
        a.copy_(b)
    for _ in range(2):
        graph.replay()
    want = layer(x, residual, ids)
    torch.cuda.synchronize()
    for name, t in want.items():
        assert torch.equal(t.contiguous().view(torch.uint8), held[name].contiguous().view(torch.uint8)), name
    assert all(layer.ws[i].status() == 0 for i in (0, 1, 2, 4))

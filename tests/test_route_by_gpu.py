"""Routing by a rule on the GPU against the 64-bit oracle: the choice is equal, ties and values that fp32 cannot tell apart
included; weights in fp32.

Weights: sigmoid 6 u (u = 2^-24), a softmax's exp also the rounding of its argument (u times its size) and its sum 40 u; a sum of at
most 16 and a division, the factor's product: 64 u + u * (largest distance of logits) cover both."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import layer as ol
from tests.gpu_util import dev_bf16, qlib, to_f64

pytestmark = pytest.mark.gpu


def compare(q, logits, topk, bias=None, tables=True, **rule):
    lg = np.ascontiguousarray(logits, np.float32)
    t, e = lg.shape
    ids, w = ol.route_by(lg, topk, bias=bias, **rule)
    rr = q.RouteRule(bias=None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda(), **rule)
    ws = q.Workspace(q.qmoe_route_workspace_size(t, e, topk))
    gi, gw, _ = q.route(torch.from_numpy(lg).cuda(), topk, workspace=ws, rule=rr)
    gi, gw = gi.cpu().numpy(), gw.cpu().numpy().astype(np.float64)
    assert np.array_equal(gi, ids), np.argwhere(gi != ids)[:5]
    fine = lg[np.isfinite(lg)]
    tol = (64 + (fine.max() - fine.min() if fine.size else 0)) * 2.0 ** -24
    assert np.array_equal(np.isnan(gw), np.isnan(w))
    ok = ~np.isnan(w)
    assert np.all(np.abs(gw - w)[ok] <= tol * np.abs(w[ok]) + 2.0 ** -140)
    if tables:  # the same tables as the router writes for logits with this choice
        lg2 = np.full((t, e), -50.0, np.float32)
        np.put_along_axis(lg2, ids, np.arange(topk, 0, -1, dtype=np.float32)[None].repeat(t, 0), axis=1)
        ws2 = q.Workspace(q.qmoe_route_workspace_size(t, e, topk))
        i2, _, _ = q.route(torch.from_numpy(lg2).cuda(), topk, workspace=ws2)
        assert np.array_equal(i2.cpu().numpy(), ids) and tables_equal(q, ws.buf, ws2.buf, t, e, topk)


def tables_equal(q, a, b, t, e, k):
    """Every table that the products read, compared as far as it is filled."""
    at, parts, pairs = 0, {}, t * k
    for name, ints in (("meta", 16), ("counts", e), ("offsets", e + 1), ("active", e), ("pair_list", pairs), ("pair_pos", pairs),
                       ("tiles", 3 * (-(-pairs // 192) + e)), ("groups", 8 * e), ("zidx", e)):
        parts[name] = (at, ints)
        at += (4 * ints + 255) // 256 * 256
    get = lambda buf, name: buf[parts[name][0]:parts[name][0] + 4 * parts[name][1]].view(torch.int32).cpu().numpy()  # noqa: E731
    n_active, n_tiles = get(a, "meta")[:2]
    used = {"meta": 2, "counts": e, "offsets": e + 1, "active": n_active, "pair_list": pairs, "pair_pos": pairs, "tiles": 3 * n_tiles}
    if not all(np.array_equal(get(a, n)[:c], get(b, n)[:c]) for n, c in used.items()):
        return False
    act = get(a, "active")[:n_active]
    if not np.array_equal(get(a, "zidx")[act], get(b, "zidx")[act]):
        return False
    ga, gb = (get(x, "groups").reshape(-1, 8)[:n_active] for x in (a, b))
    rows = np.arange(4)[None] < np.minimum(ga[:, 2:3], 4)
    return np.array_equal(ga[:, :3], gb[:, :3]) and np.array_equal(np.where(rows, ga[:, 4:], 0), np.where(rows, gb[:, 4:], 0))


RULES = [dict(score="sigmoid"), dict(score="softmax"), dict(score="softmax", renormalise=False, scale=16.0),
         dict(score="sigmoid", renormalise=False), dict(score="sigmoid", scale=2.5)]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (1, 512, 10), (3, 100, 16), (31, 33, 5), (33, 256, 8), (64, 512, 10), (102, 160, 10),
                                   (128, 64, 8), (129, 40, 3), (700, 512, 16)])
def test_no_groups(t, e, k, biased, rule):
    q = qlib()
    rng = np.random.default_rng(t * 1000 + e)
    compare(q, 1.5 * rng.standard_normal((t, e)), k, bias=0.2 * rng.standard_normal(e) if biased else None, **rule)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("t,e,k,groups,kept", [(1, 256, 8, 8, 4), (1, 64, 4, 32, 2), (5, 160, 6, 8, 3), (40, 96, 6, 3, 1), (200, 512, 16, 4, 2),
                                               (33, 10, 2, 5, 1), (64, 62, 2, 31, 30), (300, 256, 8, 8, 8), (17, 512, 10, 1, 1)])
def test_groups(t, e, k, groups, kept, best, biased, score):
    q = qlib()
    rng = np.random.default_rng(t + e + best)
    compare(q, 1.5 * rng.standard_normal((t, e)), k, bias=0.2 * rng.standard_normal(e) if biased else None, score=score, groups=groups,
            topk_groups=kept, group_best=best)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("near", [4, 20, 31, 33, 200])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_values_that_fp32_cannot_order(score, near, groups, kept):
    """`near` experts whose score plus bias is one value up to the bias's rounding (half a ulp), the others below."""
    q = qlib()
    t, e = 70, 256
    rng = np.random.default_rng(near)
    lg = rng.standard_normal((t, e)).astype(np.float32)
    lg[:] = lg[0]  # one bias for all tokens: the same scores, in another place by a common shift for softmax
    s = 1 / (1 + np.exp(-lg[0].astype(np.float64))) if score == "sigmoid" else np.exp(lg[0].astype(np.float64)) / np.exp(lg[0].astype(np.float64)).sum()
    bias = (-0.5 - rng.random(e)).astype(np.float32)
    who = rng.permutation(e)[:near]
    bias[who] = (1.25 - s[who]).astype(np.float32)
    lg[1::2] += (rng.integers(-8, 9, (t // 2, 1)) if score == "softmax" else 0)
    compare(q, lg, 10 if near > 10 else 4, bias=bias, score=score, groups=groups, topk_groups=kept)


def test_groups_that_fp32_cannot_order():
    q = qlib()
    rng = np.random.default_rng(3)
    e, groups = 64, 8
    lg = rng.standard_normal((1, e)).astype(np.float32).repeat(40, 0)
    s = 1 / (1 + np.exp(-lg[0].astype(np.float64)))
    bias = (-1.0 - rng.random(e)).astype(np.float32)
    for g in range(groups):  # each group's two best sum to 1.5 up to rounding
        i, j = 8 * g + rng.permutation(8)[:2]
        bias[i] = np.float32(1.0 - s[i])
        bias[j] = np.float32(1.5 - (s[i] + np.float64(bias[i])) - s[j])
    compare(q, lg, 6, bias=bias, score="sigmoid", groups=groups, topk_groups=4)


@pytest.mark.parametrize("t", [6, 140])
def test_ties_and_special_values(t):
    q = qlib()
    rng = np.random.default_rng(4)
    e = 96
    same = np.zeros((t, e), np.float32)
    for rule in (dict(score="sigmoid"), dict(score="softmax"), dict(score="sigmoid", groups=8, topk_groups=2),
                 dict(score="softmax", groups=8, topk_groups=2, group_best=1)):
        compare(q, same, 8, **rule)
        compare(q, same, 8, bias=np.zeros(e), **rule)
        compare(q, rng.integers(-2, 3, (t, e)).astype(np.float32), 8, bias=rng.integers(0, 2, e).astype(np.float32), **rule)
    lg = rng.standard_normal((t, e)).astype(np.float32)
    lg[0, ::2] = -np.inf  # experts that are out
    lg[1, 5:] = -np.inf
    lg[2, 7] = np.nan
    lg[3, 3:] = np.nan    # fewer numbers than experts to choose
    lg[4] = -60 + lg[4]   # sigmoid scores of 1e-26
    lg[5] = -120 + lg[5]  # below fp32's numbers
    for score in ("sigmoid", "softmax"):
        for bias in (None, 0.1 * rng.standard_normal(e)):
            compare(q, lg, 8, score=score, bias=bias)
            compare(q, lg, 8, score=score, bias=bias, renormalise=False)
    bias = 0.1 * rng.standard_normal(e)
    bias[:40] = -np.inf   # experts taken out by their bias
    compare(q, lg[6:] if t > 6 else lg[:1], 8, score="sigmoid", bias=bias)


def test_large_batch():
    q = qlib()
    rng = np.random.default_rng(5)
    compare(q, rng.standard_normal((8191, 512)).astype(np.float32), 10, bias=0.1 * rng.standard_normal(512), score="sigmoid")


def test_without_a_rule_nothing_changes():
    q = qlib()
    lg = torch.randn(50, 64, device="cuda")
    a, b = q.route(lg, 6), q.route(lg, 6, rule=q.RouteRule("softmax"))
    assert torch.equal(a[0], b[0])
    assert torch.allclose(a[1], b[1], rtol=2.0 ** -20, atol=0)


@pytest.mark.parametrize("t", [1, 4, 40])
def test_layer_by_a_rule(t):
    """Router and experts together, in one call and in two, against the oracle's experts with the oracle's weights."""
    q = qlib()
    layer = wl.moe_layer(wl.MXFP4, 16, 256, 128, seed=1, shared=True)
    pm = q.PackedMoE(layer)
    x, lg = wl.moe_tokens(t, 256, seed=2), wl.router_logits(t, 16, seed=3)
    bias = np.random.default_rng(1).standard_normal(16).astype(np.float32)
    kw = dict(score="sigmoid", groups=4, topk_groups=2, scale=2.5)
    rule = q.RouteRule(bias=torch.from_numpy(bias).cuda(), **kw)
    xt, lt = dev_bf16(x), torch.from_numpy(lg).cuda()
    out, ids, w, _ = q.moe_forward(pm, xt, lt, 4, rule=rule)
    i2, w2, rws = q.route(lt, 4, rule=rule)
    assert torch.equal(ids, i2) and torch.equal(w, w2) and torch.equal(out, q.moe_ffn(pm, xt, w2, rws))
    want_ids, p = ol.route_by(lg, 4, bias=bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    xv = oracle.bf16_value(x)
    ref, tol = np.zeros((t, 256)), np.zeros((t, 256))
    for i in range(t):  # each product within the GEMV's bound, h and (prefill) the pair's output rounded to bf16
        for e, pe in [*zip(want_ids[i], p[i]), (-1, 1.0)]:
            gu, dn = (layer.shared_gate_up, layer.shared_down) if e < 0 else (layer.gate_up[e], layer.down[e])
            _, _, h, d = oracle.expert_ffn(oracle.dequant(gu), oracle.dequant(dn), xv[i:i + 1])
            ref[i] += pe * d[0]
            tol[i] += pe * ((2e-3 + 2.0 ** -8) * np.linalg.norm(h) * float(np.max(oracle.row_norms(dn))) + 2.0 ** -8 * np.abs(d[0]))
    assert np.all(np.abs(to_f64(out) - ref) <= tol + 2.0 ** -7 * np.abs(ref))


def test_graph_and_stream():
    q = qlib()
    rule = q.RouteRule("sigmoid", bias=0.1 * torch.randn(64, device="cuda"), groups=8, topk_groups=4)
    for t in (20, 400):
        lg = torch.randn(t, 64, device="cuda")
        ws = q.Workspace(q.qmoe_route_workspace_size(t, 64, 6))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            q.route(lg, 6, workspace=ws, rule=rule)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ids, w, _ = q.route(lg, 6, workspace=ws, rule=rule)
        lg.copy_(torch.randn(t, 64, device="cuda"))
        graph.replay()
        i2, w2, ws2 = q.route(lg, 6, rule=rule)
        torch.cuda.synchronize()
        assert torch.equal(ids, i2) and torch.equal(w, w2) and tables_equal(q, ws.buf, ws2.buf, t, 64, 6)


@pytest.mark.parametrize("t", [1, 2, 3, 50])
def test_infinite_and_saturated_values(t):
    """Biases of +infinity (in groups too, two in a group), logits of +infinity, and scores that are 1 to the last bit."""
    q = qlib()
    rng = np.random.default_rng(6)
    e = 96
    lg = rng.standard_normal((t, e)).astype(np.float32)
    bias = 0.1 * rng.standard_normal(e)
    one, two = bias.copy(), bias.copy()
    one[70] = np.inf
    two[[50, 51, 53, 90, 91]] = np.inf
    for b in (one, two):
        for kw in (dict(), dict(groups=8, topk_groups=2), dict(groups=8, topk_groups=2, group_best=1), dict(groups=32, topk_groups=9)):
            for score in ("sigmoid", "softmax"):
                compare(q, lg, 6, bias=b, score=score, **kw)
    top = lg.copy()
    top[:, [3, 40]] = np.inf
    compare(q, top, 6, score="sigmoid")
    for score in ("sigmoid", "softmax"):  # softmax: the logits choose (with a bias the index, every score being NaN), weights NaN
        compare(q, top, 6, score=score)
        compare(q, top, 6, score=score, bias=bias)
    compare(q, 40 + 10 * np.abs(lg), 6, score="sigmoid")
    compare(q, 40 + 10 * np.abs(lg), 6, score="sigmoid", bias=bias)
    compare(q, 1e4 * lg, 6, score="softmax", bias=bias)


def test_two_streams_at_once_and_wrong_devices():
    q = qlib()
    rule = q.RouteRule("softmax", bias=0.01 * torch.randn(128, device="cuda"), groups=8, topk_groups=4)
    lg = torch.randn(3000, 128, device="cuda")
    want = q.route(lg, 8, rule=rule)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(q.route(lg, 8, rule=rule))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) and tables_equal(q, g[2].buf, want[2].buf, 3000, 128, 8)
    with pytest.raises(q.QGError):
        q.route(lg.cpu(), 8, rule=rule)
    with pytest.raises(q.QGError):
        q.route(lg, 8, rule=q.RouteRule("softmax", bias=torch.zeros(128)))


@pytest.mark.parametrize("t", [2, 3, 7, 8, 9, 32, 33, 40, 57, 64, 65, 72, 128, 129])
@pytest.mark.parametrize("e,k", [(16, 16), (130, 6), (512, 16)])
def test_borders_between_the_launches(t, e, k):
    """One CTA, a cluster, launches of blocks; and without a rule, whose tables are the same."""
    q = qlib()
    rng = np.random.default_rng(t + e)
    lg = rng.standard_normal((t, e)).astype(np.float32)
    compare(q, lg, k, bias=0.1 * rng.standard_normal(e), score="sigmoid")
    dev = torch.from_numpy(lg).cuda()
    (i1, w1, s1), (i2, w2, s2) = q.route(dev, k), q.route(dev, k, rule=q.RouteRule("softmax"))
    assert torch.equal(i1, i2) and torch.allclose(w1, w2, rtol=2.0 ** -20, atol=0) and tables_equal(q, s1.buf, s2.buf, t, e, k)

"""Refusals of the RMS norm, the low-rank adapters and the routing by a rule, found on the host before anything is launched
(no GPU)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, MISALIGNED, SMALL, CUDA = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def q():
    from prefill_dequant_gemv_gb300 import build as b
    b.build()
    import prefill_dequant_gemv_gb300 as q
    q.lib()
    return q


def norm(q, x=0x10000, ldx=512, res=0x20000, ldr=512, m=4, k=512, w=0x1000, eps=1e-6, off=0.0, out="out", **over):
    f = dict(sum=0x30000, ldh=512, y=0x40000, ldy=512, codes=None, ldc=0, scales=None, lds=0, group=0)
    return q.lib().qg_rms_norm(x, ldx, res, ldr, m, k, w, eps, off, q.qg_norm_out(**{**f, **over}) if out == "out" else out, None)


FP8 = dict(y=None, codes=0x50000, ldc=512, scales=0x60000, lds=4, group=128)


@pytest.mark.parametrize("over,want", [
    (dict(out=None), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(off=float("inf")), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(res=None), INVALID),
    (dict(ldx=504), INVALID), (dict(ldr=504), INVALID), (dict(ldh=504), INVALID), (dict(ldy=504), INVALID),
    (dict(ldx=516), MISALIGNED), (dict(ldr=516), MISALIGNED), (dict(ldh=516), MISALIGNED), (dict(ldy=516), MISALIGNED),
    (dict(x=0x10008), MISALIGNED), (dict(w=0x1008), MISALIGNED), (dict(res=0x20002), MISALIGNED), (dict(sum=0x30004), MISALIGNED),
    (dict(y=0x40008), MISALIGNED), (dict(k=65537, ldx=65544, ldr=65544, ldh=65544, ldy=65544), UNSUPPORTED),
    (dict(m=1 << 31), UNSUPPORTED), (dict(sum=0x10000, ldh=1024), INVALID), (dict(y=0x20000, ldy=1024), INVALID),
    (dict(y=0x30000), INVALID), (dict(codes=0x50000, ldc=512), INVALID), (dict(scales=0x50000, lds=4), INVALID),
    (dict(FP8, group=16), UNSUPPORTED), (dict(FP8, group=100), UNSUPPORTED), (dict(FP8, group=-1), INVALID),
    (dict(FP8, lds=3), INVALID), (dict(FP8, ldc=504), INVALID), (dict(FP8, ldc=516), MISALIGNED),
    (dict(FP8, codes=0x50008), MISALIGNED), (dict(FP8, scales=0x60002), MISALIGNED), (dict(FP8, codes=0x10000), INVALID),
    (dict(FP8, group=0, lds=0), INVALID)])
def test_norm_refusals(q, over, want):
    assert norm(q, **over) == want


def test_nothing_to_do_is_fine_without_pointers(q):
    assert norm(q, m=0, x=None, res=None, w=None, sum=None, y=None) == 0
    assert lora(q, m=0, ids=None, x=None, y=None, out=None, ws=None, wsb=0) == 0


def lora_desc(q, **over):
    f = dict(n_adapters=4, max_rank=16, n=256, k=512, a=0x1000, lda=512, b=0x2000, scales=0x3000, ranks=0x4000)
    return q.qg_lora(**{**f, **over})


def lora(q, d=None, ids=0x5000, m=8, x=0x10000, ldx=512, y=0x20000, ldy=256, out=0x30000, ldo=256, ws=0x40000, wsb=256, **over):
    return q.lib().qlora(lora_desc(q, **over) if d is None else d, ids, m, x, ldx, y, ldy, out, ldo, ws, wsb, None)


@pytest.mark.parametrize("over,want", [
    (dict(n_adapters=0), INVALID), (dict(n_adapters=1025), UNSUPPORTED), (dict(max_rank=0), INVALID), (dict(max_rank=12), UNSUPPORTED),
    (dict(max_rank=136), UNSUPPORTED), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(n=1 << 24, ldy=1 << 24, ldo=1 << 24), UNSUPPORTED),
    (dict(k=1 << 24), UNSUPPORTED), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(scales=None), INVALID),
    (dict(lda=504), INVALID), (dict(lda=516), MISALIGNED), (dict(a=0x1008), MISALIGNED), (dict(b=0x2008), MISALIGNED),
    (dict(scales=0x3002), MISALIGNED), (dict(ranks=0x4001), MISALIGNED), (dict(ids=None), INVALID), (dict(ids=0x5002), MISALIGNED),
    (dict(m=-1), INVALID), (dict(m=1 << 27), UNSUPPORTED), (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(out=None), INVALID),
    (dict(ldx=504), INVALID), (dict(ldy=248), INVALID), (dict(ldo=248), INVALID), (dict(ldx=516), MISALIGNED), (dict(ldy=260), MISALIGNED),
    (dict(ldo=260), MISALIGNED), (dict(x=0x10008), MISALIGNED), (dict(y=0x20008), MISALIGNED), (dict(out=0x30008), MISALIGNED),
    (dict(out=0x20000, ldo=512), INVALID), (dict(out=0x10000), INVALID), (dict(ws=None), INVALID), (dict(ws=0x40008), MISALIGNED),
    (dict(wsb=255), SMALL)])
def test_lora_refusals(q, over, want):
    assert lora(q, **over) == want


def test_lora_refuses_no_descriptor(q):
    assert q.lib().qlora(None, 0x5000, 8, 0x10000, 512, 0x20000, 256, 0x30000, 256, 0x40000, 256, None) == INVALID
    assert q.qlora_workspace_size(lora_desc(q), 8) == 256 and q.qlora_workspace_size(lora_desc(q, max_rank=136), 8) == 0


def route(q, logits=0x10000, t=4, e=64, k=4, ids=0x20000, w=0x30000, ws=0x40000, wsb=1 << 30, rule="rule", **over):
    f = dict(score=2, n_groups=8, topk_groups=4, group_best=2, renormalise=1, scale=1.0, bias=0x1000)
    return q.lib().qmoe_route_by(q.qg_route_rule(**{**f, **over}) if rule == "rule" else rule, logits, t, e, k, ids, w, ws, wsb, None)


@pytest.mark.parametrize("over,want", [
    (dict(score=0), INVALID), (dict(score=3), INVALID), (dict(n_groups=0), INVALID), (dict(n_groups=7), INVALID),
    (dict(n_groups=64, topk_groups=32), INVALID), (dict(n_groups=64, topk_groups=32, group_best=1), UNSUPPORTED),
    (dict(topk_groups=0), INVALID), (dict(topk_groups=9), INVALID), (dict(topk_groups=1, k=9), INVALID), (dict(group_best=0), INVALID),
    (dict(group_best=3), INVALID), (dict(renormalise=2), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(bias=0x1002), MISALIGNED), (dict(t=0), INVALID), (dict(e=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(e=520), UNSUPPORTED), (dict(k=17), UNSUPPORTED), (dict(t=1 << 31), UNSUPPORTED), (dict(logits=None), INVALID),
    (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(logits=0x10004), MISALIGNED),
    (dict(ids=0x20004), MISALIGNED), (dict(ws=0x40008), MISALIGNED), (dict(wsb=64), SMALL)])
def test_route_refusals(q, over, want):
    assert route(q, **over) == want


def test_route_without_a_rule_has_the_router_s_refusals(q):
    assert route(q, rule=None, e=520) == UNSUPPORTED
    assert route(q, rule=None, logits=None) == INVALID
    assert route(q, rule=None, wsb=64) == SMALL


def test_python_helpers_refuse_wrong_tensors(q):
    torch = pytest.importorskip("torch")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    a, b, sc = bf(3, 16, 64), bf(3, 32, 16), torch.ones(3)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ad = q.LoraAdapters(a, b, sc, i32(3))
    assert isinstance(ad.desc, ctypes.Structure) and (ad.n, ad.k) == (32, 64)
    for bad in (lambda: q.LoraAdapters(a.float(), b, sc), lambda: q.LoraAdapters(a, b[:2], sc), lambda: q.LoraAdapters(a, b, sc[:2]),
                lambda: q.LoraAdapters(a, b, sc, i32(4)), lambda: q.LoraAdapters(a, b, sc, i32(3).long()),
                lambda: q.LoraAdapters(a[:, ::2], b[..., :8], sc), lambda: q.LoraAdapters(a[..., ::2], b, sc),
                lambda: q.LoraAdapters(bf(0, 16, 64), bf(0, 32, 16), torch.ones(0)), lambda: q.RouteRule("other"),
                lambda: q.RouteRule(bias=torch.zeros(4, dtype=torch.float64)), lambda: q.RouteRule(bias=torch.zeros(4, 2)),
                # no CUDA tensors
                lambda: q.lora(ad, i32(2), bf(2, 64), bf(2, 32)), lambda: q.rms_norm(bf(2, 64), bf(64)),
                lambda: q.rms_norm_fp8(bf(2, 64), bf(64)), lambda: q.route(torch.zeros(2, 8), 2, rule=q.RouteRule())):
        with pytest.raises(q.QGError) as e:
            bad()
        assert e.value.status == INVALID


def test_a_layer_by_a_rule_refuses_logits_of_other_shapes(q):
    torch = pytest.importorskip("torch")

    class Experts:
        n_experts = 8

    x, rule = torch.zeros(4, 64, dtype=torch.bfloat16), q.RouteRule("sigmoid")
    for logits in (torch.zeros(3, 8), torch.zeros(4, 9), torch.zeros(8, 4), torch.zeros(4, 8)):  # the last: no CUDA tensor
        with pytest.raises(q.QGError) as e:
            q.moe_forward(Experts(), x, logits, 2, rule=rule)
        assert e.value.status == INVALID
    for counts in (dict(groups=-1), dict(groups=1 << 32), dict(topk_groups=1 << 31), dict(group_best=-2)):
        with pytest.raises(q.QGError):
            q.RouteRule("sigmoid", **counts)


def test_workspaces_of_refused_sizes(q):
    size = lambda **over: q.qlora_workspace_size(lora_desc(q, **over), 8)  # noqa: E731
    assert size() == 256
    for bad in (dict(max_rank=12), dict(n=0), dict(k=0), dict(n=1 << 24), dict(k=1 << 24), dict(n_adapters=0), dict(n_adapters=1025)):
        assert size(**bad) == 0

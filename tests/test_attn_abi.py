"""Refusals of the cache append and the attention, found on the host before anything is launched (no GPU)."""
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


def cache(q, **over):
    f = dict(fmt=1, page_tokens=64, n_kv_heads=2, head_dim=128, n_pages=10, k_codes=0x1000, v_codes=0x2000,
             k_scales=0x3000, v_scales=0x4000)
    return q.qg_kv_cache(**{**f, **over})


def batch(q, **over):
    f = dict(n_seqs=2, max_new=4, max_len=200, q_start=0x5000, lens=0x6000, pages=0x7000, page_stride=4)
    return q.qg_kv_batch(**{**f, **over})


def norm_rope(q, **over):
    f = dict(q_weight=0x8000, k_weight=0x9000, eps=1e-6, weight_offset=0.0, cos_sin=0xA000, n_positions=200,
             rotary_dim=64, interleaved=0)
    return q.qg_norm_rope(**{**f, **over})


def attn(q, c=None, b=None, n=8, hq=4, qp=0x10000, ldq=512, hsq=128, scale=0.1, window=0, out=0x20000, ldo=512, hso=128,
         ws=0x30000, wsb=1 << 30):
    return q.lib().qattn(c or cache(q), b or batch(q), n, hq, qp, ldq, hsq, scale, window, out, ldo, hso, ws, wsb, None)


def append(q, c=None, b=None, nr="nr", n=8, hq=4, qp=0x10000, ldq=512, hsq=128, kp=0x11000, ldk=256, hsk=128, vp=0x12000,
           ldv=256, hsv=128, out=0x20000, ldo=512, hso=128, ws=0x30000, wsb=1 << 30):
    return q.lib().qkv_append(c or cache(q), b or batch(q), norm_rope(q) if nr == "nr" else nr, n, hq, qp, ldq, hsq, kp, ldk,
                              hsk, vp, ldv, hsv, out, ldo, hso, ws, wsb, None)


CACHE = [(dict(fmt=2), INVALID), (dict(n_kv_heads=0), INVALID), (dict(n_pages=0), INVALID), (dict(page_tokens=48), UNSUPPORTED),
         (dict(page_tokens=256), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(n_pages=1 << 32), UNSUPPORTED),
         (dict(k_codes=None), INVALID), (dict(v_scales=None), INVALID), (dict(v_codes=0x2008), MISALIGNED),
         (dict(k_scales=0x3004), MISALIGNED)]
BATCH = [(dict(n_seqs=0), INVALID), (dict(max_new=0), INVALID), (dict(max_len=0), INVALID), (dict(page_stride=0), INVALID),
         (dict(n_seqs=70000), UNSUPPORTED), (dict(max_len=257), INVALID), (dict(max_len=1 << 31, page_stride=1 << 30), UNSUPPORTED),
         (dict(q_start=None), INVALID), (dict(lens=None), INVALID), (dict(pages=None), INVALID), (dict(lens=0x6002), MISALIGNED)]


@pytest.mark.parametrize("over,want", CACHE)
def test_cache_refusals(q, over, want):
    assert attn(q, c=cache(q, **over)) == want
    assert append(q, c=cache(q, **over)) == want


@pytest.mark.parametrize("over,want", BATCH)
def test_batch_refusals(q, over, want):
    assert attn(q, b=batch(q, **over)) == want
    assert append(q, b=batch(q, **over)) == want


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), INVALID), (dict(hq=0), INVALID), (dict(hq=5), INVALID), (dict(hq=2 * 129), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=-1.0), INVALID), (dict(window=-1), INVALID), (dict(qp=None), INVALID), (dict(out=None), INVALID),
    (dict(qp=0x10008), MISALIGNED), (dict(ldq=516), MISALIGNED), (dict(hso=132), MISALIGNED), (dict(hsq=64), INVALID),
    (dict(ldo=64), INVALID), (dict(ws=None), INVALID), (dict(ws=0x30008), MISALIGNED)])
def test_attention_refusals(q, over, want):
    assert attn(q, **over) == want


@pytest.mark.parametrize("over,want", [
    (dict(n=-1), INVALID), (dict(hq=0), INVALID), (dict(qp=None), INVALID), (dict(qp=None, hq=0), INVALID),
    (dict(out=None), INVALID), (dict(hq=-1), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID),
    (dict(kp=0x11002), MISALIGNED), (dict(ldv=260), MISALIGNED), (dict(hsk=8), INVALID), (dict(ldk=8), INVALID),
    (dict(out=0x10000, ldo=1024), INVALID), (dict(ws=None), INVALID), (dict(wsb=255), SMALL), (dict(ws=0x30001), MISALIGNED)])
def test_append_refusals(q, over, want):
    assert append(q, **over) == want


@pytest.mark.parametrize("over,want", [
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(weight_offset=float("inf")), INVALID),
    (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=144), INVALID), (dict(rotary_dim=24), UNSUPPORTED),
    (dict(rotary_dim=0), INVALID), (dict(cos_sin=None), INVALID), (dict(n_positions=199), INVALID),
    (dict(interleaved=2), INVALID), (dict(q_weight=0x8002), MISALIGNED), (dict(cos_sin=0xA004), MISALIGNED)])
def test_norm_rope_refusals(q, over, want):
    assert append(q, nr=norm_rope(q, **over)) == want


def test_nothing_to_do_is_fine_without_pointers(q):
    empty = dict(k_codes=None, v_codes=None, k_scales=None, v_scales=None)
    assert attn(q, c=cache(q, **empty), n=0, qp=None, out=None, ws=None, wsb=0) == 0
    assert append(q, c=cache(q, **empty), n=0, kp=None, vp=None, ws=None, wsb=0) == 0


def test_workspace_sizes(q):
    assert q.qkv_append_workspace_size() == 256
    assert q.qattn_workspace_size(cache(q, head_dim=96), batch(q), 8, 4) == 0
    assert q.qattn_workspace_size(cache(q), batch(q), 8, 5) == 0
    assert q.lib().qattn(None, batch(q), 8, 4, 0x1000, 512, 128, 0.1, 0, 0x2000, 512, 128, 0x3000, 256, None) == INVALID
    assert q.lib().qkv_append(cache(q), None, None, 8, 0, None, 0, 0, 0x1000, 256, 128, 0x1000, 256, 128, None, 0, 0, 0x3000, 256,
                              None) == INVALID


def test_python_helpers_refuse_wrong_tensors(q):
    torch = pytest.importorskip("torch")
    codes, scales = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.ones(4, 2)
    kv = q.KVCache(codes, codes.clone(), scales, scales.clone())
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = q.KVBatch(i32(3), i32(2), i32(2, 2), 1, 32)
    for bad in (lambda: q.KVCache(codes.float(), codes.float(), scales, scales), lambda: q.KVCache(codes, codes, scales[:2], scales),
                lambda: q.KVCache(codes[..., :32], codes[..., :32], scales, scales), lambda: q.KVBatch(i32(2), i32(2), i32(2, 2), 1, 32),
                lambda: q.KVBatch(i32(3).long(), i32(2), i32(2, 2), 1, 32), lambda: q.KVBatch(i32(3), i32(2), i32(3, 2), 1, 32),
                lambda: q.NormRope(torch.ones(64)), lambda: q.NormRope(cos_sin=torch.ones(64)),
                lambda: q.attention(kv, b, torch.zeros(2, 4, 64)), lambda: q.attention(kv, b, torch.zeros(2, 4, 32, dtype=torch.bfloat16)),
                lambda: q.kv_append(kv, b, None, torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16))):
        with pytest.raises(q.QGError) as e:
            bad()
        assert e.value.status == INVALID
    assert isinstance(kv.desc, ctypes.Structure)


def test_attention_in_place_needs_the_same_strides(q):
    for over in (dict(ldo=1024), dict(hso=256, ldo=1024), dict(ldq=1024)):
        assert attn(q, out=0x10000, **over) == INVALID

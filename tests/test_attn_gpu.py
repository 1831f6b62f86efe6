"""Cache append and attention on the GPU against the 64-bit oracle.

Bounds.  Rounding to bf16 costs half a unit of 8 significant bits, 2^-8 of the value at most; to E4M3
2^-4 of it, or half of the subnormal step 2^-9.  The fp32 work before it adds 2^-20 of the largest
term (a few roundings of 2^-24 each, norm and rotation together).  Attention rounds each weight to 11
significant bits (2^-11 of it, or 2^-25 of the largest weight), takes exp2 and the sums in fp32 (2^-11 covers
them) and each score to D roundings of its fp32 sum: a score off by e moves a weight by e of it, and the sum
of weights by as much."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.gpu_util import qlib, to_f64

pytestmark = pytest.mark.gpu


class Case:
    """A cache with the sequences' pages scattered in it; every token slot that no sequence has filled holds NaN
    codes, every unused page NaN scales."""

    def __init__(self, seed, news, lens, page, hkv, d, before=None, spread=0.3, spare=3):
        rng = np.random.default_rng(seed)
        self.rng, self.news, self.lens, self.page, self.hkv, self.d = rng, list(news), list(lens), page, hkv, d
        per = [-(-l // page) for l in lens]
        n_pages = sum(per) + spare
        order = rng.permutation(n_pages)[:sum(per)]
        self.pages = np.full((len(lens), max(per + [1]) + 1), 2 ** 30, np.int32)  # ids out of range where unused
        self.kc = np.where(rng.random((n_pages, hkv, page, d)) < 0.5, 0x7F, 0xFF).astype(np.uint8)
        self.vc = self.kc.copy()
        self.ks, self.vs = (np.full((n_pages, hkv), np.nan, np.float32) for _ in range(2))
        at = 0
        filled = lens if before is None else before  # tokens of each sequence that the cache holds already
        for b, c in enumerate(per):
            self.pages[b, :c] = order[at:at + c]
            at += c
            for i in range(-(-filled[b] // page)):
                pg, n = self.pages[b, i], min(page, filled[b] - i * page)
                for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
                    x = rng.standard_normal((hkv, n, d)) * np.exp(spread * rng.standard_normal((hkv, 1, 1)))
                    scales[pg] = [oa.page_scale(np.abs(x[h]).max()) for h in range(hkv)]
                    codes[pg, :, :n] = oa.e4m3_encode(x / scales[pg][:, None, None])
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.n = int(self.starts[-1])

    def heads(self, h, size=1.0):
        x = torch.from_numpy((self.rng.standard_normal((self.n, h, self.d)) * size).astype(np.float32))
        return x.to(torch.bfloat16)

    def device(self, q, max_new=None, max_len=None):
        t = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        cache = q.KVCache(t(self.kc), t(self.vc), t(self.ks), t(self.vs))
        batch = q.KVBatch(t(self.starts), t(np.array(self.lens, np.int32)), t(self.pages),
                          max_new=max_new or max(self.news + [1]), max_len=max_len or max(self.lens + [1]))
        return cache, batch

    def attention(self, qh, scale, window=0):
        return oa.attention(to_f64(qh.cpu()), self.news, self.lens, self.pages, self.page, self.kc, self.ks, self.vc,
                            self.vs, scale, window)


def attention_bound(ref, d, keys):
    out, mag, load, vmax = ref
    score = 2 * d * 2.0 ** -24 * load
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -10 + 2 * score[..., None]) * mag + keys * 2.0 ** -25 * vmax[..., None] + 1e-30


def check_attention(got, ref, d, keys):
    got = to_f64(got)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - ref[0]) > attention_bound(ref, d, keys)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[0][bad][:5])


def _device_reference(c, qh, window, scale):
    """The oracle's attention in torch float64 on the GPU, for batches too large for loops over rows."""
    from oracle.attention import e4m3_decode
    grid = torch.from_numpy(np.nan_to_num(e4m3_decode(np.arange(256)))).cuda()
    out, mag, load, vmax = (torch.zeros(c.n, qh.shape[1], w, dtype=torch.float64, device="cuda") for w in (c.d, c.d, 1, 1))
    kc, vc = (torch.from_numpy(x).cuda().long() for x in (c.kc, c.vc))
    ks, vs = (torch.from_numpy(np.nan_to_num(x)).cuda().double() for x in (c.ks, c.vs))
    grp = qh.shape[1] // c.hkv
    for b, (t, length) in enumerate(zip(c.news, c.lens)):
        if not t or not length:
            continue
        ids = torch.from_numpy(c.pages[b, :-(-length // c.page)]).cuda().long()
        pos = torch.arange(length - t, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")
        see = (j <= pos) & ((j > pos - window) if window else True)
        k, v = ((grid[x[ids]] * y[ids][..., None, None]).transpose(0, 1).reshape(c.hkv, -1, c.d)[:, :length]
                for x, y in ((kc, ks), (vc, vs)))
        q = qh[c.starts[b]:c.starts[b + 1]].cuda().double().view(t, c.hkv, grp, c.d).permute(1, 2, 0, 3)
        s = torch.matmul(q, k[:, None].transpose(-1, -2)) * scale
        p = torch.softmax(s.masked_fill(~see, -torch.inf), -1)
        r = slice(c.starts[b], c.starts[b + 1])
        put = lambda x: x.permute(2, 0, 1, 3).reshape(t, -1, x.shape[-1])  # noqa: E731
        out[r], mag[r] = put(torch.matmul(p, v[:, None])), put(torch.matmul(p, v.abs()[:, None]))
        load[r] = put((torch.matmul(q.abs(), k.abs()[:, None].transpose(-1, -2)) * scale).amax(-1, keepdim=True))
        vmax[r] = v.abs().amax()
    return out.cpu().numpy(), mag.cpu().numpy(), load[..., 0].cpu().numpy(), vmax[..., 0].cpu().numpy()


# ------------------------------------------------------------------ append
def _table(rot, n):
    if not rot:
        return None
    f = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("d,page,hkv,hq,news,lens,rot,inter,off", [
    (128, 64, 8, 40, [1], [901], 128, False, 0.0),
    (128, 16, 2, 6, [1, 1, 1, 0, 1], [16, 17, 1, 40, 33], 128, True, 0.0),
    (64, 32, 3, 3, [4, 2, 3], [34, 2, 129], 64, True, 1.0),
    (256, 16, 4, 24, [3, 4], [18, 20], 64, False, 1.0),
    (256, 128, 1, 2, [150, 5, 131], [150, 133, 140], 64, False, 0.0),
    (256, 64, 2, 2, [77], [140], 256, False, 0.0),
    (128, 64, 2, 10, [200, 1, 65, 64], [200, 500, 70, 128], 32, False, 0.0),
    (128, 128, 1, 1, [300], [301], 16, True, 0.0),
    (64, 16, 4, 32, [45, 7, 0, 18], [45, 20, 33, 18], 0, False, 0.0),
    (64, 128, 2, 4, [9], [9], 64, False, 0.0),
    (128, 16, 2, 4, [500] + [1] * 70, [500] + list(range(1, 71)), 128, False, 0.0),  # found by the scan
])
def test_append_against_oracle(d, page, hkv, hq, news, lens, rot, inter, off):
    q = qlib()
    c = Case(d + page + sum(news), news, lens, page, hkv, d, before=[l - t for t, l in zip(news, lens)])
    x = torch.cat([c.heads(hq, 2.0), c.heads(hkv, 2.0), c.heads(hkv)], 1).cuda()  # a fused projection's rows
    qh, kh, vh = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    w = [torch.from_numpy((1 - off + 0.2 * c.rng.standard_normal(d)).astype(np.float32)).to(torch.bfloat16) for _ in range(2)]
    cs = _table(rot, max(lens))
    nr = q.NormRope(w[0].cuda(), w[1].cuda(), eps=1e-5, weight_offset=off,
                    cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), interleaved=inter)
    cache, batch = c.device(q)
    ws = q.Workspace(q.qkv_append_workspace_size())
    out = q.kv_append(cache, batch, qh, kh, vh, nr, workspace=ws)
    assert ws.status() == 0
    pos = np.concatenate([np.arange(l - t, l) for t, l in zip(news, lens)])
    nrm = lambda t, wt: np.stack([oa.norm_rope(to_f64(t[i]), to_f64(wt), 1e-5, off, cs, inter, pos[i])  # noqa: E731
                                  for i in range(c.n)])
    ref = nrm(qh, w[0])
    assert np.all(np.abs(to_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.abs(ref).max(-1, keepdims=True))
    for name, new, codes, scales, gc, gs in (("k", nrm(kh, w[1]), c.kc, c.ks, cache.k_codes, cache.k_scales),
                                             ("v", to_f64(vh), c.vc, c.vs, cache.v_codes, cache.v_scales)):
        rc, rs, exact = oa.append(new, news, lens, c.pages, page, codes, scales)
        gc, gs = gc.view(torch.uint8).cpu().numpy(), to_f64(gs)
        assert np.array_equal(gs, rs, equal_nan=True), name
        fresh = ~np.isnan(exact)
        assert np.array_equal(gc[~fresh], rc[~fresh]), name  # older tokens moved alike, everything else untouched
        got = oa.e4m3_decode(gc) * gs[:, :, None, None]
        bound = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10 * gs[:, :, None, None]) + 2.0 ** -20 * np.abs(new).max()
        assert np.all(np.abs(got - exact)[fresh] <= bound[fresh]), name
        assert np.mean(gc[fresh] != rc[fresh]) < 1e-3, name  # flips at ties only


def test_append_token_by_token_equals_the_oracle_chain():
    """Values of growing size: a page's scale grows step after step and its codes move with it."""
    q = qlib()
    c = Case(5, [1], [50], 32, 2, 64, before=[0])
    cache, _ = c.device(q)
    kc, ks, vc, vs = c.kc, c.ks, c.vc, c.vs
    ws = q.Workspace(q.qkv_append_workspace_size())
    for t in range(50):
        kh, vh = c.heads(2, 1.1 ** t).cuda(), c.heads(2, 10.0 * 0.9 ** t).cuda()
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        batch = q.KVBatch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"), lens, torch.from_numpy(c.pages).cuda(), 1, 50)
        assert q.kv_append(cache, batch, None, kh, vh, workspace=ws) is None  # no queries, no norm, no rotation
        kc, ks, _ = oa.append(to_f64(kh), [1], [t + 1], c.pages, 32, kc, ks)
        vc, vs, _ = oa.append(to_f64(vh), [1], [t + 1], c.pages, 32, vc, vs)
    assert ws.status() == 0
    for g, r in ((cache.k_codes, kc), (cache.v_codes, vc)):
        assert np.array_equal(g.view(torch.uint8).cpu().numpy(), r)
    for g, r in ((cache.k_scales, ks), (cache.v_scales, vs)):
        assert np.array_equal(to_f64(g), r, equal_nan=True)


def test_append_special_values_and_in_place_queries():
    q = qlib()
    c = Case(6, [20], [20], 16, 1, 64, before=[0])
    qh, kh, vh = c.heads(3), c.heads(1), c.heads(1)
    kh[2, 0, 3], kh[2, 0, 4], kh[2, 0, 5] = float("inf"), float("-inf"), float("nan")
    vh[16:] = 0.0  # a page of zeros
    cache, batch = c.device(q)
    nr = q.NormRope(torch.ones(64, dtype=torch.bfloat16, device="cuda"), None, eps=0.0)
    qd = qh.cuda()
    out = q.kv_append(cache, batch, qd, kh.cuda(), vh.cuda(), nr, out=qd)
    assert out.data_ptr() == qd.data_ptr()
    ref = np.stack([oa.norm_rope(to_f64(x), np.ones(64), 0, 0, None, False, 0) for x in qh])
    assert np.all(np.abs(to_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * np.abs(ref).max())
    rc, rs, _ = oa.append(to_f64(kh), [20], [20], c.pages, 16, c.kc, c.ks)
    g = cache.k_codes.view(torch.uint8).cpu().numpy()
    nan = np.isnan(oa.e4m3_decode(rc))
    assert np.array_equal(np.isnan(oa.e4m3_decode(g)), nan) and np.array_equal(g[~nan], rc[~nan])
    assert np.array_equal(to_f64(cache.k_scales), rs, equal_nan=True)
    pg = c.pages[0, 1]
    assert float(cache.v_scales[pg, 0]) == 2.0 ** -100 and not cache.v_codes[pg, 0, :4].float().any()


# ------------------------------------------------------------------ attention
SHAPES = [
    # d, page, hkv, hq, news, lens, window
    (128, 64, 8, 40, [1], [777], 0),
    (128, 32, 2, 10, [1, 1, 1, 1], [1, 33, 4000, 129], 0),
    (256, 64, 4, 24, [1], [6001], 0),
    (256, 16, 1, 16, [1, 1], [17, 600], 0),
    (64, 16, 4, 32, [1, 0, 1], [1000, 77, 15], 100),
    (64, 128, 1, 7, [2, 2], [300, 2], 0),
    (128, 128, 2, 6, [4, 3, 1], [4, 500, 257], 64),
    (256, 64, 4, 24, [4, 4, 4], [900, 4, 2000], 0),
    (128, 64, 1, 1, [1], [3000], 0),
    (128, 16, 2, 34, [3, 2], [100, 2], 0),
    (64, 32, 2, 2, [5, 61, 1], [5, 400, 1], 0),
    (128, 64, 2, 10, [300], [300], 0),
    (128, 64, 2, 8, [129, 64], [1000, 64], 0),
    (128, 16, 1, 5, [77, 130, 20], [77, 131, 500], 50),
    (64, 16, 2, 16, [260, 33], [260, 700], 1),
    (256, 64, 2, 12, [140], [700], 0),
    (256, 32, 1, 3, [257, 1, 90], [257, 1200, 91], 200),
    (128, 128, 1, 128, [3], [300], 0),
    (64, 64, 1, 48, [1, 6], [65, 130], 0),
]


@pytest.mark.parametrize("d,page,hkv,hq,news,lens,window", SHAPES)
def test_attention_against_oracle(d, page, hkv, hq, news, lens, window):
    q = qlib()
    c = Case(7 * d + page + hq, news, lens, page, hkv, d)
    qh = c.heads(hq, 2.0)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    qd = qh.cuda()
    got = q.attention(cache, batch, qd, window=window, workspace=ws)
    assert ws.status() == 0
    check_attention(got, c.attention(qh, d ** -0.5, window), d, max(lens))
    assert torch.equal(got, q.attention(cache, batch, qd, window=window, workspace=ws))  # again, bit for bit
    loose = c.device(q, max_new=max(news) + 300, max_len=(c.pages.shape[1]) * page)[1]  # looser bounds
    check_attention(q.attention(cache, loose, qd, window=window), c.attention(qh, d ** -0.5, window), d, max(lens))


@pytest.mark.parametrize("d,hkv,hq,page,new,most", [(128, 4, 20, 32, 1, 900), (64, 4, 32, 16, 1, 500), (256, 2, 12, 64, 2, 700),
                                                    (128, 8, 8, 64, 3, 6000), (64, 2, 40, 128, 3, 3000), (256, 4, 4, 16, 1, 5000)])
def test_many_sequences_of_all_lengths(d, hkv, hq, page, new, most):
    """More work than CTAs: pairs of fewer tiles than a CTA works on at once, rings that go round, pairs cut between
    CTAs.  Every one of many calls gives the same bits."""
    q = qlib()
    rng = np.random.default_rng(most)
    lens = [int(x) for x in np.exp(rng.uniform(np.log(new), np.log(most), 96))] + [most, new]
    c = Case(most, [new if i % 7 else 0 for i in range(len(lens))], lens, page, hkv, d)
    qh = c.heads(hq, 2.0)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    qd = qh.cuda()
    first = q.attention(cache, batch, qd, workspace=ws).clone()
    check_attention(first, _device_reference(c, qh, 0, d ** -0.5), d, most)
    outs = [q.attention(cache, batch, qd, workspace=ws) for _ in range(200)]
    assert ws.status() == 0
    assert all(torch.equal(first, o) for o in outs)


@pytest.mark.parametrize("d,hkv,hq,page,news,lens,window", [
    (128, 8, 40, 64, [1500, 300, 1, 700], [1500, 4000, 900, 701], 0), (256, 4, 24, 16, [600, 20], [5000, 20], 0),
    (64, 4, 32, 32, [999, 1200, 64], [1000, 1500, 3000], 700)])
def test_long_prompts(d, hkv, hq, page, news, lens, window):
    q = qlib()
    c = Case(sum(news), news, lens, page, hkv, d)
    qh = c.heads(hq, 2.0)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    qd = qh.cuda()
    first = q.attention(cache, batch, qd, window=window, workspace=ws).clone()
    check_attention(first, _device_reference(c, qh, window, d ** -0.5), d, max(lens))
    outs = [q.attention(cache, batch, qd, window=window, workspace=ws) for _ in range(50)]
    assert ws.status() == 0
    assert all(torch.equal(first, o) for o in outs)


@pytest.mark.parametrize("news,lens", [([1, 1], [300, 40]), ([150], [400])])
@pytest.mark.parametrize("layout", ["fused", "head_major", "padded"])
def test_attention_strides(news, lens, layout):
    q = qlib()
    d, hkv, hq = 128, 2, 6
    c = Case(11, news, lens, 32, hkv, d)
    qh = c.heads(hq)
    if layout == "fused":
        qd = torch.cat([qh, c.heads(2 * hkv)], 1).cuda()[:, :hq]
        out = torch.full((c.n, hq, 2 * d), 3.0, dtype=torch.bfloat16, device="cuda")[..., d:]
    elif layout == "head_major":
        qd = qh.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        out = torch.empty(hq, c.n, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    else:
        qd = torch.zeros(c.n, hq + 1, d + 8, dtype=torch.bfloat16, device="cuda")[:, :hq, :d]
        qd.copy_(qh)
        out = torch.empty(c.n, hq, d + 8, dtype=torch.bfloat16, device="cuda")[..., :d]
    cache, batch = c.device(q)
    got = q.attention(cache, batch, qd, scale=0.2, out=out)
    assert got is out
    check_attention(out, c.attention(qh, 0.2), d, max(lens))
    if layout == "fused":
        assert bool((out.as_strided((c.n, hq, d), out.stride(), 0) == 3.0).all())  # the other half stays


@pytest.mark.parametrize("news,lens", [([4, 1, 3], [2, 0, 3]), ([70, 40], [50, 0])])
def test_rows_that_see_nothing_are_zero(news, lens):
    q = qlib()
    c = Case(12, news, lens, 16, 2, 64)
    qh = c.heads(4)
    cache, batch = c.device(q)
    got = q.attention(cache, batch, qh.cuda(), out=torch.full((c.n, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda"))
    ref = c.attention(qh, 64 ** -0.5)
    check_attention(got, ref, 64, 50)
    empty = np.concatenate([np.arange(l - t, l) < 0 for t, l in zip(news, lens)])
    assert empty.any() and not to_f64(got)[empty].any()


@pytest.mark.parametrize("news,lens", [([1, 1], [500, 90]), ([100], [260])])
def test_attention_extreme_scales(news, lens):
    """Value scales 2^70 apart, queries of 2^60 and of 2^-60 (bf16's range, not fp16's)."""
    q = qlib()
    c = Case(13, news, lens, 16, 2, 128)
    f = np.exp2(c.rng.integers(-50, 21, c.vs.shape)).astype(np.float32)
    c.vs *= f
    qh = c.heads(4)
    cache, batch = c.device(q)
    check_attention(q.attention(cache, batch, qh.cuda()), c.attention(qh, 128 ** -0.5), 128, 500)
    for e in (60, -60):
        big = (qh.float() * 2.0 ** e).to(torch.bfloat16)
        scale = 128 ** -0.5 * 2.0 ** -e
        check_attention(q.attention(cache, batch, big.cuda(), scale=scale), c.attention(big, scale), 128, 500)
    tiny = (qh.float() * 2.0 ** -100).to(torch.bfloat16)  # scores near zero: an even mean
    check_attention(q.attention(cache, batch, tiny.cuda()), c.attention(tiny, 128 ** -0.5), 128, 500)
    zero = torch.zeros_like(qh)
    check_attention(q.attention(cache, batch, zero.cuda()), c.attention(zero, 128 ** -0.5), 128, 500)


@pytest.mark.parametrize("news,lens", [([1, 1, 1], [200, 90, 40]), ([100, 30, 20], [260, 40, 20])])
def test_bad_device_data_is_reported_and_skipped(news, lens):
    q = qlib()
    d, hq = 128, 4
    for kind in ("page", "length", "rows"):
        c = Case(14, news, lens, 16, 2, d)
        qh = c.heads(hq)
        cache, batch = c.device(q)
        if kind == "page":
            batch.pages[1, 0] = 2 ** 31 - 1
        elif kind == "length":
            batch.lens[1] = 10 ** 9
        else:
            batch.q_start[3] = c.n + 1000  # the last sequence's rows would pass the end
        ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
        got = q.attention(cache, batch, qh.cuda(), workspace=ws)
        assert ws.status() == 1 and ws.status() == 0  # reported once, cleared by the read
        ref = c.attention(qh, d ** -0.5)
        b = 2 if kind == "rows" else 1
        keep = np.ones(c.n, bool)
        keep[c.starts[b]:c.starts[b + 1]] = False
        check_attention(got[torch.from_numpy(keep).cuda()], [r[keep] for r in ref], d, 260)
        ap = q.Workspace(q.qkv_append_workspace_size())
        before = cache.k_codes.view(torch.uint8).clone()
        q.kv_append(cache, batch, qh.cuda(), c.heads(2).cuda(), c.heads(2).cuda(), workspace=ap)
        assert ap.status() == (1 if kind != "page" or news[0] > 1 and lens[1] - news[1] < 16 else 0)
        if kind == "length":  # the skipped sequence's pages are as they were
            own = [int(p) for p in c.pages[1][:-(-lens[1] // 16)]]
            assert torch.equal(cache.k_codes.view(torch.uint8)[own], before[own])


def test_no_rows_and_no_keys():
    q = qlib()
    c = Case(15, [0, 0], [30, 0], 16, 1, 64)
    cache, batch = c.device(q)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert q.attention(cache, batch, e).shape == (0, 2, 64)
    assert q.kv_append(cache, batch, e, e[:, :1], e[:, :1]).shape == (0, 2, 64)


def test_cache_beyond_4_gib():
    q = qlib()
    hkv, page, d, n_pages = 8, 128, 256, 17000  # 4.4e9 bytes of codes each
    kc, vc = (torch.zeros(n_pages, hkv, page, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(n_pages, hkv, device="cuda") for _ in range(2))
    cache = q.KVCache(kc, vc, ks, vs)
    rng = np.random.default_rng(16)
    lens = [200]
    ids = np.array([[n_pages - 1, n_pages - 2]], np.int32)
    x = [torch.from_numpy(rng.standard_normal((200, h, d)).astype(np.float32)).to(torch.bfloat16).cuda() for h in (8, hkv, hkv)]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = q.KVBatch(t([0, 200]), t(lens), t(ids), 200, 200)
    q.kv_append(cache, batch, None, x[1], x[2])
    tail = [a[-2:].cpu().numpy() for a in (kc, ks, vc, vs)]
    rc, rs, _ = oa.append(to_f64(x[1]), [200], lens, [[1, 0]], page, np.zeros_like(tail[0]), np.ones_like(tail[1]))
    assert np.array_equal(tail[0], rc) and np.array_equal(tail[1], rs)
    for rows in (1, 30):
        b = q.KVBatch(t([0, rows]), t(lens), t(ids), rows, 200)
        got = q.attention(cache, b, x[0][:rows])
        ref = oa.attention(to_f64(x[0][:rows]), [rows], lens, [[1, 0]], page, *tail, d ** -0.5)
        check_attention(got, ref, d, 200)


def test_prompt_then_decode_on_another_stream():
    """A prompt and three decoded tokens through both operators on a stream of the caller's, one workspace each."""
    q = qlib()
    d, hkv, hq, page = 128, 2, 8, 32
    c = Case(17, [70], [73], page, hkv, d, before=[0])
    cs = _table(64, 80)
    s = torch.cuda.Stream()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    nr = q.NormRope(w, w, cos_sin=torch.from_numpy(cs).cuda())
    cache, _ = c.device(q)
    pages = torch.from_numpy(c.pages).cuda()
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batches = [q.KVBatch(t([0, n]), t([l]), pages, n, 73) for n, l in [(70, 70), (1, 71), (1, 72), (1, 73)]]
    xs = [[torch.from_numpy(c.rng.standard_normal((b.max_new, h, d)).astype(np.float32)).to(torch.bfloat16).cuda()
           for h in (hq, hkv, hkv)] for b in batches]
    ws = q.Workspace(max(q.attention_workspace_size(cache, b, b.max_new, hq) for b in batches))
    wa = q.Workspace(q.qkv_append_workspace_size())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        steps = []
        for b, (qh, kh, vh) in zip(batches, xs):
            qn = q.kv_append(cache, b, qh, kh, vh, nr, workspace=wa)
            steps.append((qn, q.attention(cache, b, qn, workspace=ws), *(a.clone() for a in (cache.k_codes, cache.k_scales,
                                                                                              cache.v_codes, cache.v_scales))))
    s.synchronize()
    for (qn, out, *state), n, l in zip(steps, (70, 1, 1, 1), (70, 71, 72, 73)):
        kc, ks, vc, vs = (a.view(torch.uint8).cpu().numpy() if a.dtype != torch.float32 else a.cpu().numpy() for a in state)
        check_attention(out, oa.attention(to_f64(qn), [n], [l], c.pages, page, kc, ks, vc, vs, d ** -0.5), d, 73)


NAN_SHAPES = [  # d, page, hkv, hq, news, lens, window: few rows a KV head, then row blocks, whole and cut along the keys
    (128, 16, 2, 6, [4, 1, 3], [300, 90, 5], 0), (64, 32, 2, 8, [2, 1], [150, 400], 40), (256, 64, 1, 4, [5, 1], [200, 77], 33),
    (128, 64, 2, 4, [3], [6000], 0), (256, 16, 2, 6, [1], [700], 300),
    (64, 16, 2, 4, [150, 90], [400, 90], 0), (128, 32, 2, 8, [70, 100], [300, 101], 37), (256, 64, 1, 2, [130], [333], 50),
    (128, 64, 1, 4, [100], [5000], 0)]


@pytest.mark.parametrize("d,page,hkv,hq,news,lens,window", NAN_SHAPES)
def test_nan_values_reach_only_rows_that_see_them(d, page, hkv, hq, news, lens, window):
    q = qlib()
    c = Case(d + sum(lens), news, lens, page, hkv, d)
    qh = c.heads(hq)
    clean = c.attention(qh, d ** -0.5, window)
    for b, (t, length) in enumerate(zip(news, lens)):
        for at in {length - 1, length - t + t // 2, length - t, max(0, length - window - 2 * (t // 3)) if window else length // 2}:
            pg, h = c.pages[b, at // page], int(c.rng.integers(hkv))
            c.vc[pg, h, at % page, c.rng.integers(0, d, 3)] = c.rng.choice([0x7F, 0xFF], 3)
    nan = np.isnan(c.attention(qh, d ** -0.5, window)[0])
    assert nan.any() and not nan.all()
    cache, batch = c.device(q)
    got = to_f64(q.attention(cache, batch, qh.cuda(), window=window))
    assert np.array_equal(np.isnan(got), nan)
    # (the other dims' exact values are those without the NaN codes)
    check_attention(torch.from_numpy(np.where(nan, clean[0], got)), clean, d, max(lens))


@pytest.mark.parametrize("d,page,hkv,hq,news,lens,window", NAN_SHAPES)
def test_nan_scores_stay_in_their_rows(d, page, hkv, hq, news, lens, window):
    """NaN key codes, and query rows with a NaN or an infinity: NaN where the formula has it, nowhere else."""
    q = qlib()
    c = Case(d + sum(lens) + 1, news, lens, page, hkv, d)
    qh = c.heads(hq)
    clean = c.attention(qh, d ** -0.5, window)
    row = 0
    for b, (t, length) in enumerate(zip(news, lens)):
        if t > 1:
            at = length - t + t // 2
            c.kc[c.pages[b, at // page], 0, at % page, int(c.rng.integers(d))] = 0x7F
            qh[row, hq - 1, int(c.rng.integers(d))] = float("inf")
        elif window == 0 or length > window:
            qh[row, 0, 1] = float("nan")
            qh[row, hq - 1, 3] = float("-inf")
        row += t
    with np.errstate(invalid="ignore"):
        nan = np.isnan(c.attention(qh, d ** -0.5, window)[0])
    assert nan.any() and not nan.all()
    cache, batch = c.device(q)
    got = to_f64(q.attention(cache, batch, qh.cuda(), window=window))
    assert np.array_equal(np.isnan(got), nan)
    check_attention(torch.from_numpy(np.where(nan, clean[0], got)), clean, d, max(lens))


@pytest.mark.parametrize("d,hkv,hq,page,new,most,window", [(128, 4, 28, 32, 3, 900, 0), (64, 4, 32, 16, 4, 1100, 0), (256, 4, 24, 64, 4, 800, 0),
                                                           (128, 8, 40, 64, 5, 2500, 300), (256, 8, 56, 16, 4, 700, 150)])
def test_many_sequences_of_17_to_32_rows(d, hkv, hq, page, new, most, window):
    """Enough keys for the streaming kernel at these rows (2^18 over all pairs), windows that begin inside pages, and NaN
    value codes in the first and the last new token's places."""
    q = qlib()
    rng = np.random.default_rng(most + d)
    lens = [int(x) for x in np.exp(rng.uniform(np.log(new), np.log(most), 96))] + [most, new]
    assert 16 < new * hq // hkv <= 32 and len(lens) * hkv * most >= 1 << 18
    c = Case(most + d, [new if i % 7 else 0 for i in range(len(lens))], lens, page, hkv, d)
    qh = c.heads(hq)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    qd = qh.cuda()
    first = q.attention(cache, batch, qd, window=window, workspace=ws).clone()
    ref = _device_reference(c, qh, window, d ** -0.5)
    check_attention(first, ref, d, most)
    outs = [q.attention(cache, batch, qd, window=window, workspace=ws) for _ in range(100)]
    assert ws.status() == 0
    assert all(torch.equal(first, o) for o in outs)
    # a NaN dim in the last new token (its row alone sees it) and, under a window, in the key that only the first row sees
    nan = np.zeros((c.n, hq, d), bool)
    grp = hq // hkv
    for b, (t, length) in enumerate(zip(c.news, c.lens)):
        if not t:
            continue
        h, dim, r = b % hkv, (17 * b) % d, c.starts[b]
        for at, row in [(length - 1, r + t - 1)] + ([(length - t - window + 1, r)] if window and length - t - window + 1 >= 0 else []):
            c.vc[c.pages[b, at // page], h, at % page, dim] = 0x7F
            nan[row, h * grp:(h + 1) * grp, dim] = True
    cache = c.device(q)[0]
    got = to_f64(q.attention(cache, batch, qd, window=window))
    assert np.array_equal(np.isnan(got), nan)
    check_attention(torch.from_numpy(np.where(nan, ref[0], got)), ref, d, most)

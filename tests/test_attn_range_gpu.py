"""Attention over the 8-bit paged cache where its numbers lie far apart, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.gpu_util import qlib, to_f64
from tests.test_attn_gpu import Case, check_attention

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ one key far above many
def _sink(d, hkv, hq, new, length, gap, value, noise, seed):
    """Keys whose scores lie `gap` (natural logarithms) below the first one's, give or take `noise`; values of about 1
    but for the first key's."""
    rng = np.random.default_rng(seed)
    page = 128
    shape = (-(-length // page), hkv, page, d)
    k = noise * rng.standard_normal(shape)
    k[..., 0] = 0.0
    v = 1.0 + 0.125 * rng.integers(-1, 2, shape)
    k[0, :, 0], v[0, :, 0] = 0.0, value
    k[0, :, 0, 0] = 8.0
    x = rng.standard_normal((new, hq, d))
    x[..., 0] = 16.0
    ones = np.ones(shape[:2], np.float32)
    return page, oa.e4m3_encode(k), oa.e4m3_encode(v), ones, torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16), gap / 128


def _check_sink(d, hkv, hq, new, n_seqs, length, gap, value, noise, floor):
    """Many sequences over the same pages, so that most pairs of a sequence and a KV head stay in one CTA.  Bound: 2^-8 of the
    output for bf16, 2^-10 of the weighted sum of magnitudes for a weight's 11 bits (and exp2, sums), 2 d fp32 roundings
    of a score, and `floor` of the largest weight for each key."""
    q = qlib()
    page, kc, vc, ones, x, scale = _sink(d, hkv, hq, new, length, gap, value, noise, 1000 * new + d)
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    ids = np.random.default_rng(1).permutation(len(kc)).astype(np.int32)
    place = np.argsort(ids)  # page i of the pool holds the sequence's page place[i]
    cache = q.KVCache(t(kc[place]), t(vc[place]), t(ones), t(ones.copy()))
    pages = t(np.tile(ids, (n_seqs, 1)))
    batch = q.KVBatch(torch.arange(0, n_seqs * new + 1, new, dtype=torch.int32, device="cuda"),
                      torch.full((n_seqs,), length, dtype=torch.int32, device="cuda"), pages, new, length)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, n_seqs * new, hq))
    got = q.attention(cache, batch, x.repeat(n_seqs, 1, 1).cuda(), scale, workspace=ws)
    assert ws.status() == 0
    out, mag, load, vmax = oa.attention(to_f64(x), [new], [length], [list(range(len(kc)))], page, kc, ones, vc, ones, scale)
    bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -10 + 4 * d * 2.0 ** -24 * load[..., None]) * mag + length * floor * vmax[..., None]
    err = np.abs(to_f64(got).reshape(n_seqs, new, hq, d) - out)
    assert np.all(err <= bound), (err.max(), bound[np.unravel_index(err.argmax(), err.shape)[1:]], out.flat[:3])


@pytest.mark.parametrize("d,hkv,hq,new,n_seqs,length,gap,value,noise", [
    (128, 4, 20, 1, 152, 20001, 14.5, 0.0, 0.0), (64, 4, 64, 1, 100, 20001, 13.0, -1.0, 0.05), (256, 2, 12, 1, 152, 20001, 14.5, 0.0, 0.05),
    (64, 1, 8, 1, 304, 130001, 16.0, -1.0, 0.0), (128, 2, 10, 5, 152, 20001, 14.5, 0.0, 0.0), (256, 2, 12, 4, 152, 20001, 13.5, -1.0, 0.0),
    (64, 2, 16, 3, 152, 30001, 15.0, 0.0, 0.05), (128, 1, 4, 2, 1, 20001, 17.0, 0.0, 0.0)])
def test_weights_far_below_the_largest_streaming(d, hkv, hq, new, n_seqs, length, gap, value, noise):
    # P is 2^6 or more at the largest weight and off by 2^-19 at most
    _check_sink(d, hkv, hq, new, n_seqs, length, gap, value, noise, 2.0 ** -25)


@pytest.mark.parametrize("d,hkv,hq,new,n_seqs,length,gap,value,noise", [
    (128, 2, 8, 40, 8, 20001, 14.5, 0.0, 0.0), (64, 1, 16, 20, 160, 20001, 14.5, -1.0, 0.0), (256, 1, 6, 50, 2, 20001, 13.0, 0.0, 0.0),
    (128, 1, 8, 33, 1, 60001, 16.0, 0.0, 0.0)])
def test_weights_far_below_the_largest_row_blocks(d, hkv, hq, new, n_seqs, length, gap, value, noise):
    # P is 2^7 or more at the largest weight, in fp16: off by 2^-25 at most
    _check_sink(d, hkv, hq, new, n_seqs, length, gap, value, noise, 2.0 ** -32)


# ------------------------------------------------------------------ pages whose key scale is 0
@pytest.mark.parametrize("d,page,hkv,hq,news,lens,window", [
    (128, 64, 2, 10, [1, 1], [900, 300], 0), (64, 16, 4, 32, [1, 2], [1000, 400], 0), (256, 128, 1, 6, [2, 1], [1200, 640], 0),
    (128, 32, 2, 6, [1], [5000], 700), (64, 128, 1, 4, [1, 1], [128, 700], 0),
    (128, 64, 2, 10, [300, 2], [900, 640], 0), (64, 16, 2, 16, [100, 260], [700, 1000], 0), (256, 128, 1, 6, [150], [1200], 0),
    (128, 32, 1, 8, [40], [6000], 900), (128, 128, 1, 64, [3], [700], 0)])
def test_pages_of_key_scale_zero_do_not_enter(d, page, hkv, hq, news, lens, window):
    """Inner pages too, with NaN codes in them, a value scale of 1, 0 or NaN; and a sequence of no other pages."""
    q = qlib()
    c = Case(d + page + sum(lens) + 2, news, lens, page, hkv, d)
    for b, length in enumerate(lens):
        for i in range(-(-length // page)):
            if i % 3 == 1 or b == 1 and len(lens) > 1 and i < 2:
                h = c.rng.integers(hkv)
                c.ks[c.pages[b, i], h], c.vs[c.pages[b, i], h] = 0.0, [1.0, 0.0, np.nan][i % 9 // 3]
                for codes in (c.kc, c.vc):
                    codes[c.pages[b, i], h, :, ::5] = 0x7F
    _check_hidden(q, c, hq, window)
    c.ks[c.pages[0, :-(-lens[0] // page)]] = 0.0
    got = _check_hidden(q, c, hq, window)
    assert not to_f64(got)[:news[0]].any()


def _check_hidden(q, c, hq, window):
    qh = c.heads(hq, 2.0)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    got = q.attention(cache, batch, qh.cuda(), window=window, workspace=ws)
    assert ws.status() == 0
    check_attention(got, c.attention(qh, c.d ** -0.5, window), c.d, max(c.lens))
    return got


@pytest.mark.parametrize("d,hkv,hq,page,new", [(128, 4, 24, 32, 4), (256, 4, 32, 16, 3), (64, 4, 40, 128, 2)])
def test_pages_of_key_scale_zero_17_to_32_rows(d, hkv, hq, page, new):
    q = qlib()
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(new, 701, 97)] + [701]
    assert 16 < new * hq // hkv <= 32 and len(lens) * hkv * max(lens) >= 1 << 18  # the streaming kernel
    c = Case(d + page, [new] * len(lens), lens, page, hkv, d)
    for b, length in enumerate(lens):
        for i in range(b % 3, -(-length // page), 3):
            c.ks[c.pages[b, i], b % hkv] = 0.0
            c.vc[c.pages[b, i], b % hkv, :, 3::7] = 0xFF
    _check_hidden(q, c, hq, 0)


# ------------------------------------------------------------------ queries with a channel far above the others
@pytest.mark.parametrize("d,page,hkv,hq,news,lens", [
    (128, 64, 2, 10, [1, 1], [900, 300]), (64, 16, 1, 8, [2], [500]), (256, 32, 1, 6, [4], [700]),
    (128, 64, 2, 8, [100], [700]), (64, 32, 1, 16, [60], [500]), (256, 64, 1, 4, [70], [400])])
@pytest.mark.parametrize("size", [64.0, 512.0, 2048.0, 65536.0])
def test_queries_with_outlier_channels(d, page, hkv, hq, news, lens, size):
    """Keys are small in those channels.  An element of 2^-13 of its row's largest or more is exact, a smaller one off by 2^-21
    of the largest at most; the scores' bound takes that beside their fp32 roundings."""
    q = qlib()
    c = Case(d + int(size), news, lens, page, hkv, d)
    out = c.rng.integers(0, d, 2)
    k = oa.e4m3_decode(c.kc[..., out])
    c.kc[..., out] = np.where(np.isnan(k), c.kc[..., out], oa.e4m3_encode(np.nan_to_num(k) / size))
    qh = c.heads(hq)
    qh[..., out] = (size * (1 + torch.from_numpy(c.rng.random((c.n, hq, 2))))).to(torch.bfloat16)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    got = q.attention(cache, batch, qh.cuda(), scale=2 * d ** -0.5, workspace=ws)
    assert ws.status() == 0
    ref = list(c.attention(qh, 2 * d ** -0.5))
    x = np.abs(to_f64(qh))
    top = x.max(-1, keepdims=True)
    off = torch.from_numpy(np.where(x < top * 2.0 ** -13, top * 2.0 ** -21, 0.0)).float()
    ref[2] = ref[2] + c.attention(off, 2 * d ** -0.5)[2] / (2 * d * 2.0 ** -24)  # (attention_bound's factor of it)
    check_attention(got, ref, d, max(lens))


# ------------------------------------------------------------------ statuses
def test_a_bad_batch_does_not_hide_a_wait_that_gave_up():
    q = qlib()
    c = Case(21, [1], [40], 16, 1, 64)
    cache, batch = c.device(q)
    batch.pages[0, 0] = 2 ** 31 - 1
    qh = c.heads(2).cuda()
    ws = q.Workspace(q.attention_workspace_size(cache, batch, 1, 2))
    for call in (lambda: q.attention(cache, batch, qh, workspace=ws),
                 lambda: q.kv_append(cache, q.KVBatch(batch.q_start, batch.lens, batch.pages, 1, 8), qh, qh[:, :1], qh[:, :1], workspace=ws)):
        q.qg_selftest_wait_timeout(ws.ptr, ws.nbytes, torch.cuda.current_stream().cuda_stream)
        call()
        assert q.STATUS[ws.status()] == "QG_ERR_TIMEOUT"
        call()
        assert q.STATUS[ws.status()] == "QG_ERR_INVALID_ARG"


# ------------------------------------------------------------------ in place
@pytest.mark.parametrize("d,hkv,hq,page,news,lens", [
    (128, 2, 10, 64, [1] * 40, [1000 + 50 * i for i in range(40)]), (256, 4, 24, 64, [4], [6000]), (64, 4, 8, 32, [1, 1], [70, 5]),
    (128, 2, 8, 64, [300, 70], [900, 70]), (256, 1, 6, 32, [60], [5000]), (64, 2, 16, 16, [200, 1], [201, 600])])
def test_attention_over_its_own_queries(d, hkv, hq, page, news, lens):
    q = qlib()
    c = Case(sum(lens), news, lens, page, hkv, d)
    qh = c.heads(hq).cuda()
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    want = q.attention(cache, batch, qh, workspace=ws)
    fused = torch.cat([qh, torch.full((c.n, 2 * hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")], 1)
    got = q.attention(cache, batch, fused[:, :hq], out=fused[:, :hq], workspace=ws)
    assert ws.status() == 0 and torch.equal(got, want) and bool((fused[:, hq:] == 3.0).all())


# ------------------------------------------------------------------ page scales at the ends of their range
@pytest.mark.parametrize("d,page,hkv,hq,news,lens", [
    (128, 16, 2, 6, [1, 1], [500, 90]), (256, 64, 1, 6, [4], [700]), (64, 16, 2, 16, [100, 30], [260, 1000]),
    (256, 32, 1, 4, [70], [3000]), (128, 32, 1, 5, [40], [3000])])
@pytest.mark.parametrize("ends", ["low", "high", "apart"])
def test_scales_at_both_ends(d, page, hkv, hq, news, lens, ends):
    """Value scales of 2^-100, of 2^120, and 2^100 apart (pages of zeros beside others); key scales likewise, with queries
    to match."""
    q = qlib()
    c = Case(d + sum(lens), news, lens, page, hkv, d)
    small = lambda codes: np.where(np.isnan(oa.e4m3_decode(codes)), codes, oa.e4m3_encode(np.nan_to_num(oa.e4m3_decode(codes)) / 64))  # noqa: E731
    qh, scale = c.heads(hq), d ** -0.5
    if ends == "low":
        c.ks *= np.float32(2.0 ** -90)
        c.vs[:] = 2.0 ** -100
        scale *= 2.0 ** 90
    elif ends == "high":
        c.ks *= np.float32(2.0 ** 120)
        c.vc = small(c.vc)  # so that the outputs are finite
        c.vs[:] = 2.0 ** 120
        qh = (qh.float() * 2.0 ** -100).to(torch.bfloat16)
        scale *= 2.0 ** -20
    else:
        dead = c.rng.random(c.vs.shape) < 0.5
        c.vs[dead] = 2.0 ** -100
        c.vc[dead] = np.where(np.isnan(oa.e4m3_decode(c.vc[dead])), c.vc[dead], 0)
    cache, batch = c.device(q)
    ws = q.Workspace(q.attention_workspace_size(cache, batch, c.n, hq))
    got = q.attention(cache, batch, qh.cuda(), scale=scale, workspace=ws)
    assert ws.status() == 0
    ref = c.attention(qh, scale)
    assert np.abs(ref[0]).max() < 2.0 ** 127 and np.abs(ref[0]).max() > 0
    check_attention(got, ref, d, max(lens))


# ------------------------------------------------------------------ NaN values of no weight
@pytest.mark.parametrize("d,hkv,hq,new,n_seqs,length", [
    (128, 2, 10, 1, 1, 20001), (256, 1, 6, 4, 1, 20001), (64, 1, 8, 1, 200, 2001), (128, 1, 16, 2, 160, 3001), (64, 1, 16, 20, 1, 20001),
    (256, 1, 6, 40, 40, 3001)])
def test_nan_values_of_no_weight(d, hkv, hq, new, n_seqs, length):
    """A key 150 nats above all others, whose weights are 0 in fp32: a NaN value code among them is a NaN in its dim all the
    same, wherever the work is cut between the two keys."""
    q = qlib()
    page, kc, vc, ones, x, scale = _sink(d, hkv, hq, new, length, 150.0, 0.5, 0.0, d + new)
    rng = np.random.default_rng(new)
    dims = rng.permutation(d)[:12]
    for i, dim in enumerate(dims):
        at = (length - new) * (i + 1) // 13  # (a key that every row sees)
        vc[at // page, :, at % page, dim] = 0x7F
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    cache = q.KVCache(t(kc), t(vc), t(ones), t(ones.copy()))
    batch = q.KVBatch(torch.arange(0, n_seqs * new + 1, new, dtype=torch.int32, device="cuda"),
                      torch.full((n_seqs,), length, dtype=torch.int32, device="cuda"),
                      t(np.tile(np.arange(len(kc), dtype=np.int32), (n_seqs, 1))), new, length)
    got = to_f64(q.attention(cache, batch, x.repeat(n_seqs, 1, 1).cuda(), scale))
    want = np.full(d, 0.5)
    want[dims] = np.nan
    assert np.array_equal(got, np.broadcast_to(want, got.shape), equal_nan=True)

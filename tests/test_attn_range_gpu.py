"""Attention over the 8-bit paged cache where its numbers lie far apart, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.gpu_util import qlib, to_f64

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

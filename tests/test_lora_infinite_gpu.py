"""Adapters with infinite elements, and h beyond bf16's largest number: infinite and NaN outputs are the formula's.

Finite outputs are within the tolerance of the adapters' other tests: h in (k / 16 + 64) steps of 2^-23 and two bf16 terms (2^-16), the second
product in (max_rank / 8 + 4) steps of 2^-23, the output 2^-8."""
import numpy as np
import pytest
import torch

from oracle import layer as ol
from tests.gpu_util import qlib, to_f64
from tests.test_lora_gpu import rows

pytestmark = pytest.mark.gpu

INF = float("inf")


def compare(q, ad, ids, x, y):
    with np.errstate(all="ignore"):
        a, b, sc = to_f64(ad.a), to_f64(ad.b), to_f64(ad.scales)
        want, h, mag = ol.lora(ids, to_f64(x), to_f64(y), a, b, sc, [a.shape[1]] * len(a))
    got = to_f64(q.lora(ad, torch.tensor(ids, dtype=torch.int32, device="cuda"), x, y, out=torch.empty_like(y)))
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:5]
    wide = np.isinf(want)
    assert np.array_equal(got[wide], want[wide]) and not np.isinf(got[~wide]).any()
    steps = (a.shape[1] / 8 + 4) * 2.0 ** -23
    eh = ((ad.k / 16 + 64) * 2.0 ** -23 + 2.0 ** -16 + steps) * mag
    for i, e in enumerate(ids):
        fine = np.isfinite(want[i])
        share = steps * np.abs(to_f64(y[i]))
        if e >= 0:
            share = share + sc[e] * np.abs(np.where(np.isfinite(b[e]), b[e], 0.0)) @ eh[i]
        tol = share + 2.0 ** -8 * (np.abs(want[i]) + share)
        assert np.all(np.abs(got[i] - want[i])[fine] <= tol[fine])
    return want


def simple(q, top, n, k, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    a, b = torch.randn(3, top, k, generator=g) * k ** -0.5, torch.randn(3, n, top, generator=g) * 0.1
    return q.LoraAdapters(a.bfloat16().cuda(), b.bfloat16().cuda(), torch.full((3,), scale).cuda())


@pytest.mark.parametrize("top", [8, 32, 64, 128])
@pytest.mark.parametrize("m", [6, 40, 300, 600])
def test_infinite_elements_of_b(m, top):
    q = qlib()
    n, k = 96, 64
    ad = simple(q, top, n, k, top)
    ad.b[0, 5, 0] = INF
    ad.b[0, 6, 1] = -INF
    ad.b[0, 7, 2], ad.b[0, 7, 3] = INF, INF
    ad.b[1, 95, 7] = INF
    ad.a[1, :, 0] = torch.tensor([2.0, 1.0, -1.0, 0.5] * (top // 4), dtype=torch.bfloat16)
    x, y = rows(m, k, m), rows(m, n, m + 1, fill=0.0)
    ids = [(0, 1, -1, 2, 0)[i % 5] for i in range(m)]
    x[1::10] = 0.0
    x[1::10, 0] = 1.0   # h of adapter 1 is 2, 1, -1 or 0.5: one bf16 term would hold it
    x[4::10] = 0.0      # h is 0: NaN where b is infinite
    want = compare(q, ad, ids, x, y)
    assert np.isinf(want).sum() > m // 10 and np.isnan(want[4::10]).any(axis=1).all()


@pytest.mark.parametrize("m", [5, 300])
def test_h_beyond_bf16(m):
    """h = 3.4e38, below fp32's largest number and above bf16's."""
    q = qlib()
    n, k = 64, 64
    ad = simple(q, 16, n, k, 3)
    ad.a.zero_()
    ad.a[:, 0, :2] = 1.0
    ad.a[:, 1, :2] = -1.0
    ad.b *= 2.0 ** -100
    x, y = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda"), rows(m, n, 1, fill=0.0)
    x[:, 0], x[:, 1] = torch.finfo(torch.bfloat16).max, 1.2e36
    want = compare(q, ad, [i % 3 for i in range(m)], x, y)
    assert np.isfinite(want).all() and np.abs(want).max() > 1e6
    ad.b[:, 3, 0] = INF
    ad.b[:, 4, 1] = INF
    want = compare(q, ad, [i % 3 for i in range(m)], x, y)
    assert (want[:, 3] == INF).all() and (want[:, 4] == -INF).all()


@pytest.mark.parametrize("m", [5, 300])
def test_infinite_h(m):
    q = qlib()
    ad = simple(q, 16, 64, 64, 4)
    ad.a[:, 3, 0] = INF
    x, y = rows(m, 64, 2), rows(m, 64, 3, fill=0.0)
    x[2, 0] = 0.0       # NaN
    ad.b[:, 7, 3] = 0.0  # NaN
    ad.b[:, 8, 3] = -INF
    compare(q, ad, [i % 3 for i in range(m)], x, y)

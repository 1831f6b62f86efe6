"""Low-rank adapters of many requests on the GPU against the 64-bit oracle.

Errors: h is summed by MMAs of 16 inputs, one fp32 accumulation each, and by at most 64 parts: (k / 16 + 64) steps within
2^-23 (tensor cores may cut instead of round) of the sum of |a x|.  scale * h rounds once and its two bf16 terms leave 2^-16 of it.  The
second product adds (max_rank / 8 + 4) steps of 2^-23 of its |b h| and |y|, and the output is rounded to bf16: 2^-8 (eps/2)."""
import numpy as np
import pytest
import torch

from oracle import layer as ol
from tests.gpu_util import qlib, to_f64

pytestmark = pytest.mark.gpu


def rows(m, k, seed, pad=0, fill=float("nan")):
    """bf16 [m, k] whose rows lie further apart, NaN between them."""
    ld = (k + 7) // 8 * 8 + pad
    t = torch.full((m, ld), fill, dtype=torch.bfloat16)
    t[:, :k] = torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).bfloat16()
    return t.cuda()[:, :k]


def adapters(q, count, top, k, n, seed, ranks=None, pad=0):
    g = torch.Generator().manual_seed(seed)
    lda = (k + 7) // 8 * 8 + pad
    a = torch.full((count, top, lda), float("nan"))
    a[:, :, :k] = torch.randn(count, top, k, generator=g) * k ** -0.5
    b = torch.randn(count, n, top, generator=g) * 0.1
    if ranks is not None:  # whatever lies past a rank does not enter
        for e, r in enumerate(ranks):
            a[e, r:] = float("nan")
            b[e, :, r:] = float("inf")
    sc = 0.25 + torch.rand(count, generator=g)
    return q.LoraAdapters(a.bfloat16().cuda()[:, :, :k], b.bfloat16().cuda(), sc.cuda(),
                          None if ranks is None else torch.tensor(ranks, dtype=torch.int32).cuda())


def check(ad, ids, x, y, got):
    a, b, sc = np.nan_to_num(to_f64(ad.a), posinf=0.0), np.nan_to_num(to_f64(ad.b), posinf=0.0), to_f64(ad.scales)
    top = a.shape[1]
    ranks = [top] * len(a) if ad.ranks is None else ad.ranks.tolist()
    y64 = to_f64(y)
    want, h, mag = ol.lora(ids, to_f64(x), y64, a, b, sc, ranks)
    eh = (ad.k / 16 + 64) * 2.0 ** -23 * mag + 2.0 ** -16 * np.abs(h)
    share = np.zeros_like(want)
    for i, e in enumerate(ids):
        if 0 <= e < len(a):
            steps = (top / 8 + 4) * 2.0 ** -23
            share[i] = sc[e] * np.abs(b[e]) @ (eh[i] + steps * np.abs(h[i])) + steps * np.abs(y64[i])
    tol = share + 2.0 ** -8 * (np.abs(want) + share)
    err = np.abs(to_f64(got) - want)
    assert np.all(err <= tol), f"{np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"
    none = np.array([not 0 <= e < len(a) or ranks[e] == 0 for e in ids])
    assert np.array_equal(to_f64(got)[none], y64[none])


def ids_of(kind, m, count, seed):
    r = np.random.default_rng(seed)
    if kind == "runs":
        cuts = np.sort(r.integers(0, m + 1, max(1, min(6, m // 2))))
        return [int(v) for v in r.integers(-1, count, len(cuts) + 1)[np.searchsorted(cuts, np.arange(m), side="right")]]
    if kind == "one":
        return [count - 1] * m
    if kind == "none":
        return [-1] * m
    return [int(v) for v in r.integers(-1, count, m)]


def run(q, ad, ids, x, y, **kw):
    ws = q.Workspace(q.lora_workspace_size(ad, len(ids)))
    t = torch.tensor(ids, dtype=torch.int32, device="cuda")
    before = y.clone()
    out = torch.full((len(ids), (ad.n + 7) // 8 * 8 + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    got = q.lora(ad, t, x, y, out=out[:, :ad.n], workspace=ws, **kw)
    assert ws.status() == 0
    assert torch.equal(y, before) and torch.all(out[:, ad.n:] == 9.0)
    here = torch.full_like(out, 5.0)
    here[:, :ad.n] = y
    assert q.lora(ad, t, x, here[:, :ad.n], workspace=ws).data_ptr() == here.data_ptr()
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731  (NaN equals itself)
    assert torch.equal(bits(here[:, :ad.n]), bits(got)) and torch.all(here[:, ad.n:] == 5.0)
    return got


@pytest.mark.parametrize("kind", ["mixed", "runs", "one"])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 64, 129, 256])
@pytest.mark.parametrize("top", [8, 16, 32, 64, 128])
def test_few_rows(m, top, kind):
    q = qlib()
    ad = adapters(q, 7, top, 512, 384, top + m)
    ids, x, y = ids_of(kind, m, 7, m), rows(m, 512, m), rows(m, 384, m + 1, fill=0.0)
    check(ad, ids, x, y, run(q, ad, ids, x, y))


@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("m", [257, 320, 1000])
@pytest.mark.parametrize("top", [8, 16, 24, 32, 48, 64, 96, 128])
def test_many_rows(m, top, kind):
    q = qlib()
    ad = adapters(q, 5, top, 320, 264, top + m)
    ids, x, y = ids_of(kind, m, 5, m + top), rows(m, 320, m), rows(m, 264, m + 1, fill=0.0)
    check(ad, ids, x, y, run(q, ad, ids, x, y))


@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("k,n", [(1, 1), (7, 9), (33, 31), (100, 257), (1001, 515), (2048, 40), (40, 2048), (17408, 72), (5120, 7168)])
def test_odd_sizes_ranks_and_strides(m, k, n):
    q = qlib()
    ranks = [16, 1, 0, 7, 9, 12]
    ad = adapters(q, 6, 16, k, n, k + n, ranks=ranks, pad=16)
    ids, x, y = ids_of("mixed", m, 6, k), rows(m, k, 3, pad=8), rows(m, n, 4, pad=24, fill=0.0)
    check(ad, ids, x, y, run(q, ad, ids, x, y))


@pytest.mark.parametrize("top,ranks", [(32, [31, 17, 8, 32]), (64, [1, 33, 64, 40]), (128, [65, 128, 100, 3])])
@pytest.mark.parametrize("m", [40, 600])
def test_ragged_ranks(m, top, ranks):
    q = qlib()
    ad = adapters(q, 4, top, 640, 520, top, ranks=ranks)
    ids, x, y = ids_of("mixed", m, 4, m), rows(m, 640, 1), rows(m, 520, 2, fill=0.0)
    check(ad, ids, x, y, run(q, ad, ids, x, y))


@pytest.mark.parametrize("m,count", [(200, 1024), (3000, 1024), (5000, 300), (70000, 3)])
def test_many_adapters_and_rows(m, count):
    q = qlib()
    ad = adapters(q, count, 8, 64, 48, m)
    ids, x, y = ids_of("mixed", m, count, m), rows(m, 64, 1), rows(m, 48, 2, fill=0.0)
    check(ad, ids, x, y, run(q, ad, ids, x, y))


@pytest.mark.parametrize("m", [9, 400])
def test_special_values_stay_in_their_rows(m):
    q = qlib()
    ad = adapters(q, 3, 16, 128, 96, 5)
    ids = [i % 3 for i in range(m)]
    x, y = rows(m, 128, 1), rows(m, 96, 2, fill=0.0)
    clean = run(q, ad, ids, x, y)
    bad = x.clone()
    bad[1, 3] = float("nan")
    bad[5, 0] = float("inf")
    got = run(q, ad, ids, bad, y)
    keep = torch.tensor([i not in (1, 5) for i in range(m)], device="cuda")
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[1]).all()
    # an infinite h times b: infinite (or NaN where two of them meet), never finite
    assert not torch.isfinite(got[5]).any()
    # an adapter of NaN reaches its own rows only
    ad.a[2] = float("nan")
    got = run(q, ad, ids, x, y)
    keep = torch.tensor([i % 3 != 2 for i in range(m)], device="cuda")
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[~keep]).all()


@pytest.mark.parametrize("m", [10, 300])
def test_bad_ids_and_ranks_are_reported(m):
    q = qlib()
    ad = adapters(q, 3, 16, 128, 96, 6, ranks=[16, 16, 16])
    ids = [0, 3, -2, 1 << 30, 2] + [1] * (m - 5)
    x, y = rows(m, 128, 1), rows(m, 96, 2, fill=0.0)
    ws = q.Workspace(q.lora_workspace_size(ad, m))
    t = torch.tensor(ids, dtype=torch.int32, device="cuda")
    got = q.lora(ad, t, x, y, out=torch.empty_like(y), workspace=ws)
    assert ws.status() == 1 and ws.status() == 0
    check(ad, ids, x, y, got)
    for rank in (-1, 17):
        ad.ranks[1] = rank
        ids = [i % 3 for i in range(m)]
        got = q.lora(ad, torch.tensor(ids, dtype=torch.int32, device="cuda"), x, y, out=torch.empty_like(y), workspace=ws)
        assert ws.status() == 1
        check(ad, [-1 if e == 1 else e for e in ids], x, y, got)


def test_graph_stream_and_repeat():
    q = qlib()
    m = 90
    ad = adapters(q, 5, 32, 512, 768, 7)
    ids = torch.tensor(ids_of("mixed", m, 5, 1), dtype=torch.int32, device="cuda")
    x, y = rows(m, 512, 1), rows(m, 768, 2, fill=0.0)
    ws = q.Workspace(q.lora_workspace_size(ad, m))
    out = torch.empty_like(y)
    q.lora(ad, ids, x, y, out=out, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = q.lora(ad, ids, x, y, out=torch.empty_like(y), workspace=ws)
    side.synchronize()
    assert torch.equal(out, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.lora(ad, ids, x, y, out=out, workspace=ws)
        q.lora(ad, ids, x, out, workspace=ws)
    ids.copy_(torch.tensor(ids_of("runs", m, 5, 2), dtype=torch.int32))
    x.copy_(rows(m, 512, 5))
    graph.replay()
    want = q.lora(ad, ids, x, y, out=torch.empty_like(y), workspace=ws)
    want = q.lora(ad, ids, x, want, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ws.status() == 0


def test_no_rows():
    q = qlib()
    ad = adapters(q, 2, 8, 64, 64, 1)
    y = rows(0, 64, 1)
    assert q.lora(ad, torch.zeros(0, dtype=torch.int32, device="cuda"), rows(0, 64, 1), y) is y


@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("m,count", [(257, 16), (300, 48), (512, 16), (512, 15), (513, 16), (512, 200)])
def test_launches_of_256_rows_and_the_border_to_many(m, count, kind):
    q = qlib()
    ad = adapters(q, count, 16, 200, 136, m + count)
    ids, x, y = ids_of(kind, m, count, m), rows(m, 200, m), rows(m, 136, m + 1, fill=0.0)
    check(ad, ids, x, y, run(q, ad, ids, x, y))


def test_many_rows_captured_on_streams_and_with_one_workspace():
    """One workspace for calls of falling and rising size, two graphs that share it, and a stream of its own for each of two
    calls with theirs."""
    q = qlib()
    ad, wide = adapters(q, 5, 32, 512, 768, 7), adapters(q, 300, 128, 256, 264, 8)
    most = 2000
    ws = q.Workspace(max(q.lora_workspace_size(a, most) for a in (ad, wide)))
    sized = {m: (torch.tensor(ids_of("mixed", m, 5, m), dtype=torch.int32, device="cuda"), rows(m, 512, m), rows(m, 768, m + 1, fill=0.0))
             for m in (2000, 300, 40, 1100)}
    graphs, outs = [], {}
    for m, (ids, x, y) in sized.items():
        outs[m] = torch.zeros_like(y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.lora(ad, ids, x, y, out=outs[m], workspace=ws)
        graphs.append(g)
    big = torch.tensor(ids_of("mixed", most, 300, 9), dtype=torch.int32, device="cuda")
    bx, by = rows(most, 256, 10), rows(most, 264, 11, fill=0.0)
    for g in graphs + graphs[::-1]:
        for o in outs.values():
            o.zero_()
        g.replay()
        got = q.lora(wide, big, bx, by, out=torch.empty_like(by), workspace=ws)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert ws.status() == 0
    check(wide, big.tolist(), bx, by, got)
    for m, (ids, x, y) in sized.items():
        check(ad, ids.tolist(), x, y, outs[m])
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [q.Workspace(q.lora_workspace_size(ad, 2000)) for _ in range(2)]
    ids, x, y = sized[2000]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, w in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(q.lora(ad, ids, x, y, out=torch.empty_like(y), workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(g, outs[2000]) for g in got) and all(w.status() == 0 for w in spaces)


def test_a_workspace_serves_on_after_bad_ids():
    q = qlib()
    ad = adapters(q, 4, 16, 256, 256, 3)
    ws = q.Workspace(q.lora_workspace_size(ad, 600))
    x, y = rows(600, 256, 1), rows(600, 256, 2, fill=0.0)
    bad = torch.full((600,), 9, dtype=torch.int32, device="cuda")
    ids = ids_of("mixed", 600, 4, 5)
    good = torch.tensor(ids, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out = q.lora(ad, bad, x, y, out=torch.empty_like(y), workspace=ws)
        assert ws.status() == 1 and torch.equal(out, y)
        out = q.lora(ad, good, x, y, out=torch.empty_like(y), workspace=ws)
        assert ws.status() == 0
        check(ad, ids, x, y, out)


@pytest.mark.parametrize("top", [8, 32, 64, 104])
@pytest.mark.parametrize("m", [16, 17, 40, 100, 256])
def test_in_place_has_the_same_bits_with_rows_without_an_adapter(m, top):
    """More tiles than clusters, some of rows without an adapter, which in place are left alone."""
    q = qlib()
    ad = adapters(q, 40, top, 304, 402, m + top)
    for seed in range(4):
        ids, x, y = ids_of("mixed", m, 40, seed), rows(m, 304, 1), rows(m, 402, 2, fill=0.0)
        ids[::3] = [-1] * len(ids[::3])
        check(ad, ids, x, y, run(q, ad, ids, x, y))

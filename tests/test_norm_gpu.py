"""RMS norm with residual and 8-bit output on the GPU against the 64-bit oracle.

Errors: u = 2^-24.  The squares are summed in at most 64 + 5 + 32 steps (a thread's elements, a warp, the warps), each within
u of positive terms, so 1/sqrt is off by half of 101 u, the mean, eps and rsqrtf (2 ulp = 4 u) add 6 u, the two products and the
weight's offset 3 u: y is within 2^-18 of itself in fp32, and the rounding to bf16 adds 2^-8 (eps/2).  Scales are y's plus a
division: 2^-17.  A code is that of a quotient within 2^-16: amax / 448, the reciprocal and the product add 3 u."""
import numpy as np
import pytest
import torch

from oracle import layer as ol
from tests.gpu_util import qlib, to_f64

pytestmark = pytest.mark.gpu


def matrix(m, k, seed, scale=1.0, pad=0, dtype=torch.bfloat16):
    ld = (k + 7) // 8 * 8 + pad
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, ld, generator=g) * scale).to(dtype).cuda()[:, :k]


def check_y(got, want):
    tol = (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + 2.0 ** -133
    assert np.all(np.abs(to_f64(got) - want) <= tol)


def check_codes(codes, scales, y, group):
    q, s = ol.quantise(y, group)
    assert np.all(np.abs(to_f64(scales) - s) <= 2.0 ** -17 * s)
    low, high = ol.codes_between(q, 2.0 ** -16)
    got = to_f64(codes)
    assert np.all((got >= low) & (got <= high))


@pytest.mark.parametrize("m", [1, 2, 37])
@pytest.mark.parametrize("k", [1, 7, 8, 31, 256, 257, 1000, 2048, 5120, 8192, 8200, 17408, 40001])
@pytest.mark.parametrize("residual", [False, True])
def test_bf16(m, k, residual):
    q = qlib()
    x, r = matrix(m, k, k + m, pad=8), matrix(m, k, k + 1, 3.0, pad=16) if residual else None
    w = matrix(1, k, 5)[0]
    y, h = q.rms_norm(x, w, r, eps=1e-5, weight_offset=1.0)
    want_h, want = ol.rms_norm(to_f64(x), None if r is None else to_f64(r), to_f64(w), 1e-5, 1.0)
    if residual:
        assert np.array_equal(to_f64(h), want_h)
    else:
        assert h is None
    check_y(y, want)


@pytest.mark.parametrize("m,k", [(1, 5120), (3, 40), (65, 129), (5, 257), (1, 1), (19, 2048), (2, 17408), (2, 65536), (3, 33001)])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_fp8(m, k, group):
    q = qlib()
    x, r, w = matrix(m, k, k, pad=8), matrix(m, k, k + 1, 2.0), matrix(1, k, 7)[0]
    both = torch.empty(m, (k + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :k]
    codes, scales, h = q.rms_norm_fp8(x, w, r, group=group, y_out=both)
    want_h, want = ol.rms_norm(to_f64(x), to_f64(r), to_f64(w), 1e-6, 0.0)
    assert np.array_equal(to_f64(h), want_h)
    check_codes(codes, scales, want, group)
    check_y(both, want)
    alone = q.rms_norm_fp8(x, w, group=group)
    assert alone[2] is None
    check_codes(alone[0], alone[1], ol.rms_norm(to_f64(x), None, to_f64(w), 1e-6, 0.0)[1], group)


def test_in_place_and_padding_untouched():
    q = qlib()
    m, k = 33, 1001
    base = torch.full((m, 1016), 7.0, dtype=torch.bfloat16, device="cuda")
    stream = torch.full((m, 1008), 5.0, dtype=torch.bfloat16, device="cuda")
    base[:, :k] = matrix(m, k, 1)
    stream[:, :k] = matrix(m, k, 2)
    w = matrix(1, k, 3)[0]
    y0, h0 = q.rms_norm(base[:, :k], w, stream[:, :k])
    y, h = q.rms_norm(base[:, :k], w, stream[:, :k], out=base[:, :k], sum_out=stream[:, :k])
    assert y.data_ptr() == base.data_ptr() and h.data_ptr() == stream.data_ptr()
    assert torch.equal(y, y0) and torch.equal(h, h0)
    assert torch.all(base[:, k:] == 7.0) and torch.all(stream[:, k:] == 5.0)
    codes = torch.full((m, 1008), 3.0, device="cuda").to(torch.float8_e4m3fn)
    scales = torch.full((m, 12), -1.0, device="cuda")
    q.rms_norm_fp8(base[:, :k], w, out=codes[:, :k], scales=scales[:, :8])
    assert torch.all(codes[:, k:].float() == 3.0) and torch.all(scales[:, 8:] == -1.0)


def test_special_values():
    q = qlib()
    k = 300
    x = matrix(7, k, 4)
    x[0] = 0.0                       # zeros: y is 0, the scale its least
    x[1, 17] = float("nan")          # the row is NaN
    x[2, 5] = float("inf")           # 1 / sqrt(inf) is 0: zeros, and NaN for the infinity itself
    x[3] *= 2.0 ** -60               # squares near fp32's smallest
    x[4] = 2.0 ** 62                 # squares of 2^124, their sum below 2^128 / 300
    x[4, 4:] = 0.0
    w = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    y, _ = q.rms_norm(x, w, eps=1e-6)
    _, want = ol.rms_norm(to_f64(x), None, to_f64(w), 1e-6, 0.0)
    got = to_f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got[1]).all() and np.isnan(got[2]).sum() == 1
    ok = ~np.isnan(want)
    assert np.all(np.abs(got[ok] - want[ok]) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want[ok]))
    codes, scales, _ = q.rms_norm_fp8(x, w, group=32)
    c, s = to_f64(codes), to_f64(scales)
    assert np.all(c[0] == 0) and np.all(s[0] == 2.0 ** -100)
    assert np.isnan(c[1]).all() and np.all(s[1] == 2.0 ** -100)
    # a weight that is infinite: the code saturates and the scale stays that of the others
    w2 = w.clone()
    w2[3] = float("inf")
    codes, scales, _ = q.rms_norm_fp8(x[5:], w2, group=32)
    c, s = to_f64(codes), to_f64(scales)
    _, want = ol.rms_norm(to_f64(x[5:]), None, to_f64(w), 1e-6, 0.0)
    want[:, 3] = 0.0
    assert np.all(np.abs(c[:, 3]) == 448.0) and np.all(np.abs(s - ol.quantise(want, 32)[1]) <= 2.0 ** -17 * s)


def test_many_rows_streams_graphs_and_repeats():
    q = qlib()
    m, k = 5003, 512
    x, r, w = matrix(m, k, 8), matrix(m, k, 9), matrix(1, k, 10)[0]
    y, h = q.rms_norm(x, w, r)
    want_h, want = ol.rms_norm(to_f64(x), to_f64(r), to_f64(w), 1e-6, 0.0)
    assert np.array_equal(to_f64(h), want_h)
    check_y(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, h2 = q.rms_norm(x, w, r)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2)
    out, sums = torch.zeros_like(y), torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.rms_norm(x, w, r, out=out, sum_out=sums)
        codes, scales, _ = q.rms_norm_fp8(sums, w, group=0)
    x.copy_(matrix(m, k, 11))
    graph.replay()
    y3, h3 = q.rms_norm(x, w, r)
    torch.cuda.synchronize()
    assert torch.equal(out, y3) and torch.equal(sums, h3)
    check_codes(codes, scales, ol.rms_norm(to_f64(h3), None, to_f64(w), 1e-6, 0.0)[1], 0)


def test_no_rows():
    q = qlib()
    y, h = q.rms_norm(matrix(0, 64, 1), matrix(1, 64, 1)[0], matrix(0, 64, 1))
    assert y.shape == (0, 64) and h.shape == (0, 64)


@pytest.mark.parametrize("group", [0, 32, 128])
def test_products_beyond_fp32_and_the_same_bits_with_codes(group):
    """h * weight past fp32's range or near its end, while y itself is an ordinary number."""
    q = qlib()
    k = 264
    x = matrix(6, k, 21)
    w = matrix(1, k, 22)[0]
    for scale_x, scale_w in ((2.0 ** 50, 2.0 ** 100), (2.0 ** 58, 2.0 ** 69), (2.0 ** -50, 2.0 ** -60), (2.0 ** -60, 2.0 ** 90),
                             (2.0 ** 58, 2.0 ** -90)):
        xs, ws = (x.float() * scale_x).bfloat16(), (w.float() * scale_w).bfloat16()
        xs[1, :k // 2] = 0.0   # groups of zeros
        xs[2, 7:] = 0.0
        _, want = ol.rms_norm(to_f64(xs), None, to_f64(ws), 0.0, 0.0)
        both = torch.empty(6, k, dtype=torch.bfloat16, device="cuda")
        codes, scales, _ = q.rms_norm_fp8(xs, ws, eps=0.0, group=group, y_out=both)
        check_codes(codes, scales, want, group)
        check_y(both, want)
        assert torch.equal(both, q.rms_norm(xs, ws, eps=0.0)[0])


@pytest.mark.parametrize("group", [0, 64])
def test_two_streams_at_once(group):
    q = qlib()
    m, k = 700, 1024
    x, r, w = matrix(m, k, 31), matrix(m, k, 32), matrix(1, k, 33)[0]
    want = q.rms_norm_fp8(x, w, r, group=group)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(q.rms_norm_fp8(x, w, r, group=group))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((t.contiguous() for t in g), (t.contiguous() for t in want)))


@pytest.mark.parametrize("group", [None, 0, 32, 128])
@pytest.mark.parametrize("m,k", [(400, 16392), (153, 24577), (307, 65536)])
def test_long_rows_in_turn(m, k, group):
    """Rows too long for registers, more of them than CTAs, in place."""
    q = qlib()
    x, r, w = matrix(m, k, k), matrix(m, k, k + 1, 2.0), matrix(1, k, 3)[0]
    want_h, want = ol.rms_norm(to_f64(x), to_f64(r), to_f64(w), 1e-6, 0.0)
    if group is None:
        y, h = q.rms_norm(x, w, r, out=x, sum_out=r)
        check_y(y, want)
    else:
        codes, scales, h = q.rms_norm_fp8(x, w, r, group=group, sum_out=r)
        check_codes(codes, scales, want, group)
    assert np.array_equal(to_f64(h), want_h)

"""Pins of the 64-bit oracle of the cache append and the attention: closed forms and another decoder."""
import numpy as np
import pytest
import torch

from oracle import attention as oa


def test_e4m3_codes_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(oa.e4m3_decode(codes), want, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).integers(-12, 8, 20000))
    x = np.clip(x.astype(np.float32), -448, 448)
    mid = (oa._GRID[1:] + oa._GRID[:-1]) / 2  # ties
    x = np.concatenate([x, mid, -mid, [0.0, -0.0, 448.0]]).astype(np.float32)
    assert np.array_equal(oa.e4m3_encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert oa.e4m3_encode(np.inf) == 0x7E and oa.e4m3_encode(-1e9) == 0xFE and oa.e4m3_encode(np.nan) == 0x7F


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (0.0, 2.0 ** -100), (7.0, 2.0 ** -6),
                                        (1e38, 2.0 ** 118)])
def test_page_scale(amax, scale):
    assert oa.page_scale(amax) == scale and amax <= 448 * scale


def test_norm_rope_closed_forms():
    x = np.array([[3.0, 4.0, 0.0, 0.0] * 4])
    y = oa.norm_rope(x, np.ones(16), 0.0, 0.0, None, False, 0)
    assert np.allclose(np.mean(y * y), 1.0) and np.allclose(y[0, 0] / y[0, 1], 0.75)
    quarter = np.concatenate([np.zeros((1, 8)), np.ones((1, 8))], 1)  # a quarter turn of every pair
    z = np.arange(16.0)[None]
    assert np.array_equal(oa.norm_rope(z, None, 0, 0, quarter, False, 0)[0], np.concatenate([-z[0, 8:], z[0, :8]]))
    assert np.array_equal(oa.norm_rope(z, None, 0, 0, quarter, True, 0)[0][:4], [-1, 0, -3, 2])


def test_append_grows_a_scale_and_moves_the_codes():
    codes, scales = np.zeros((2, 1, 16, 4), np.uint8), np.ones((2, 1))
    c, s, _ = oa.append(np.full((1, 1, 4), 1.0), [1], [1], [[1]], 16, codes, scales)
    assert s[1, 0] == 2.0 ** -8 and np.all(oa.e4m3_decode(c[1, 0, 0]) * s[1, 0] == 1.0)
    c, s, _ = oa.append(np.full((1, 1, 4), 100.0), [1], [2], [[1]], 16, c, s)
    assert s[1, 0] == 0.25 and np.all(oa.e4m3_decode(c[1, 0, :2, 0]) * s[1, 0] == [1.0, 96.0])  # 100 is a tie: even code
    assert s[0, 0] == 1.0 and not c[0].any()


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    kc = np.zeros((2, 1, 16, 8), np.uint8)
    vc = oa.e4m3_encode(rng.standard_normal(kc.shape))
    vs = np.array([[1.0], [4.0]])
    q = rng.standard_normal((3, 2, 8))
    out, *_ = oa.attention(q, [3], [18], [[1, 0]], 16, kc, np.ones((2, 1)), vc, vs, 0.3)  # all scores 0: a mean
    v = np.concatenate([oa.e4m3_decode(vc[1, 0]) * 4.0, oa.e4m3_decode(vc[0, 0])])
    for i in range(3):
        assert np.allclose(out[i], v[:16 + i].mean(0))
    out, *_ = oa.attention(q, [3], [18], [[1, 0]], 16, kc, np.ones((2, 1)), vc, vs, 0.3, window=1)
    assert np.allclose(out[:, 0], v[15:18])  # a window of one token: its own value
    out, *_ = oa.attention(q, [3], [2], [[1, 0]], 16, kc, np.ones((2, 1)), vc, vs, 0.3)
    assert not out[0].any() and out[1].any()  # the first row stands before the sequence and sees nothing


def test_attention_leaves_out_pages_of_key_scale_zero():
    rng = np.random.default_rng(3)
    kc, vc = (oa.e4m3_encode(rng.standard_normal((3, 1, 16, 8))) for _ in range(2))
    ks, vs = np.ones((3, 1)), np.ones((3, 1))
    q = rng.standard_normal((1, 2, 8))
    want, *_ = oa.attention(q, [1], [32], [[0, 2]], 16, kc, ks, vc, vs, 0.3)
    ks[1], vs[1], kc[1], vc[1, :, ::3] = 0.0, np.nan, 0x7F, 0x7F
    out, mag, load, vmax = oa.attention(q, [1], [48], [[0, 1, 2]], 16, kc, ks, vc, vs, 0.3)
    assert np.array_equal(out, want) and np.all(np.isfinite([mag.max(), load.max(), vmax.max()]))
    out, *_ = oa.attention(q, [1], [16], [[1]], 16, kc, ks, vc, vs, 0.3)
    assert not out.any()

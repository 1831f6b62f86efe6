"""The norm's codes, value by value: that of h * weight * 448 / (the group's largest |h * weight|), which is y / scale.

Without an offset h * weight is exact in fp32 (two factors of 8 bits), so is the largest of them; 448 / largest and the
product with it round once each: 2 u, u = 2^-24.  An offset rounds the weight's sum and the product, in the value and in the largest: 4 u
more.  The code is within half an E4M3 step of that."""
import pytest
import torch

from tests.gpu_util import qlib
from tests.test_norm_bits_gpu import randn

pytestmark = pytest.mark.gpu


def steps(q):
    """The distance of E4M3 numbers around |q| <= 448."""
    return torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)


def values(h, w, offset, group):
    """y over its scale in 64 bits (1 / sqrt cancels)."""
    v = h.double() * (w.double() + offset)
    m, k = v.shape
    g = group or k
    pad = torch.nn.functional.pad(v, (0, -k % g)).view(m, -1, g)
    return (pad * 448.0 / pad.abs().amax(-1, keepdim=True).clamp_min(1e-30)).flatten(1)[:, :k]


@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("m,k", [(4000, 5120), (9000, 2048), (600, 20000), (20000, 1000)])
def test_each_code_is_the_nearest(m, k, group, offset):
    q = qlib()
    x, w = randn(m, (k + 7) // 8 * 8, m + group)[:, :k], randn(1, k, 2)[0]
    codes = q.rms_norm_fp8(x, w, weight_offset=offset, group=group)[0].double()
    want = values(x, w, offset, group)
    off = (codes - want).abs() - steps(want) / 2
    u = 2.0 ** -24
    assert bool((off <= (2 if offset == 0.0 else 6) * 1.001 * u * want.abs()).all()), float((off / want.abs()).max() / u)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_a_group_s_codes_do_not_go_by_its_neighbours(group):
    """Between others, at a row's end, beside groups of zeros and beside some beyond fp32's range."""
    q = qlib()
    m, k = 3000, 512
    x, w = randn(m, k, 5), randn(1, k, 6)[0]
    want = q.rms_norm_fp8(x, w, group=group)[0].view(torch.uint8)
    short = q.rms_norm_fp8(x[:, :2 * group].contiguous(), w[:2 * group].contiguous(), group=group)[0].view(torch.uint8)
    assert torch.equal(short, want[:, :2 * group])
    zeros = x.clone()
    zeros[:, group:2 * group] = 0.0
    got = q.rms_norm_fp8(zeros, w, group=group)[0].view(torch.uint8)
    assert torch.equal(got[:, :group], want[:, :group]) and torch.equal(got[:, 2 * group:], want[:, 2 * group:])
    far = w.clone()
    far[group:2 * group] = 3e38
    got = q.rms_norm_fp8(x, far, group=group)[0].view(torch.uint8)
    assert torch.equal(got[:, :group], want[:, :group]) and torch.equal(got[:, 2 * group:], want[:, 2 * group:])

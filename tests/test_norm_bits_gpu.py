"""The norm's bf16 output has the same bits with codes and without, whatever the codes' groups."""
import pytest
import torch

from tests.gpu_util import qlib

pytestmark = pytest.mark.gpu


def randn(m, k, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(m, k, device="cuda", generator=g) * scale).bfloat16()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,k", [(4096, 5120), (9000, 2048), (1200, 16392), (150, 8192), (150, 16384)])
def test_the_same_bits_with_codes_and_without(m, k, residual):
    """Millions of values: a last bit of 1 / sqrt shows in one bf16 value of some 2^16."""
    q = qlib()
    x, w, r = randn(m, k, 1), randn(1, k, 2)[0], randn(m, k, 3, 2.0) if residual else None
    want, h = q.rms_norm(x, w, r)
    for group in (0, 32, 64, 128):
        both = torch.empty_like(x)
        got = q.rms_norm_fp8(x, w, r, group=group, y_out=both)
        assert torch.equal(both, want), (group, int((both != want).sum()))
        assert h is None or torch.equal(got[2], h)

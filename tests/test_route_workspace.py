"""The router's workspace grows with the tokens, so that one made for the longest batch serves every shorter one (no GPU)."""
import random

import pytest


@pytest.fixture(scope="module")
def size():
    from prefill_dequant_gemv_gb300 import build as b
    b.build()
    import prefill_dequant_gemv_gb300 as q
    return q.qmoe_route_workspace_size


@pytest.mark.parametrize("experts,topk", [(512, 10), (512, 16), (512, 1), (256, 8), (160, 6), (64, 4), (8, 2), (1, 1)])
def test_never_smaller_for_more_tokens(size, experts, topk):
    sizes = [size(t, experts, topk) for t in range(1, 20001)]
    assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
    longer = sorted(random.Random(experts + topk).sample(range(20001, 1 << 26), 2000))
    longer = [size(t, experts, topk) for t in longer]
    assert sizes[-1] <= longer[0] and all(a <= b for a, b in zip(longer, longer[1:]))


def test_a_workspace_for_5000_tokens_serves_4096(size):
    assert size(4096, 512, 10) <= size(5000, 512, 10)

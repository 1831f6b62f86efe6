"""The example layer: quantised projections, cache append and attention together, prompts and then tokens from a graph."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (6, 3, 128), (4, 1, 256)])
def test_tokens_one_by_one_equal_one_call(heads, kv_heads, dim):
    import attention_layer
    outs, diff, _ = attention_layer.run(512, heads, kv_heads, dim, prompts=(150, 33, 1), steps=9)
    assert [len(o) for o in outs] == [159, 42, 10]
    # What differs between the two ways: a page that grew token by token may have had a smaller scale before, so that a
    # code was rounded twice (to a neighbour: 2^-3 of one value at most, of few), and sums in another order and bf16
    # roundings between the stages (2^-8 each of up to the layer's largest output, a handful of them).
    assert diff <= 2.0 ** -4

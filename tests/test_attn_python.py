"""Checks of the Python entry points of the cache append and the attention (no GPU: each ends in a refusal)."""
import pytest
import torch

INVALID = 1
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def q():
    from prefill_dequant_gemv_gb300 import build as b
    b.build()
    import prefill_dequant_gemv_gb300 as q
    q.lib()
    return q


def i32(*s, device="cpu"):
    return torch.zeros(*s, dtype=torch.int32, device=device)


def cache(q, device="cpu"):
    codes = torch.zeros(20, 2, 16, 64, dtype=torch.uint8, device=device)
    scales = torch.ones(20, 2, device=device)
    return q.KVCache(codes, codes.clone(), scales, scales.clone())


def refused(q, call, word):
    with pytest.raises(q.QGError, match=word) as e:
        call()
    assert e.value.status == INVALID


@pytest.mark.parametrize("rows", [1, 3])
def test_length_beyond_the_page_table(q, rows):
    """A table that is a slice of a wider one: the width counts, not the stride."""
    wide = i32(rows, 100)
    for table, pages in ((wide[:, 90:], 10), (wide[:, :7], 7), (i32(rows, 9), 9)):
        kv, x = cache(q), torch.zeros(rows, 2, 64, dtype=BF16)
        b = q.KVBatch(i32(rows + 1), i32(rows), table, 1, 16 * pages + 1)
        refused(q, lambda: q.attention(kv, b, x, workspace=q.Workspace(1 << 20, "cpu")), "max_len")
        refused(q, lambda: q.kv_append(kv, b, x, x, x, workspace=q.Workspace(256, "cpu")), "max_len")

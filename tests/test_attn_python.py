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


def calls(q, kv, b, x, y, out, ws, nr=None):
    """Both entry points; x are the queries, y the keys and values."""
    return [(lambda: q.attention(kv, b, x, out=out, workspace=ws)), (lambda: q.kv_append(kv, b, x, y, y, nr, out=out, workspace=ws))]


def test_nothing_runs_on_host_tensors(q):
    kv, b, x = cache(q), q.KVBatch(i32(3), i32(2), i32(2, 2), 1, 32), torch.zeros(2, 2, 64, dtype=BF16)
    for call in calls(q, kv, b, x, x, x.clone(), q.Workspace(1 << 20, "cpu")):
        refused(q, call, "CUDA device")


def test_tensors_of_another_device_than_the_cache(q):
    """The cache's device index is set by hand, as there need be no GPU: the other tensors are elsewhere."""
    x = torch.zeros(2, 2, 64, dtype=BF16)

    ws = q.Workspace(1 << 20, "cpu")
    kv, b = cache(q), q.KVBatch(i32(3), i32(2), i32(2, 2), 1, 32)
    kv.index = 0
    for call in calls(q, kv, b, x, x, None, None):
        refused(q, call, "on one CUDA device")
    b.index = 0
    for call in calls(q, kv, b, x, x, None, ws):
        refused(q, call, "on one CUDA device")
    for call in calls(q, kv, b, x, x, None, None):
        refused(q, call, "on the cache's device")


@pytest.mark.gpu
def test_host_tensors_beside_a_cache_on_the_gpu():
    from tests.gpu_util import qlib
    q = qlib()
    kv = cache(q, "cuda")
    good = dict(b=q.KVBatch(i32(3, device="cuda"), i32(2, device="cuda"), i32(2, 2, device="cuda"), 1, 32),
                x=torch.zeros(2, 2, 64, dtype=BF16, device="cuda"), y=torch.zeros(2, 2, 64, dtype=BF16, device="cuda"),
                out=torch.zeros(2, 2, 64, dtype=BF16, device="cuda"), ws=q.Workspace(1 << 20),
                nr=q.NormRope(torch.ones(64, dtype=BF16, device="cuda")))
    bad = dict(b=q.KVBatch(i32(3), i32(2), i32(2, 2), 1, 32), x=torch.zeros(2, 2, 64, dtype=BF16),
               y=torch.zeros(2, 2, 64, dtype=BF16), out=torch.zeros(2, 2, 64, dtype=BF16), ws=q.Workspace(1 << 20, "cpu"),
               nr=q.NormRope(torch.ones(64, dtype=BF16)))
    for name, value in bad.items():
        attend, append = calls(q, kv, **{**good, name: value})
        refused(q, append, "device")
        if name not in ("y", "nr"):
            refused(q, attend, "device")

"""A rank out of range is reported where a row names its adapter, and only there, whichever kernel takes the call."""
import pytest
import torch

from tests.gpu_util import qlib
from tests.test_lora_gpu import adapters, check, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [3, 256, 257, 700])
@pytest.mark.parametrize("rank", [-1, 17])
def test_a_bad_rank_counts_where_it_is_met(m, rank):
    q = qlib()
    ad = adapters(q, 5, 16, 128, 96, 6, ranks=[16] * 5)
    ad.ranks[3] = rank
    x, y = rows(m, 128, 1), rows(m, 96, 2, fill=0.0)
    ws = q.Workspace(q.lora_workspace_size(ad, m))
    ids = [(0, 1, -1, 4, 2)[i % 5] for i in range(m)]  # not adapter 3
    got = q.lora(ad, torch.tensor(ids, dtype=torch.int32, device="cuda"), x, y, out=torch.empty_like(y), workspace=ws)
    assert ws.status() == 0
    check(ad, ids, x, y, got)
    ids[m - 1] = 3
    got = q.lora(ad, torch.tensor(ids, dtype=torch.int32, device="cuda"), x, y, out=torch.empty_like(y), workspace=ws)
    assert ws.status() == 1
    ids[m - 1] = -1
    check(ad, ids, x, y, got)

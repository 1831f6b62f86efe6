"""The router without a rule around the border from one CTA to a cluster, which goes by the experts: its choice is that of the rule
that says the same, whose launches change elsewhere, and so are its tables."""
import numpy as np
import pytest
import torch

from tests.gpu_util import qlib
from tests.test_route_by_gpu import tables_equal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [8, 9, 12, 13, 16])
@pytest.mark.parametrize("e,k", [(256, 8), (257, 16), (384, 8), (512, 4), (512, 16)])
def test_one_cta_and_a_cluster(t, e, k):
    q = qlib()
    lg = torch.from_numpy(np.random.default_rng(t + e + k).standard_normal((t, e)).astype(np.float32)).cuda()
    (i1, w1, s1), (i2, w2, s2) = q.route(lg, k), q.route(lg, k, rule=q.RouteRule("softmax"))
    want = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k].int()
    assert torch.equal(i1, want) and torch.equal(i2, want)
    assert torch.allclose(w1, w2, rtol=2.0 ** -20, atol=0) and tables_equal(q, s1.buf, s2.buf, t, e, k)

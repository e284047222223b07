"""GPU: the binding passes on that a neighbourhood holds more blocks than the budget."""
import pytest
import torch

from tests.test_gpu_k_blockmean import bsa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,keep,local,over", [(1000, 2, 1, True), (1000, 3, 1, False), (1000, 1, 0, False),
                                               (100, 1, 5, False), (1000, 7, 9, True), (1000, 8, 9, False)])
def test_over_budget_is_returned(bsa, N, keep, local, over):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(N + keep)
    q, k = (torch.randn((N, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    idx, cnt, got = bsa.blockmean_select(q, k, keep, local, return_over_budget=True)
    assert got is over and bool((cnt > keep).any()) is over
    plain = bsa.blockmean_select(q, k, keep, local)
    assert len(plain) == 2 and torch.equal(plain[0], idx) and torch.equal(plain[1], cnt)

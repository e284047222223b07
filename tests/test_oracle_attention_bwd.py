"""Pins of the attention-gradient oracle: central differences of the forward
oracle, torch's autograd in float64, and rows and keys without partners."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import attention_bwd as obwd


def case(seed, N=19, H=2, d=5):
    rng = np.random.default_rng(seed)
    q, k, v, go = rng.standard_normal((4, N, H, d))
    mask = rng.random((N, N)) < 0.4
    mask[3] = False                                       # a query without keys
    mask[:, 7] = False                                    # a key nobody attends
    return go, q, k, v, mask


def test_against_differences_of_the_forward():
    go, q, k, v, mask = case(1)
    grads = obwd.attention_back(go, q, k, v, 0.7, mask)
    f = lambda q, k, v: float((oatt.attention_dense_masked(q, k, v, 0.7, mask)[0] * go).sum())  # noqa: E731
    rng = np.random.default_rng(2)
    for n in range(3):
        x = [q, k, v]
        dx = rng.standard_normal(q.shape)
        e = 1e-5
        up, dn = list(x), list(x)
        up[n], dn[n] = x[n] + e * dx, x[n] - e * dx
        assert (f(*up) - f(*dn)) / (2 * e) == pytest.approx(float((grads[n] * dx).sum()), abs=1e-7)


def test_against_autograd():
    go, q, k, v, mask = case(3)
    mask[3, 5] = True                                     # autograd has no empty rows
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    s = torch.einsum("nhd,mhd->hnm", t[0], t[1]) * 0.3
    p = s.masked_fill(~torch.tensor(mask), float("-inf")).softmax(-1)
    (torch.einsum("hnm,mhd->nhd", p, t[2]) * torch.tensor(go)).sum().backward()
    for got, want in zip(obwd.attention_back(go, q, k, v, 0.3, mask), t):
        assert got == pytest.approx(want.grad.numpy(), abs=1e-12)


def test_without_partners():
    go, q, k, v, mask = case(4)
    dq, dk, dv = obwd.attention_back(go, q, k, v, 1.0, mask)
    assert (dq[3] == 0).all() and (dk[7] == 0).all() and (dv[7] == 0).all()

"""GPU: the rotation calls where blocks stride over the tokens several times, the
last time with part of the groups, against the float64 oracle.

A block takes 256 / (d / 8) tokens at a time; up to 444 blocks run forward and 296
backward, shared out to the tensors of the call.  So one round is 7,104 tokens of
d = 128 (14,208 of d = 64) for one tensor, half of that for q and k, and 2,368
(4,736) backward.  Tolerances: those of tests/test_gpu_j_rope.py, but for the
weight gradient, where a group now adds the heads of several tokens: a lane's sum
takes rounds x heads additions, then come at most 32 groups, 19 blocks of a slice
and 16 slices, and each term is off by 20u: under (rounds heads + 150) u sum|g xh|."""
import numpy as np
import pytest
import torch

from oracle import rope as orope
from tests.test_gpu_j_rope import TYPES, U, bsa, close, f64, make, pair_sum, randn, setup  # noqa: F401

pytestmark = pytest.mark.gpu

FORWARD = [
    # grid, tail, H, d, dtype, pairing, layout, listed
    ((23, 31, 29), 5, 3, 128, "bf16", "adjacent", "packed", False),      # 20,682 tokens: 3 rounds
    ((23, 31, 29), 0, 1, 128, "fp32", "split", "whole", True),
    ((23, 31, 29), 77, 5, 128, "fp16", "split", "heads first", False),
    ((37, 31, 29), 3, 2, 64, "bf16", "split", "padded", True),           # 33,266 tokens: 3 rounds
    ((37, 31, 29), 0, 5, 64, "fp16", "adjacent", "packed", False),
    ((1, 1, 14209), 0, 1, 64, "fp32", "adjacent", "whole", False),       # one token in the second round
]
BOTH = [
    # grid, tail, Hq, Hk, d, dtype, pairing, layout, listed
    ((23, 31, 29), 5, 3, 1, 128, "bf16", "adjacent", "packed", False),   # 6 rounds forward, 9 backward
    ((23, 31, 29), 0, 1, 2, 128, "fp32", "split", "whole", True),
    ((13, 31, 29), 77, 6, 5, 128, "fp16", "split", "heads first", False),
    ((37, 31, 29), 3, 2, 1, 64, "bf16", "split", "padded", True),        # 5 rounds forward, 8 backward
    ((17, 31, 29), 0, 5, 3, 64, "fp16", "adjacent", "packed", False),
    ((1, 1, 2369), 0, 2, 2, 128, "fp32", "adjacent", "whole", False),    # one token in the second backward round
]


@pytest.mark.parametrize("grid,tail,H,d,dtype,pairing,layout,listed", FORWARD)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_apply(bsa, grid, tail, H, d, dtype, pairing, layout, listed, inverse):  # noqa: F811
    r, ang = setup(bsa, grid, tail, d, listed, start=17.0, first=(2, 0, 1), pairing=pairing)
    x = make((ang.shape[0], H, d), TYPES[dtype], layout, 1)
    y = bsa.rope_apply(x, r, inverse=inverse)
    assert bsa.get_device_status() == bsa.BSA_OK
    x64 = f64(x)
    close(y, orope.turn(x64, -ang if inverse else ang, pairing), 4 * U * pair_sum(x64, pairing), x.dtype, "rope")


@pytest.mark.parametrize("grid,tail,Hq,Hk,d,dtype,pairing,layout,listed", BOTH)
def test_norm_rope_and_gradient(bsa, grid, tail, Hq, Hk, d, dtype, pairing, layout, listed):  # noqa: F811
    eps, dt = 1e-5, TYPES[dtype]
    r, ang = setup(bsa, grid, tail, d, listed, pairing=pairing)
    N = ang.shape[0]
    q, k = make((N, Hq, d), dt, layout, 2, 3.0), make((N, Hk, d), dt, layout, 3, 0.5)
    g = torch.Generator(device="cuda").manual_seed(4)
    wq, wk = (1 + 0.3 * randn(g, d) for _ in range(2))
    qo, ko = bsa.qk_norm_rope_fwd(q, k, wq, wk, r, eps=eps)
    gq, gk = make(q.shape, dt, "whole", 5), make(k.shape, dt, layout, 6)
    dq, dk, dwq, dwk = bsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, r, eps=eps)
    assert bsa.get_device_status() == bsa.BSA_OK
    rounds = -(-N // (148 * (256 // (d // 8))))
    for x, w, y, gy, dx, dw in [(q, wq, qo, gq, dq, dwq), (k, wk, ko, gk, dk, dwk)]:
        x64, w64, g64 = f64(x), f64(w), f64(gy)
        rr = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
        close(y, orope.norm_turn(x64, w64, ang, pairing, eps), 24 * U * pair_sum(x64 * rr * w64, pairing), dt, "fwd")
        rdx, rdw = orope.norm_turn_back(g64, x64, w64, ang, pairing, eps)
        turned = pair_sum(orope.turn(g64, -ang, pairing), pairing)
        gb, xh = turned * np.abs(w64), np.abs(x64 * rr)
        close(dx, rdx, 64 * U * rr * (gb + xh * (gb * xh).mean(-1, keepdims=True)), dt, "dx")
        bound = (rounds * x.shape[1] + 150) * U * (turned * xh).sum((0, 1))
        assert np.all(np.abs(f64(dw) - rdw) <= bound)

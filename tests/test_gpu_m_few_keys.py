"""GPU: gradient of rows of few keys at scores of hundreds to thousands, where
the 32-bit lse of a row is off by more than small scores leave it: its D is
still the one of its own probabilities, and a row of one key still gives zeros.

Tolerances (bf16: half a step is at most h = 2^-8 of the value).  lse is the
running maximum and a logarithm, three products and two rounded constants away
from the exponent it comes back into: |lse log2 e| is off by less than 2^-22 of
itself.  A score is a sum of d products, each addition off by at most a step of
2^-23 of the magnitudes: d 2^-23 <= 2^-16 of <|q|, |k|>.  An exponent that is off
by x makes p off by 2^x - 1, the same for every key of a row where the keys are
equal, as they are here (equal operands give equal scores)."""
import numpy as np
import pytest
import torch

from oracle import attention_bwd as obwd
from tests.test_gpu_l_attn_bwd import both, bsa, f64  # noqa: F401

pytestmark = pytest.mark.gpu

HALF, P32, LOG2E = 2.0 ** -8, 2.0 ** -13, 1.4426950408889634
SCORES = [500.0, 2000.0, 8000.0, -500.0, -2000.0, -8000.0]


def aligned(N, H, d, score, seed):
    """go, q, k, v [N, H, d] with scale <q, k> near `score` for every pair; the keys of a head are equal."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")         # noqa: E731
    b = randn(1, H, d) * (abs(score) / d ** 0.5) ** 0.5
    q = (b + 0.05 * b.abs() * randn(N, H, d)).bfloat16()
    k = (b if score > 0 else -b).expand(N, H, d).bfloat16().contiguous()
    return randn(N, H, d).bfloat16(), q, k, randn(N, H, d).bfloat16()


def p_error(q, k, scale):
    """Bound of the relative error that all p of a row share, [queries, 1]."""
    size = scale * LOG2E * (np.abs(q) @ np.abs(k).T).max(1, keepdims=True)
    return 2.0 ** (size * (2.0 ** -22 + 2.0 ** -16)) - 1 + P32


def compare_equal_keys(grads, go, q, k, v, mask, what):
    """As the tests' bound for few keys, with the common error of p: ds = p (dp - D)
    with D = sum p dp / sum p of the same p, dp off by 2^-16 of <|go|, |v|>."""
    go, q, k, v = map(f64, (go, q, k, v))
    scale = q.shape[2] ** -0.5
    want = obwd.attention_back(go, q, k, v, scale, mask)
    for h in range(q.shape[1]):
        m = mask if mask.ndim == 2 else mask[h]
        p = obwd.probabilities(q[:, h], k[:, h], scale, m)
        g, vh = go[:, h], v[:, h]
        dp, size = g @ vh.T, 2.0 ** -16 * np.abs(g) @ np.abs(vh).T
        D, eD = ((p * x).sum(1, keepdims=True) for x in (dp, size))
        ep = p_error(q[:, h], k[:, h], scale)
        eds = p * ((HALF + ep) * np.abs(dp - D) + (1 + ep) * (size + eD + P32 * np.abs(D)))
        eds = np.where(m.sum(1, keepdims=True) == 1, 0.0, eds)           # one key: exactly zero
        bounds = (scale * eds @ np.abs(k[:, h]), scale * eds.T @ np.abs(q[:, h]), ((HALF + ep) * p).T @ np.abs(g))
        for name, got, ref, b in zip(("dq", "dk", "dv"), grads, want, bounds):
            err = np.abs(f64(got)[:, h] - ref[:, h])
            bound = b * (1 + HALF) + HALF * np.abs(ref[:, h]) + 1e-30
            assert np.all(err <= bound), f"{what} {name} h={h}: worst err/bound {(err / bound).max()}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("score", SCORES)
def test_one_key(bsa, score, d):  # noqa: F811
    """One token; and 2 x 128 + 1 tokens of which the first and the last block see the last key alone."""
    H = 48
    go, q, k, v = aligned(1, H, d, score, 1)
    idx, cnt = torch.zeros((H, 1, 1), dtype=torch.int32, device="cuda"), torch.ones((H, 1), dtype=torch.int32, device="cuda")
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    assert not grads[0].any() and not grads[1].any()
    compare_equal_keys(grads, go, q, k, v, np.ones((1, 1), dtype=bool), "one token")
    H = 3
    go, q, k, v = aligned(257, H, d, score, 2)
    idx = torch.tensor([[2, -1, -1], [-1, -1, -1], [2, -1, -1]], dtype=torch.int32, device="cuda").expand(H, 3, 3).contiguous()
    cnt = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda").expand(H, 3).contiguous()
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    assert not grads[0].any() and not grads[1].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("score", SCORES)
def test_one_key_of_short_frames(bsa, score, d):  # noqa: F811
    T, H = 300, 2
    go, q, k, v = aligned(T, H, d, score, 3)
    A = [[(7 * t + 3) % T] for t in range(T)]
    frames = torch.full((T, T), -1, dtype=torch.int32)
    frames[:, 0] = torch.tensor([a[0] for a in A], dtype=torch.int32)
    _, _, grads = both(bsa, go, q, k, v, bsa.lvsa_index(T, frames.cuda(), torch.ones(T, dtype=torch.int32, device="cuda")))
    assert bsa.get_device_status() == bsa.BSA_OK
    assert not grads[0].any() and not grads[1].any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("N", [2, 5, 32])
def test_equal_keys(bsa, N, score, d):  # noqa: F811
    """Values that differ by bf16 steps around a common one: dp - D is as small as
    the rounding of o."""
    H = 24
    go, q, k, v = aligned(N, H, d, score, 4 + N)
    g = torch.Generator(device="cuda").manual_seed(N)
    steps = torch.randint(-1, 2, (N, H, d), generator=g, device="cuda", dtype=torch.int16)
    v = (v[:1].expand(N, H, d).contiguous().view(torch.int16) + steps).view(torch.bfloat16)
    idx, cnt = torch.zeros((H, 1, 1), dtype=torch.int32, device="cuda"), torch.ones((H, 1), dtype=torch.int32, device="cuda")
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare_equal_keys(grads, go, q, k, v, np.ones((N, N), dtype=bool), f"N={N} score={score}")


@pytest.mark.parametrize("score", [500.0, -8000.0])
def test_lists_that_split_large_scores(bsa, score):  # noqa: F811
    """Lists that hold some of the keys, with o and lse of all of them: D stays the
    whole row's, whose o is off by h of its terms (twice where the list's own D is
    within that and taken)."""
    N, H, d = 128 + 4, 2, 64
    go, q, k, v = aligned(N, H, d, score, 50)
    full = torch.tensor([0, 1], dtype=torch.int32, device="cuda").expand(H, 2, 2).contiguous()
    two, one = (torch.full((H, 2), n, dtype=torch.int32, device="cuda") for n in (2, 1))
    o, lse = bsa.blocksparse_attn_fwd(q, k, v, bsa.block_index(full, two))
    idx = torch.full((H, 2, 2), -1, dtype=torch.int32, device="cuda")
    idx[:, :, 0] = 1
    grads = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(idx, one))
    assert bsa.get_device_status() == bsa.BSA_OK
    go, q, k, v = map(f64, (go, q, k, v))
    scale = d ** -0.5
    for h in range(H):
        p = obwd.probabilities(q[:, h], k[:, h], scale, np.ones((N, N), dtype=bool))
        g, vh = go[:, h], v[:, h]
        dp, o64, size = g @ vh.T, p @ vh, 2.0 ** -16 * np.abs(g) @ np.abs(vh).T
        D = (g * o64).sum(1, keepdims=True)
        ep = p_error(q[:, h], k[:, h], scale)
        eD = 2.25 * HALF * (np.abs(g) * (np.abs(o64) + (1 + ep) * (p @ np.abs(vh)))).sum(1, keepdims=True)
        ds, eds = p * (dp - D), p * ((HALF + ep) * np.abs(dp - D) + (1 + ep) * (size + eD))
        ref, bound = scale * ds[:, 128:] @ k[128:, h], scale * eds[:, 128:] @ np.abs(k[128:, h])
        assert np.all(np.abs(f64(grads[0])[:, h] - ref) <= bound * (1 + HALF) + HALF * np.abs(ref))
        ref, bound = scale * ds[:, 128:].T @ q[:, h], scale * eds[:, 128:].T @ np.abs(q[:, h])
        assert np.all(np.abs(f64(grads[1])[128:, h] - ref) <= bound * (1 + HALF) + HALF * np.abs(ref))

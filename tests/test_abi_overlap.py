"""The rotation calls refuse outputs that share memory with another tensor, other
than an output that is exactly its own input: host-side, no GPU work is enqueued."""
import ctypes
import random

import pytest
import torch

# an accepted call would launch on these addresses; without a GPU it fails at the launch
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would launch")


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_lvsa_b200 import build
    build.build()
    from block_sparse_attention_lvsa_b200 import binding
    return binding


AT = 1 << 30            # never dereferenced: there is no GPU here, or the call is refused
NUL = ctypes.c_void_p(0)
D = 64


def heads(bsa, at, ts, hs, H=4):
    """`at` in elements of bf16."""
    return bsa.bsa_heads(AT + 2 * at, H, ts, hs)


def rope(bsa):
    r = bsa.bsa_rope()
    r.pairs[0], r.len[0], r.table[0] = 8, 4, AT
    for a in range(3):
        r.grid[a] = 1
    return r


def apply(bsa, x, y, N=16, dtype=0, d=D):
    return bsa.lib().rope_apply(ctypes.byref(x), ctypes.byref(y), dtype, N, d, ctypes.byref(rope(bsa)), 0, NUL)


def ref(t):
    return None if t is None else ctypes.byref(t)


def fwd(bsa, q, k, qo, ko, N=16):
    return bsa.lib().qk_norm_rope_fwd(ref(q), ref(k), ref(qo), ref(ko), 0, N, D, NUL, NUL, 2, 1e-6, None, NUL)


def bwd(bsa, gq, gk, q, k, dq, dk, N=16):
    n = bsa.lib().qk_norm_rope_bwd_workspace_bytes(N, q.H, k.H if k else 0, D)
    return bsa.lib().qk_norm_rope_bwd(ref(gq), ref(gk), ref(q), ref(k), ref(dq), ref(dk), 0, N, D, NUL, NUL, 2, 1e-6,
                                      None, None, None, ctypes.c_void_p(1 << 44), n, NUL)


def test_output_and_its_own_input(bsa):
    A = bsa.BSA_ERR_ARG
    x = heads(bsa, 0, 256, 64)
    assert apply(bsa, x, x) != A                                     # in place
    assert apply(bsa, x, heads(bsa, 16 * 256, 256, 64)) != A         # right behind it
    assert apply(bsa, x, heads(bsa, -16 * 256, 256, 64)) != A        # right before it
    for at in (8, 64, 256, -8, -256, 16 * 256 - 8, -16 * 256 + 8):
        assert apply(bsa, x, heads(bsa, at, 256, 64)) == A, at       # shifted
    y = heads(bsa, 0, 64, 256)                                       # the same memory, tokens and heads exchanged
    assert apply(bsa, heads(bsa, 0, 256, 64), y, N=4) == A
    assert apply(bsa, heads(bsa, 0, 0, 64), x) == A                  # a repeated row and the tensor around it
    assert apply(bsa, heads(bsa, 0, 256, 64), heads(bsa, 0, 512, 64)) == A
    # one token, one head: strides that are never used do not tell tensors apart
    assert apply(bsa, heads(bsa, 0, 256, 64), heads(bsa, 0, 512, 64), N=1) != A
    assert apply(bsa, heads(bsa, 0, 256, 64, H=1), heads(bsa, 0, 256, 128, H=1)) != A
    f32 = [bsa.bsa_heads(AT + 4 * at, 4, 256, 64) for at in (0, 16 * 256, 16 * 256 - 4)]
    assert apply(bsa, f32[0], f32[1], dtype=2) != A and apply(bsa, f32[0], f32[2], dtype=2) == A


def test_slices_of_one_buffer(bsa):
    A = bsa.BSA_ERR_ARG
    for ts, hs, step in [(768, 64, 256), (768, 192, 64), (64, 3072, 1024), (192, 3072, 64), (256, 64, 16 * 256)]:
        # [N, 3, H, d], [N, H, 3, d], [3, H, N, d], [H, N, 3, d] and [3, N, H, d]
        q, k, v = (heads(bsa, i * step, ts, hs) for i in range(3))
        assert apply(bsa, q, k) != A and apply(bsa, v, q) != A
        assert fwd(bsa, q, k, q, k) != A
        assert fwd(bsa, q, k, v, k) != A
        far = [heads(bsa, 10 ** 6 * i, 256, 64) for i in range(1, 5)]
        assert bwd(bsa, far[0], far[1], far[2], far[3], q, k) != A
        assert bwd(bsa, far[0], far[1], q, k, q, k) != A
        assert bwd(bsa, far[0], k, q, v, far[0], k) != A
    # fewer heads of k in the token's row: [N, 4 + 2 + 2, d]
    q, k, v = heads(bsa, 0, 512, 64), heads(bsa, 256, 512, 64, H=2), heads(bsa, 384, 512, 64, H=2)
    assert fwd(bsa, q, k, q, v) != A
    assert fwd(bsa, q, heads(bsa, 256, 512, 128, H=2), heads(bsa, 10 ** 6, 256, 64), heads(bsa, 320, 512, 128, H=2)) != A
    assert fwd(bsa, q, k, q, heads(bsa, 192, 512, 64, H=2)) == A     # k's output over q's last head


def test_outputs_and_other_tensors(bsa):
    A = bsa.BSA_ERR_ARG
    t = [heads(bsa, 10 ** 6 * i, 256, 64) for i in range(8)]
    assert fwd(bsa, t[0], t[1], t[2], t[3]) != A
    assert fwd(bsa, t[0], t[1], t[1], t[2]) == A                     # q's output over k
    assert fwd(bsa, t[0], t[1], t[2], t[0]) == A
    assert fwd(bsa, t[0], t[1], t[2], t[2]) == A                     # one output for both
    assert fwd(bsa, t[0], None, heads(bsa, 256, 256, 64), None) == A
    gq, gk, q, k, dq, dk = t[:6]
    assert bwd(bsa, gq, gk, q, k, dq, dk) != A
    assert bwd(bsa, gq, gk, q, k, gq, k) != A and bwd(bsa, gq, gk, q, k, q, gk) != A
    assert bwd(bsa, gq, gk, q, k, gk, dk) == A and bwd(bsa, gq, gk, q, k, k, dk) == A
    assert bwd(bsa, gq, gk, q, k, dq, gq) == A and bwd(bsa, gq, gk, q, k, dq, q) == A
    assert bwd(bsa, gq, gk, q, k, dq, dq) == A
    assert bwd(bsa, gq, None, q, None, gq, None) != A
    assert bwd(bsa, gq, None, q, None, heads(bsa, 256, 256, 64), None) == A
    assert bwd(bsa, gq, None, q, None, heads(bsa, 2 * 10 ** 6 + 8, 256, 64), None) == A


def elements(at, ts, hs, H, N):
    return {at + n * ts + h * hs + c for n in range(N) for h in range(H) for c in range(0, D, 8)}


def test_against_the_elements_themselves(bsa):
    """Random layouts on a grid of 8 elements: with equal strides, or tokens a row
    apart in both, the answer is exact; other strides may be refused for a shared range."""
    A = bsa.BSA_ERR_ARG
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        N, H = rng.choice([1, 2, 3, 5]), rng.choice([1, 2, 3])
        inner, outer = rng.choice([64, 72, 128, 192]), rng.choice([1, 2, 3])
        ts, hs = (inner * H * outer, inner) if rng.random() < 0.5 else (inner, inner * N * outer)
        at = 8 * rng.randint(-90, 90)
        xs = (ts, hs) if rng.random() < 0.7 else ((ts, rng.choice([64, 128, 200])) if ts > hs else (0, 64))
        x, y = heads(bsa, at, *xs, H=H), heads(bsa, 0, ts, hs, H=H)
        shared = bool(elements(at, *xs, H, N) & elements(0, ts, hs, H, N))
        used = lambda s: (s[0] if N > 1 else 0, s[1] if H > 1 else 0)    # noqa: E731
        same = at == 0 and used(xs) == used((ts, hs))
        got = apply(bsa, x, y, N=N) == A
        if shared and not same:
            assert got, (N, H, at, xs, ts, hs)
        elif same or used(xs)[0] == used((ts, hs))[0]:
            assert not got, (N, H, at, xs, ts, hs)
        seen[shared] += 1
    assert min(seen.values()) > 500

"""Refusals of the rotation calls: host-side validation through the C ABI (no
GPU work is enqueued) and the binding's own checks."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_lvsa_b200 import build
    build.build()
    from block_sparse_attention_lvsa_b200 import binding
    return binding


FAKE = 0x10000          # never dereferenced: rejected on the host first
NUL = ctypes.c_void_p(0)


def heads(bsa, data=FAKE, H=2, ts=256, hs=128):
    return bsa.bsa_heads(data, H, ts, hs)


def rope(bsa, **kw):
    r = bsa.bsa_rope()
    r.pairing = kw.get("pairing", 0)
    for a in range(3):
        r.pairs[a] = kw.get("pairs", (22, 21, 21))[a]
        r.len[a] = kw.get("len", (4, 4, 4))[a]
        r.table[a] = kw.get("table", (FAKE,) * 3)[a]
        r.grid[a] = kw.get("grid", (2, 3, 4))[a]
        r.first[a] = kw.get("first", (0, 0, 0))[a]
    r.pos = kw.get("pos")
    return r


def test_table_arguments(bsa):
    f = bsa.lib().rope_build_table
    p = ctypes.c_void_p(FAKE)
    for args in [(0, 4, 1e4, 0.0, 1.0, p), (4, 0, 1e4, 0.0, 1.0, p), (4, 4, 0.0, 0.0, 1.0, p),
                 (4, 4, float("nan"), 0.0, 1.0, p), (4, 4, 1e4, float("inf"), 1.0, p),
                 (4, 4, 1e4, 0.0, float("nan"), p), (4, 4, 1e4, 0.0, 1.0, NUL),
                 (4, 4, 1e4, 0.0, 1.0, ctypes.c_void_p(FAKE + 4))]:
        assert f(*args, NUL) == bsa.BSA_ERR_ARG


def apply(bsa, x=None, y=None, dtype=0, N=24, d=128, r=None):
    x, y, r = x or heads(bsa), y or heads(bsa, FAKE * 2), r or rope(bsa)
    return bsa.lib().rope_apply(ctypes.byref(x), ctypes.byref(y), dtype, N, d, ctypes.byref(r), 0, NUL)


def test_rope_apply_arguments(bsa):
    A, S, U = bsa.BSA_ERR_ARG, bsa.BSA_ERR_SHAPE, bsa.BSA_ERR_UNSUPPORTED
    assert apply(bsa, dtype=3) == A
    assert apply(bsa, N=0) == A
    assert apply(bsa, d=96) == U
    assert apply(bsa, x=heads(bsa, 0)) == A
    assert apply(bsa, x=heads(bsa, FAKE + 8)) == A                    # misaligned
    assert apply(bsa, x=heads(bsa, ts=258)) == A                      # 516 bytes: not a multiple of 16
    assert apply(bsa, x=heads(bsa, hs=-128)) == A
    assert apply(bsa, x=heads(bsa, H=3)) == S                         # H differs
    assert apply(bsa, y=heads(bsa, ts=128, hs=128)) == A              # output rows overlap
    assert apply(bsa, y=heads(bsa, ts=0, hs=128)) == A
    assert apply(bsa, y=heads(bsa, ts=64, hs=64 * 24)) == A
    assert apply(bsa, x=heads(bsa, ts=1 << 60)) == U
    assert apply(bsa, r=rope(bsa, pairing=2)) == A
    assert apply(bsa, r=rope(bsa, pairs=(22, -1, 21))) == A
    assert apply(bsa, r=rope(bsa, pairs=(0, 0, 0))) == S
    assert apply(bsa, r=rope(bsa, pairs=(22, 22, 21))) == S           # 65 pairs of 64
    assert apply(bsa, r=rope(bsa, table=(FAKE, 0, FAKE))) == A
    assert apply(bsa, r=rope(bsa, table=(FAKE, FAKE + 4, FAKE))) == A
    assert apply(bsa, r=rope(bsa, len=(4, 0, 4))) == A
    assert apply(bsa, r=rope(bsa, grid=(2, 3, 5))) == S               # 30 tokens of 24
    assert apply(bsa, r=rope(bsa, grid=(2, 0, 4))) == A
    assert apply(bsa, r=rope(bsa, first=(0, 0, 1))) == S              # past the table
    assert apply(bsa, r=rope(bsa, first=(-1, 0, 0))) == A
    big = heads(bsa, ts=256)
    assert apply(bsa, x=big, y=big, N=1 << 33, r=rope(bsa, grid=(1 << 11, 1 << 11, 1 << 11), len=(4096,) * 3)) == S


def test_norm_rope_arguments(bsa):
    A, S, W = bsa.BSA_ERR_ARG, bsa.BSA_ERR_SHAPE, bsa.BSA_ERR_WORKSPACE
    f, b = bsa.lib().qk_norm_rope_fwd, bsa.lib().qk_norm_rope_bwd
    h = lambda **kw: ctypes.byref(heads(bsa, **kw))                   # noqa: E731
    r = ctypes.byref(rope(bsa))
    p = ctypes.c_void_p(FAKE)
    ok = dict(wtype=2, eps=1e-6)

    def fwd(q=None, k=None, qo=None, ko=None, wq=p, wk=p, wtype=2, eps=1e-6):
        return f(q or h(), k or h(), qo or h(), ko or h(), 0, 24, 128, wq, wk, wtype, eps, r, NUL)

    assert fwd(eps=0.0) == A and fwd(eps=float("nan")) == A and fwd(eps=float("inf")) == A
    assert fwd(wtype=1) == A                                          # neither fp32 nor the tensors' bf16
    assert fwd(wq=ctypes.c_void_p(FAKE + 4)) == A
    assert fwd(ko=h(H=4, ts=512)) == S
    assert f(h(), None, h(), h(), 0, 24, 128, p, p, 2, 1e-6, r, NUL) == A
    del ok
    n = bsa.lib().qk_norm_rope_bwd_workspace_bytes(24, 2, 2, 128)
    assert n > 0 and bsa.lib().qk_norm_rope_bwd_workspace_bytes(24, 2, 2, 96) == ctypes.c_size_t(-1).value

    def bwd(ws=p, n=n, gk=True, dwk=p, gq=None):
        return b(gq or h(), h() if gk else None, h(), h(), h(), h(), 0, 24, 128, p, p, 2, 1e-6, r, p, dwk, ws, n, NUL)

    assert bwd(n=n - 1) == W and bwd(ws=NUL) == W and bwd(ws=ctypes.c_void_p(FAKE + 16)) == W
    assert bwd(gk=False) == A
    assert bwd(gq=h(H=1)) == S
    assert b(h(), None, h(), None, h(), None, 0, 24, 128, p, NUL, 2, 1e-6, r, p, p, p, n, NUL) == A   # dwk without k


def test_binding_refuses_cpu_and_wrong_tensors(bsa):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsa.qk_norm_rope_fwd(x, x)                                    # not on a CUDA device
    with pytest.raises(ValueError):
        bsa.rope_axes([torch.zeros((4, 8, 2))], grid=(4,))            # table not on a CUDA device
    with pytest.raises(ValueError):
        bsa.rope_axes([], grid=())
    with pytest.raises(ValueError):
        bsa.rope_axes([torch.zeros((4, 8, 2))], grid=(4,), pairing="interleaved")
    with pytest.raises(ValueError):
        bsa.rope_build_table(0, 4, device="cuda:0")


def test_packed_rope_fills_the_struct_field_by_field(bsa):
    """The one-call packing puts every value where the struct has its field."""
    assert bsa._ROPE.size == ctypes.sizeof(bsa.bsa_rope)
    r = bsa.bsa_rope.from_buffer_copy(bsa._ROPE.pack(*range(1, 18)))
    seen = []
    for name, kind in bsa.bsa_rope._fields_:
        v = getattr(r, name)
        seen += list(v) if issubclass(kind, ctypes.Array) else [v]
    assert seen == list(range(1, 18))

"""Refusals of blocksparse_attn_bwd, on the host before any launch."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_lvsa_b200 import build
    build.build()
    from block_sparse_attention_lvsa_b200 import binding
    return binding


def test_arguments(bsa):
    f = bsa.lib().blocksparse_attn_bwd
    nul = ctypes.c_void_p(0)
    ix = bsa.bsa_index()
    ix.kind, ix.block, ix.H, ix.nQB, ix.nKB, ix.idx, ix.cnt = bsa.BSA_INDEX_BLOCKS, 128, 2, 4, 4, 0x10000, 0x10000
    need = bsa.workspace_bytes(bsa.BSA_OP_BLOCKSPARSE_BWD, 512, 2, 64, ix)
    # padded rows of nl and nd, bit sets, counts and lists
    assert need >= 2 * 2 * 512 * 4 + 2 * 4 * 4 + 2 * 4 * 4 + 2 * 16 * 4 and need % 256 == 0
    at = {n: 0x1000000 * (i + 1) for i, n in enumerate(("go", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws"))}

    def call(N=512, H=2, d=64, scale=0.1, index=ix, n=need, oH=2, ots=128, ohs=64, **kw):
        p = {k: ctypes.c_void_p(kw.get(k, v)) for k, v in at.items()}
        o = bsa.bsa_heads(p["o"].value, oH, ots, ohs)
        return f(p["go"], p["q"], p["k"], p["v"], ctypes.byref(o), p["lse"], N, H, d, scale,
                 None if index is None else ctypes.byref(index), p["dq"], p["dk"], p["dv"], p["ws"], n, nul)

    A, S, U, W = bsa.BSA_ERR_ARG, bsa.BSA_ERR_SHAPE, bsa.BSA_ERR_UNSUPPORTED, bsa.BSA_ERR_WORKSPACE
    for name in ("go", "q", "k", "v", "o", "lse", "dq", "dk", "dv"):
        assert call(**{name: 0}) == A, name
    for name in ("go", "q", "k", "v", "o", "dq", "dk", "dv"):
        assert call(**{name: at[name] + 8}) == A, name
    assert call(index=None) == A and call(scale=float("nan")) == A and call(scale=0.0) == A and call(scale=-0.2) == A and call(N=0) == A
    assert call(d=96) == U
    assert call(dq=at["q"]) == A and call(dk=at["go"] + 64) == A and call(dv=at["dk"]) == A
    assert call(dv=at["lse"]) == A and call(dq=at["o"]) == A
    assert call(ots=64, ohs=512 * 64, dk=at["o"] + 512 * 2 * 64) == A   # inside o laid out heads first
    assert call(oH=1) == S and call(ots=130) == A and call(ohs=-64) == A
    assert call(n=need - 1) == W and call(ws=0) == W and call(ws=at["ws"] + 16) == W
    ix.nKB = 5
    assert call() == S and call(n=0) == S
    ix.nKB, ix.block = 4, 64
    assert call() == U and call(n=0) == U
    ix.kind = 9
    assert call() == A
    fx = bsa.bsa_index()
    fx.kind, fx.T, fx.frames, fx.counts = bsa.BSA_INDEX_LVSA_FRAMES, 7, 0x10000, 0x10000
    assert call(index=fx) == S                                     # 7 does not divide 512
    fx.T = 8
    need = bsa.workspace_bytes(bsa.BSA_OP_BLOCKSPARSE_BWD, 512, 2, 64, fx)
    assert call(index=fx, n=need - 1) == W
    fx.frames = None
    assert call(index=fx, n=need) == A


def test_binding_checks(bsa):
    t = torch.zeros((10, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsa.blocksparse_attn_bwd(t, t, t, t, t, torch.zeros((2, 10)), bsa.bsa_index())

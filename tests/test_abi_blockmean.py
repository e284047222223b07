"""Refusals of blockmean_select, on the host before any launch."""
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
    f = bsa.lib().blockmean_select
    p, nul = ctypes.c_void_p(0x10000), ctypes.c_void_p(0)
    n = bsa.lib().blockmean_select_workspace_bytes(1000, 2, 64)
    A, U, W = bsa.BSA_ERR_ARG, bsa.BSA_ERR_UNSUPPORTED, bsa.BSA_ERR_WORKSPACE

    def call(q=p, k=p, N=1000, H=2, d=64, block=128, keep=2, local=0, idx=p, cnt=p, ws=p, n=n):
        return f(q, k, N, H, d, block, keep, local, idx, cnt, ws, n, nul)

    assert call(q=nul) == A and call(k=nul) == A and call(idx=nul) == A and call(cnt=nul) == A
    assert call(q=ctypes.c_void_p(0x10008)) == A
    assert call(N=0) == A and call(H=0) == A and call(keep=0) == A and call(local=-2) == A
    assert call(d=96) == U and call(N=1, H=40000) == U and call(block=64) == U
    assert call(N=128 * 8192 + 1, H=1) == U and call(N=1 << 20, H=64) == U
    assert call(n=n - 1) == W and call(ws=nul) == W and call(ws=ctypes.c_void_p(0x10010)) == W
    none = ctypes.c_size_t(-1).value
    g = bsa.lib().blockmean_select_workspace_bytes
    assert g(0, 1, 64) == none and g(10, 1, 32) == none and g(128 * 8192 + 1, 1, 64) == none
    assert n % 256 == 0 and n >= 2 * 2 * 8 * 64 * 8


def test_binding_checks(bsa):
    q = torch.zeros((10, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsa.blockmean_select(q, q, 1)

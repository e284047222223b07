"""GPU: key blocks by block means, bit-exact against the float64 oracle, and the
attention over them."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import blockmean as obm
from block_sparse_attention_lvsa_b200 import inputs
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_lvsa_b200 import binding
    assert torch.cuda.is_available()
    return binding


def f64(t):
    return t.detach().cpu().double().numpy()


def check(bsa, q, k, keep, local, what=""):
    idx, cnt = bsa.blockmean_select(q, k, keep, local)
    assert bsa.get_device_status() == bsa.BSA_OK
    ridx, rcnt = obm.select(f64(q), f64(k), keep, local)
    assert np.array_equal(cnt.cpu().numpy(), rcnt), what
    assert np.array_equal(idx.cpu().numpy(), ridx), what
    return idx, cnt


@pytest.mark.parametrize("N,H,d", [(1, 1, 64), (127, 3, 128), (128, 2, 64), (129, 1, 128), (1000, 5, 64),
                                   (4097, 3, 128), (16001, 2, 128), (33300, 1, 64)])
@pytest.mark.parametrize("keep,local", [(1, -1), (1, 0), (3, 1), (40, 2), (10 ** 6, 0)])
def test_select(bsa, N, H, d, keep, local):
    q, k, _ = inputs.make_qkv(N, H, d, seed=N + d, device="cuda")
    check(bsa, q, k, keep, local)


@pytest.mark.parametrize("locality", [0.0, 2.0])
def test_select_with_temporal_locality(bsa, locality):
    """The frame structure moves a row's scores far from its spread's size."""
    q, k, _ = inputs.make_qkv(21 * 1560, 2, 128, seed=4, device="cuda", T=21, locality=locality)
    check(bsa, q, k, 32, 1)


def test_equal_blocks_tie_to_the_lower_index(bsa):
    q, k, _ = inputs.make_qkv(128 * 40, 2, 64, seed=5, device="cuda")
    for j in range(40):
        k[128 * j:128 * (j + 1)] = k[128 * (j % 3):128 * (j % 3 + 1)].clone()
    idx, cnt = check(bsa, q, k, 11, -1)
    check(bsa, torch.zeros_like(q), k, 7, 0)                 # every score equal
    check(bsa, -torch.zeros_like(q), k, 7, 0)


def test_close_scores_are_told_apart(bsa):
    """Blocks whose means differ in one bf16 step of one value: far below what
    32-bit scores tell apart next to a large common part."""
    q, k, _ = inputs.make_qkv(128 * 64, 1, 128, seed=6, device="cuda")
    one = k[:128].clone() * 30
    g = np.random.default_rng(7)
    for j in range(64):
        k[128 * j:128 * (j + 1)] = one
        t, c = int(g.integers(128)), int(g.integers(128))
        k[128 * j + t, 0, c] *= 1 + 2.0 ** -7 * (1 + j % 2)
    check(bsa, q * 30, k, 20, 0)


def test_large_small_and_not_finite(bsa):
    q, k, _ = inputs.make_qkv(128 * 12, 2, 64, seed=8, device="cuda")
    k[128 * 2, 0, 3] = 3e38                                   # a wide block sum: 64 bits hold it
    check(bsa, q, k, 4, 0)
    check(bsa, (q.float() * 1e-20).bfloat16(), (k.float() * 1e-18).bfloat16(), 4, 0)
    check(bsa, (q.float() * 1e-30).bfloat16(), (k.float() * 1e-10).bfloat16(), 4, 0)
    k[128 * 4 + 5, 1, 7] = float("nan")
    k[128 * 5 + 5, 1, 7] = float("inf")
    k[128 * 6 + 5, 1, 7] = -float("inf")
    q[128 * 9 + 1, 0, 0] = float("nan")
    check(bsa, q, k, 4, 0)


def test_longest_rows(bsa):
    """8192 blocks: the longest row, and one past it is refused."""
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k = (torch.randn((128 * 8192, 1, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    idx, cnt = bsa.blockmean_select(q, k, 100, 0)
    mq, mk = (x.double().view(8192, 128, 64).mean(1) for x in (q, k))
    rows = [0, 1, 4095, 8191]
    s = f64(mq[rows] @ mk.T)
    for n, i in enumerate(rows):
        assert idx[0, i, :100].tolist() == obm.keep_row(list(s[n]), i, 100, 0)
        assert bool((idx[0, i, 100:] == -1).all()) and int(cnt[0, i]) == 100
    big = torch.zeros((128 * 8192 + 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bsa.BsaError):
        bsa.blockmean_select(big, big, 1)


@pytest.mark.parametrize("N", [128 * 300, 128 * 700 - 5, 128 * 1537, 128 * 2048, 128 * 2100 + 1])
def test_row_lengths(bsa, N):
    """Rows in registers and in shared memory, with many and with few candidates
    at the border (every second block of k is a copy of another)."""
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k = (torch.randn((N, 1, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    nB = -(-N // 128)
    for copies in (False, True):
        if copies:
            for j in range(1, nB - 1, 2):
                k[128 * j:128 * (j + 1)] = k[:128]
        idx, cnt = bsa.blockmean_select(q, k, nB // 3, 1)
        assert bsa.get_device_status() == bsa.BSA_OK
        m = []
        for x in (q, k):
            p = torch.zeros((nB * 128, 64), dtype=torch.float64, device="cuda")
            p[:N] = x[:, 0].double()
            s = p.view(nB, 128, 64).sum(1)
            s[-1] /= N - (nB - 1) * 128
            s[:-1] /= 128
            m.append(f64(s))
        for i in sorted({0, 1, nB // 2, nB - 2, nB - 1} | set(range(0, nB, 97))):
            # each score by itself: equal blocks get equal scores, whatever order a library adds in
            sc = [float((m[0][i] * m[1][j]).sum()) for j in range(nB)]
            n = int(cnt[0, i])
            assert idx[0, i, :n].tolist() == obm.keep_row(sc, i, nB // 3, 1), (copies, i)
            assert bool((idx[0, i, n:] == -1).all())


def test_full_size_step(bsa):
    """One head's rows of the 6x-horizon shape among all 12 heads."""
    q, k, _ = inputs.make_qkv(196560, 12, 128, seed=10, device="cuda")
    idx, cnt = bsa.blockmean_select(q, k, 256, 1)
    nB = 1536
    assert bool((cnt == 256).all())
    for h in (0, 11):
        m = []
        for x in (q, k):
            p = torch.zeros((nB * 128, 128), dtype=torch.float64, device="cuda")
            p[:196560] = x[:, h].double()
            s = p.view(nB, 128, 128).sum(1)
            s[-1] /= 196560 - 1535 * 128
            s[:-1] /= 128
            m.append(s)
        sc = f64(m[0] @ m[1].T)
        for i in list(range(0, nB, 97)) + [nB - 1]:
            assert idx[h, i, :256].tolist() == obm.keep_row(list(sc[i]), i, 256, 1)


def test_chosen_blocks_feed_the_attention(bsa):
    N, H, d = 1300, 2, 128
    q, k, v = inputs.make_qkv(N, H, d, seed=11, device="cuda")
    idx, cnt = bsa.blockmean_select(q, k, 4, 1)
    o, lse = bsa.blocksparse_attn_fwd(q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    mask = np.zeros((H, N, N), dtype=bool)
    I, C = idx.cpu().numpy(), cnt.cpu().numpy()
    for h in range(H):
        for i in range(I.shape[1]):
            for j in I[h, i, :C[h, i]]:
                mask[h, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = True
    O, L = oatt.attention_dense_masked(f64(q), f64(k), f64(v), d ** -0.5, mask)
    err = np.abs(f64(o) - O)
    assert err.max() <= gu.O_MAX and err.mean() <= gu.O_MEAN
    assert np.abs(f64(lse) - L).max() <= gu.LSE_MAX


def test_stream_graph_and_own_buffers(bsa):
    q, k, _ = inputs.make_qkv(5000, 3, 64, seed=12, device="cuda")
    ref = bsa.blockmean_select(q, k, 9, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bsa.blockmean_select(q, k, 9, 1, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    idx, cnt = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bsa.blockmean_select(q, k, 9, 1, idx=idx, cnt=cnt)
    for _ in range(2):
        idx.fill_(-7)
        cnt.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, ref[0]) and torch.equal(cnt, ref[1])
    room = torch.full((ref[0].numel() + 2,), -7, dtype=torch.int32, device="cuda")    # a list off the 16-byte grid
    odd = room[1:-1].view(ref[0].shape)
    bsa.blockmean_select(q, k, 9, 1, idx=odd)
    assert torch.equal(odd, ref[0]) and room[0] == -7 and room[-1] == -7
    with pytest.raises(ValueError):
        bsa.blockmean_select(q, k, 9, idx=idx[:, :, :-1])
    with pytest.raises(bsa.BsaError):
        bsa.blockmean_select(q, k, 9, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(bsa.BsaError):
        bsa.blockmean_select(q, k, 0)
    with pytest.raises(bsa.BsaError):
        bsa.blockmean_select(q, k, 1, block=64)


def test_over_budget_is_a_warning(bsa):
    q, k, _ = inputs.make_qkv(1000, 1, 64, seed=13, device="cuda")
    idx = torch.empty((1, 8, 8), dtype=torch.int32, device="cuda")
    cnt = torch.empty((1, 8), dtype=torch.int32, device="cuda")
    n = bsa.lib().blockmean_select_workspace_bytes(1000, 1, 64)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())               # noqa: E731
    call = lambda keep, local: bsa.lib().blockmean_select(    # noqa: E731
        p(q), p(k), 1000, 1, 64, 128, keep, local, p(idx), p(cnt), p(ws), n,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert call(2, 1) == bsa.BSA_WARN_OVER_BUDGET
    assert cnt[0].tolist() == [2, 3, 3, 3, 3, 3, 3, 2]
    assert call(3, 1) == bsa.BSA_OK
    assert call(100, 10 ** 9) == bsa.BSA_OK and cnt[0].tolist() == [8] * 8


@pytest.mark.parametrize("N,H,d", [(128 * 1537, 1, 64), (128 * 700 - 5, 2, 64), (128 * 300, 3, 128)])
def test_repeated_calls_agree(bsa, N, H, d):
    """q and k in L2, where the pooling's loads are fastest: a box of its ring that
    is written again too early would change means, and with them the choice."""
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k = (torch.randn((N, H, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    nB = -(-N // 128)
    first = bsa.blockmean_select(q, k, nB // 3, 1)
    idx, cnt = (torch.empty_like(x) for x in first)
    for _ in range(60):
        bsa.blockmean_select(q, k, nB // 3, 1, idx=idx, cnt=cnt)
        assert torch.equal(idx, first[0]) and torch.equal(cnt, first[1])
    assert bsa.get_device_status() == bsa.BSA_OK

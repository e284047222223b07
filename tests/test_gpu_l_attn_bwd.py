"""GPU: gradient of the block-sparse attention against the float64 oracle, for
the three kinds of index.

Tolerance, by counting roundings (bf16: half a step is at most h = 2^-8 of the
value; 32-bit scores, exponentials and lse move p by less than 2^-13 of itself):
  dv: h |dv| for the store, (h + 2^-13) sum p |go| for the bf16 p;
  ds: h |ds| for its bf16 form, 2^-13 p (|dp| + |D|) for p, and p eD, where D
      comes from the forward's o: its store and its own bf16 p give
      eD = h sum_c |go_c| (|o_c| + sum_k p |v_kc|);
  dq = scale sum ds k, dk = scale sum ds q: those errors times |k|, |q|, plus
      h of the value for the store.
"""
import numpy as np
import pytest
import torch

from oracle import attention_bwd as obwd
from oracle import blockmean as obm
from oracle import lvsa as olvsa
from block_sparse_attention_lvsa_b200 import inputs

pytestmark = pytest.mark.gpu

HALF, P32 = 2.0 ** -8, 2.0 ** -13


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_lvsa_b200 import binding
    assert torch.cuda.is_available()
    return binding


def f64(t):
    return t.detach().cpu().double().numpy()


def make(N, H, d, seed, scale=1.0):
    q, k, v = inputs.make_qkv(N, H, d, seed=seed, device="cuda")
    go = inputs.make_qkv(N, H, d, seed=seed + 1, device="cuda")[0]
    return [(x.float() * s).bfloat16() for x, s in ((go, 1.0), (q, scale), (k, scale), (v, 1.0))]


def compare(grads, go, q, k, v, scale, mask, what):
    go, q, k, v = map(f64, (go, q, k, v))
    want = obwd.attention_back(go, q, k, v, scale, mask)
    for h in range(q.shape[1]):
        p = obwd.probabilities(q[:, h], k[:, h], scale, mask if mask.ndim == 2 else mask[h])
        g, vh = go[:, h], v[:, h]
        dp, o = g @ vh.T, p @ vh
        D = (g * o).sum(1, keepdims=True)
        eD = HALF * (np.abs(g) * (np.abs(o) + p @ np.abs(vh))).sum(1, keepdims=True)
        eds = HALF * np.abs(p * (dp - D)) + P32 * p * (np.abs(dp) + np.abs(D)) + p * eD
        bounds = (abs(scale) * eds @ np.abs(k[:, h]), abs(scale) * eds.T @ np.abs(q[:, h]), (HALF + P32) * p.T @ np.abs(g))
        for name, got, ref, b in zip(("dq", "dk", "dv"), grads, want, bounds):
            err = np.abs(f64(got)[:, h] - ref[:, h])
            bound = b * (1 + HALF) + HALF * np.abs(ref[:, h]) + 1e-30
            assert np.all(err <= bound), f"{what} {name} h={h}: worst err/bound {(err / bound).max()}"


def block_mask(idx, cnt, N):
    idx, cnt = idx.cpu().numpy(), cnt.cpu().numpy()
    mask = np.zeros((idx.shape[0], N, N), dtype=bool)
    for h in range(idx.shape[0]):
        for i in range(idx.shape[1]):
            for j in idx[h, i, :cnt[h, i]]:
                if 0 <= j < idx.shape[2]:
                    mask[h, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] = True
    return mask


def both(bsa, go, q, k, v, ix, scale=None, **kw):
    o, lse = bsa.blocksparse_attn_fwd(q, k, v, ix, scale=scale)
    grads = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix, scale=scale, **kw)
    return o, lse, grads


def random_lists(H, nB, density, seed):
    g = torch.Generator().manual_seed(seed)
    on = torch.rand((H, nB, nB), generator=g) < density
    cnt = on.sum(2).to(torch.int32)
    at = torch.where(on, torch.arange(nB), nB).sort(2).values
    return torch.where(at < nB, at, -1).to(torch.int32).cuda(), cnt.cuda()


@pytest.mark.parametrize("N,H,d,density", [(1, 1, 64, 1.0), (1, 2, 128, 1.0), (100, 1, 128, 1.0), (128, 2, 64, 1.0),
                                           (129, 1, 64, 1.0), (700, 2, 128, 0.5), (1001, 3, 64, 0.3),
                                           (1280, 2, 128, 0.15), (4500, 1, 128, 0.4)])
def test_block_lists(bsa, N, H, d, density):
    """Random lists: rows and columns without a block among them."""
    go, q, k, v = make(N, H, d, seed=N + d)
    nB = -(-N // 128)
    idx, cnt = random_lists(H, nB, density, N)
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare(grads, go, q, k, v, d ** -0.5, block_mask(idx, cnt, N), f"N={N}")


@pytest.mark.parametrize("T,P,H,d,C", [(1, 1, 1, 64, 1), (8, 64, 2, 64, 4), (5, 150, 2, 128, 2), (13, 37, 1, 128, 5),
                                       (700, 1, 1, 64, 50), (3, 700, 1, 128, 1), (21, 97, 2, 64, 7)])
def test_frame_sets(bsa, T, P, H, d, C):
    go, q, k, v = make(T * P, H, d, seed=T)
    frames, counts, _ = bsa.lvsa_build_index(T, 4, 3, C, 1, device="cuda")
    A, _ = olvsa.attended_frames(T, 4, 3, C, 1)
    _, _, grads = both(bsa, go, q, k, v, bsa.lvsa_index(T, frames, counts))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare(grads, go, q, k, v, d ** -0.5, olvsa.dense_token_mask(A, P, T * P), f"T={T}")


def test_frame_sets_one_sided_and_empty(bsa):
    """Frames seen by nobody, frames that see nobody: the transposed lists differ from the lists."""
    T, P, H, d = 6, 90, 2, 64
    go, q, k, v = make(T * P, H, d, seed=30)
    A = [[0, 5], [], [1], [0, 1, 2, 3], [5], []]
    frames = torch.full((T, T), -1, dtype=torch.int32)
    for t, a in enumerate(A):
        frames[t, :len(a)] = torch.tensor(a, dtype=torch.int32)
    counts = torch.tensor([len(a) for a in A], dtype=torch.int32)
    ix = bsa.lvsa_index(T, frames.cuda(), counts.cuda())
    _, lse, grads = both(bsa, go, q, k, v, ix)
    assert bsa.get_device_status() == bsa.BSA_OK
    assert bool((lse[:, P:2 * P] == -float("inf")).all())
    assert bool((grads[0][P:2 * P] == 0).all())
    for x in grads[1:]:
        assert bool((x[4 * P:5 * P] == 0).all())
    compare(grads, go, q, k, v, d ** -0.5, olvsa.dense_token_mask(A, P, T * P), "one-sided")


@pytest.mark.parametrize("d", [64, 128])
def test_frames_within_blocks(bsa, d):
    T, P, H = 9, 110, 2
    N = T * P
    go, q, k, v = make(N, H, d, seed=40 + d)
    frames, counts, _ = bsa.lvsa_build_index(T, 3, 2, 4, 0, device="cuda")
    A, _ = olvsa.attended_frames(T, 3, 2, 4, 0)
    idx, cnt = random_lists(H, -(-N // 128), 0.6, 5)
    _, _, grads = both(bsa, go, q, k, v, bsa.lvsa_block_index(T, frames, counts, idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare(grads, go, q, k, v, d ** -0.5, olvsa.dense_token_mask(A, P, N)[None] & block_mask(idx, cnt, N), "both")


@pytest.mark.parametrize("scale", [1.0, 1e-3])
def test_other_scales(bsa, scale):
    """Peaked rows (probabilities near 0 and 1) and flat ones; a scale that is not positive is refused."""
    N, H, d = 600, 2, 64
    go, q, k, v = make(N, H, d, seed=50)
    idx, cnt = random_lists(H, 5, 0.7, 6)
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt), scale=scale)
    assert bsa.get_device_status() == bsa.BSA_OK
    compare(grads, go, q, k, v, scale, block_mask(idx, cnt, N), f"scale={scale}")
    with pytest.raises(bsa.BsaError):
        bsa.blocksparse_attn_bwd(go, q, k, v, *bsa.blocksparse_attn_fwd(q, k, v, bsa.block_index(idx, cnt)),
                                 bsa.block_index(idx, cnt), scale=-scale)


def test_lists_out_of_order_and_bad_entries(bsa):
    N, H, d = 640, 1, 128
    go, q, k, v = make(N, H, d, seed=60)
    idx, cnt = random_lists(H, 5, 1.0, 7)
    a = bsa.block_index(idx, cnt)
    o, lse = bsa.blocksparse_attn_fwd(q, k, v, a)
    ref = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, a)
    back = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(idx.flip(2).contiguous(), cnt))
    assert torch.equal(ref[1], back[1]) and torch.equal(ref[2], back[2])       # the transposed lists are the same
    compare(back, go, q, k, v, d ** -0.5, np.ones((N, N), dtype=bool), "any order")
    assert bsa.get_device_status() == bsa.BSA_OK
    bad = idx.clone()
    bad[0, 2, 1], bad[0, 3, 0], bad[0, 4, 4] = 99, -5, 5
    few = bsa.block_index(bad, cnt)
    o, lse = bsa.blocksparse_attn_fwd(q, k, v, few)
    bsa.get_device_status()
    got = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, few)
    assert bsa.get_device_status() == bsa.BSA_ERR_INDEX_RANGE
    compare(got, go, q, k, v, d ** -0.5, block_mask(bad, cnt, N), "bad entries skipped")
    twice = idx.clone()
    twice[0, 1, 1] = twice[0, 1, 0]
    bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(twice, cnt))
    assert bsa.get_device_status() == bsa.BSA_ERR_INDEX_RANGE
    over = cnt.clone()
    over[0, 0] = 77
    bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(idx, over))
    assert bsa.get_device_status() == bsa.BSA_ERR_INDEX_RANGE


def test_unlisted_tiles_are_not_read(bsa):
    """Not-a-number in a key block that no list holds, and in q of a block with an empty list."""
    N, H, d = 512, 1, 64
    go, q, k, v = make(N, H, d, seed=70)
    idx = torch.tensor([[[0, 1, -1, -1], [1, 3, -1, -1], [-1] * 4, [0, 3, -1, -1]]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([[2, 2, 0, 2]], dtype=torch.int32, device="cuda")
    ix = bsa.block_index(idx, cnt)
    ref = both(bsa, go, q, k, v, ix)
    k2, v2, q2, go2 = (x.clone() for x in (k, v, q, go))
    k2[256:384], v2[256:384], q2[256:384] = float("nan"), float("inf"), float("nan")
    go2[256:384] = 0
    got = both(bsa, go2, q2, k2, v2, ix)
    assert all(torch.equal(a, b) for a, b in zip(ref[2], got[2]))


def test_repeats_stream_graph_and_workspace(bsa):
    N, H, d = 2000, 3, 128
    go, q, k, v = make(N, H, d, seed=80)
    idx, cnt = random_lists(H, 16, 0.4, 8)
    ix = bsa.block_index(idx, cnt)
    o, lse, ref = both(bsa, go, q, k, v, ix)
    need = bsa.workspace_bytes(bsa.BSA_OP_BLOCKSPARSE_BWD, N, H, d, ix)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")          # whatever was there before
    room = torch.full((3, N + 64, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    outs = [room[i, :N] for i in range(3)]
    got = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and bool((room[:, N:] == 5.0).all())
    heads_first = o.transpose(0, 1).contiguous().transpose(0, 1)              # o by strides
    got = bsa.blocksparse_attn_bwd(go, q, k, v, heads_first, lse, ix)
    assert not heads_first.is_contiguous() and all(torch.equal(a, b) for a, b in zip(ref, got))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graphs, res = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(both(bsa, go, q, k, v, ix)[2])
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for r in res:
        assert all(torch.equal(a, b) for a, b in zip(ref, r))
    with pytest.raises(bsa.BsaError):
        bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix, workspace=ws[:need - 256])
    with pytest.raises(bsa.BsaError):                                          # outputs over an input, over one another
        bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix, dq=q)
    with pytest.raises(bsa.BsaError):
        bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix, dk=outs[0], dv=outs[0])
    with pytest.raises(ValueError):
        bsa.blocksparse_attn_bwd(go, q, k, v, o, lse.t(), ix)
    with pytest.raises(ValueError):
        bsa.blocksparse_attn_bwd(go[:-1], q, k, v, o, lse, ix)
    with pytest.raises(bsa.BsaError):
        bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(idx[:, :15, :15].contiguous(), cnt[:, :15].contiguous()))


def test_many_calls_in_a_row(bsa):
    """The groups of threads run ahead of one another differently from call to
    call; every call ends, with the same result (both head sizes, masks in every
    tile)."""
    for d in (64, 128):
        T, P = 21, 157
        go, q, k, v = make(T * P, 4, d, seed=85)
        frames, counts, _ = bsa.lvsa_build_index(T, 5, 3, 7, 0, device="cuda")
        ix = bsa.lvsa_index(T, frames, counts)
        o, lse, ref = both(bsa, go, q, k, v, ix)
        for _ in range(300):
            got = bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, ix)
        assert bsa.get_device_status() == bsa.BSA_OK
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_two_streams_at_once(bsa):
    """The whole chain on two streams at the same time, scratch from each stream's own pool."""
    N, H, d = 3000, 4, 128
    g = torch.Generator(device="cuda").manual_seed(95)
    x = [torch.randn((N, 3, H, d), generator=g, device="cuda").bfloat16() for _ in range(2)]
    go = torch.randn((N, H, d), generator=g, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    rope = bsa.rope_axes([bsa.rope_build_table(n, p, device="cuda") for n, p in zip((30, 10, 10), (22, 21, 21))],
                         grid=(30, 10, 10))

    def chain(x, stream):
        with torch.cuda.stream(stream):
            v = x[:, 2].contiguous()
            q, k = bsa.qk_norm_rope_fwd(x[:, 0], x[:, 1], w, w, rope)
            idx, cnt = bsa.blockmean_select(q, k, 6, 1)
            o, lse, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
            return (q, k, idx, cnt, o, *grads, *bsa.qk_norm_rope_bwd(grads[0], grads[1], x[:, 0], x[:, 1], w, w, rope))

    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    ref = []
    for i in range(2):
        ref.append(chain(x[i], streams[i]))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [chain(x[i], streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    assert bsa.get_device_status() == bsa.BSA_OK
    for a, b in zip(ref, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_against_differences_of_the_oracle(bsa):
    """Directional central differences of the float64 forward; the gradient's own
    tolerance is the bound above, summed along the direction."""
    from oracle import attention as oatt
    N, H, d = 300, 1, 64
    go, q, k, v = make(N, H, d, seed=90)
    idx, cnt = random_lists(H, 3, 0.8, 9)
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    mask = block_mask(idx, cnt, N)
    x = [f64(t) for t in (q, k, v)]
    g64 = f64(go)
    rng = np.random.default_rng(3)
    for n in range(3):
        dx = rng.standard_normal(x[n].shape)
        e = 1e-5
        up, dn = list(x), list(x)
        up[n], dn[n] = x[n] + e * dx, x[n] - e * dx
        f = lambda y: float((oatt.attention_dense_masked(*y, d ** -0.5, mask)[0] * g64).sum())  # noqa: E731
        got = float((f64(grads[n]) * dx).sum())
        # errors of the entries are at most a few h of their terms' size and have independent signs
        size = float(np.sqrt((f64(grads[n]) ** 2 * dx ** 2).sum()))
        assert abs((f(up) - f(dn)) / (2 * e) - got) <= 8 * HALF * size + 1e-6


@pytest.mark.parametrize("name", ["wan1.3b_1x_c11", "lists"])
def test_full_size_rows(bsa, name):
    """1x horizon, 12 heads: one head against a float64 computation on the device
    in the tolerance above (summed over whole rows)."""
    N, H, d, T = 32760, 12, 128, 21
    go, q, k, v = make(N, H, d, seed=100)
    if name == "lists":
        idx, cnt = bsa.blockmean_select(q, k, 24, 1)
        ix = bsa.block_index(idx, cnt)
    else:
        frames, counts, _ = bsa.lvsa_build_index(T, 5, 7, 11, 2, device="cuda")
        ix = bsa.lvsa_index(T, frames, counts)
    _, _, grads = both(bsa, go, q, k, v, ix)
    assert bsa.get_device_status() == bsa.BSA_OK
    h, scale = 7, d ** -0.5
    x = [t[:, h].double() for t in (q, k, v, go)]
    want = [torch.zeros(N, d, dtype=torch.float64, device="cuda") for _ in range(3)]
    bound = [torch.zeros_like(w) for w in want]
    frame = torch.arange(N, device="cuda") // (N // T)
    for i in range(-(-N // 128)):
        r = slice(i * 128, min(N, i * 128 + 128))
        if name == "lists":
            on = torch.zeros(N, dtype=torch.bool, device="cuda")
            for j in idx[h, i, :24].tolist():
                on[j * 128:(j + 1) * 128] = True
            on = on.expand(r.stop - r.start, N)
        else:
            allowed = torch.zeros((T, T), dtype=torch.bool, device="cuda")
            for t in range(T):
                allowed[t, frames[t, :int(counts[t])].long()] = True
            on = allowed[frame[r]][:, frame]
        p = torch.where(on, x[0][r] @ x[1].T * scale, -torch.inf).softmax(1)
        dp, o, g = x[3][r] @ x[2].T, p @ x[2], x[3][r]
        D = (g * o).sum(1, keepdim=True)
        eD = HALF * (g.abs() * (o.abs() + p @ x[2].abs())).sum(1, keepdim=True)
        ds = p * (dp - D)
        eds = HALF * ds.abs() + P32 * p * (dp.abs() + D.abs()) + p * eD
        want[0][r], bound[0][r] = scale * ds @ x[1], scale * eds @ x[1].abs()
        want[1] += scale * ds.T @ x[0][r]
        bound[1] += scale * eds.T @ x[0][r].abs()
        want[2] += p.T @ g
        bound[2] += (HALF + P32) * p.T @ g.abs()
    for got, w, b in zip(grads, want, bound):
        err = (got[:, h].double() - w).abs()
        assert bool((err <= b * (1 + HALF) + HALF * w.abs()).all())
        assert float(err.norm() / w.norm()) <= HALF            # rounding errors average out


def test_chain_of_all_operators(bsa):
    """Packed projection -> normed rotation -> chosen blocks -> attention, and the
    gradient back to the projection and the weights, against float64 autograd on
    the same blocks."""
    T, hh, w, H, d = 5, 8, 16, 2, 64
    N, eps = T * hh * w, 1e-5
    g = torch.Generator(device="cuda").manual_seed(110)
    x = torch.randn((N, 3, H, d), generator=g, device="cuda").bfloat16()
    go = torch.randn((N, H, d), generator=g, device="cuda").bfloat16()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    pairs = (12, 10, 10)
    rope = bsa.rope_axes([bsa.rope_build_table(n, p, device="cuda") for n, p in zip((T, hh, w), pairs)], grid=(T, hh, w))
    v = x[:, 2].contiguous()
    q, k = bsa.qk_norm_rope_fwd(x[:, 0], x[:, 1], wq, wk, rope, eps=eps)
    idx, cnt = bsa.blockmean_select(q, k, 3, 0)
    ix = bsa.block_index(idx, cnt)
    o, lse, (dq, dk, dv) = both(bsa, go, q, k, v, ix)
    dx = torch.empty_like(x)
    _, _, dwq, dwk = bsa.qk_norm_rope_bwd(dq, dk, x[:, 0], x[:, 1], wq, wk, rope, eps=eps, dq=dx[:, 0], dk=dx[:, 1])
    dx[:, 2] = dv
    assert bsa.get_device_status() == bsa.BSA_OK
    ridx, rcnt = obm.select(f64(q), f64(k), 3, 0)
    assert np.array_equal(idx.cpu().numpy(), ridx)
    # float64 autograd of the same chain
    X = x.double().requires_grad_()
    W = [t.double().requires_grad_() for t in (wq, wk)]
    pos = torch.stack(torch.meshgrid(*(torch.arange(n) for n in (T, hh, w)), indexing="ij"), -1).reshape(N, 3).cuda()
    ang = torch.cat([pos[:, a:a + 1] * 10000.0 ** (-torch.arange(p, device="cuda", dtype=torch.float64) / p)
                     for a, p in enumerate(pairs)], 1)
    turned = []
    for i in range(2):
        z = X[:, i] * (X[:, i].square().mean(-1, keepdim=True) + eps).rsqrt() * W[i]
        z = torch.view_as_complex(z.reshape(N, H, d // 2, 2)) * torch.polar(torch.ones_like(ang), ang)[:, None]
        turned.append(torch.view_as_real(z).flatten(2))
    mask = torch.from_numpy(block_mask(idx, cnt, N)).cuda()
    s = torch.einsum("nhd,mhd->hnm", *turned) * d ** -0.5
    out = torch.einsum("hnm,mhd->nhd", s.masked_fill(~mask, float("-inf")).softmax(-1), X[:, 2])
    (out * go.double()).sum().backward()
    # q, k, p, ds, dq, dk and the stores are each rounded to bf16 once, errors of
    # independent signs: the 2-norms are off by less than sqrt(7) half steps
    for got, want in [(o, out), (dx, X.grad), (dwq, W[0].grad), (dwk, W[1].grad)]:
        rel = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert rel <= 7 ** 0.5 * HALF, rel


def compare_few(grads, go, q, k, v, scale, mask, what):
    """As `compare`, for rows of at most 32 keys, whose D is not formed from the
    rounded o: eD = 2^-13 sum p |dp| for its p; and the 32-bit sums over d
    channels, each addition off by at most a step of 2^-23 of the magnitudes:
    d 2^-23 <= 2^-16 of <|go|, |v|> in dp, and of its mean in D."""
    go, q, k, v = map(f64, (go, q, k, v))
    assert mask.sum(-1).max() <= 32
    want = obwd.attention_back(go, q, k, v, scale, mask)
    for h in range(q.shape[1]):
        p = obwd.probabilities(q[:, h], k[:, h], scale, mask if mask.ndim == 2 else mask[h])
        g, vh = go[:, h], v[:, h]
        dp, size = g @ vh.T, 2.0 ** -16 * np.abs(g) @ np.abs(vh).T
        D = (p * dp).sum(1, keepdims=True)
        eD = (p * (2 * P32 * np.abs(dp) + size)).sum(1, keepdims=True)
        eds = HALF * np.abs(p * (dp - D)) + p * (P32 * (np.abs(dp) + np.abs(D)) + size + eD)
        bounds = (scale * eds @ np.abs(k[:, h]), scale * eds.T @ np.abs(q[:, h]), (HALF + P32) * p.T @ np.abs(g))
        for name, got, ref, b in zip(("dq", "dk", "dv"), grads, want, bounds):
            err = np.abs(f64(got)[:, h] - ref[:, h])
            bound = b * (1 + HALF) + HALF * np.abs(ref[:, h]) + 1e-30
            assert np.all(err <= bound), f"{what} {name} h={h}: worst err/bound {(err / bound).max()}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 7, 31, 32])
def test_few_keys(bsa, N, d):
    idx, cnt = torch.zeros((2, 1, 1), dtype=torch.int32, device="cuda"), torch.ones((2, 1), dtype=torch.int32, device="cuda")
    for seed in range(4):
        go, q, k, v = make(N, 2, d, seed=200 + 10 * seed)
        _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
        assert bsa.get_device_status() == bsa.BSA_OK
        compare_few(grads, go, q, k, v, d ** -0.5, np.ones((N, N), dtype=bool), f"N={N}")
        if N == 1:                                          # p = 1: nothing that q or k could change
            assert not grads[0].any() and not grads[1].any() and torch.equal(grads[2], go)


@pytest.mark.parametrize("d", [64, 128])
def test_one_key_or_many(bsa, d):
    """Query block 0 sees the single key of the last block, block 1 that and a whole block, the last block itself."""
    N, H = 2 * 128 + 1, 2
    go, q, k, v = make(N, H, d, seed=240)
    idx = torch.tensor([[2, -1, -1], [0, 2, -1], [2, -1, -1]], dtype=torch.int32, device="cuda").expand(H, 3, 3).contiguous()
    cnt = torch.tensor([1, 2, 1], dtype=torch.int32, device="cuda").expand(H, 3).contiguous()
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare(grads, go, q, k, v, d ** -0.5, block_mask(idx, cnt, N), "one key or many")
    dq = grads[0]
    assert not dq[:128].any() and dq[128:256].any() and not dq[256:].any()
    cnt[:, 1] = 0                                           # only rows of one key and of none
    _, _, (dq, dk, dv) = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    assert not dq.any() and not dk.any() and not dv[:256].any() and dv[256].any()


@pytest.mark.parametrize("tail", [3, 32])
def test_few_keys_of_a_short_last_block(bsa, tail):
    """All queries but those of one block see the last block's keys, that block none."""
    N, H, d = 3 * 128 + tail, 2, 64
    go, q, k, v = make(N, H, d, seed=250)
    idx = torch.full((H, 4, 4), -1, dtype=torch.int32, device="cuda")
    cnt = torch.ones((H, 4), dtype=torch.int32, device="cuda")
    idx[:, :, 0] = 3
    cnt[:, 1] = 0
    _, _, grads = both(bsa, go, q, k, v, bsa.block_index(idx, cnt))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare_few(grads, go, q, k, v, d ** -0.5, block_mask(idx, cnt, N), "last block")


@pytest.mark.parametrize("T,P,C,d", [(21, 1, 1, 64), (300, 1, 2, 128), (200, 3, 4, 64), (40, 16, 2, 128), (140, 32, 1, 64)])
def test_few_keys_of_short_frames(bsa, T, P, C, d):
    """The C frames of every row far apart: keys of several partial tiles."""
    H, N = 2, T * P
    go, q, k, v = make(N, H, d, seed=260 + T)
    A = [sorted({(t + i * (T // C + 7)) % T for i in range(C)}) for t in range(T)]
    frames = torch.full((T, T), -1, dtype=torch.int32)
    for t, a in enumerate(A):
        frames[t, :len(a)] = torch.tensor(a, dtype=torch.int32)
    counts = torch.tensor([len(a) for a in A], dtype=torch.int32)
    _, _, grads = both(bsa, go, q, k, v, bsa.lvsa_index(T, frames.cuda(), counts.cuda()))
    assert bsa.get_device_status() == bsa.BSA_OK
    compare_few(grads, go, q, k, v, d ** -0.5, olvsa.dense_token_mask(A, P, N), f"T={T} P={P}")
    if P * C == 1:
        assert not grads[0].any() and not grads[1].any()


def test_few_keys_of_frames_within_blocks(bsa):
    """Frames of 40 tokens, own frame and own block only: rows with 1 to 40 keys,
    the ones in question where frames cross a block's border."""
    T, P, H, d = 13, 40, 2, 128
    N = T * P
    go, q, k, v = make(N, H, d, seed=270)
    frames = torch.full((T, T), -1, dtype=torch.int32)
    frames[:, 0] = torch.arange(T, dtype=torch.int32)
    nB = -(-N // 128)
    idx = torch.full((H, nB, nB), -1, dtype=torch.int32, device="cuda")
    idx[:, :, 0] = torch.arange(nB, device="cuda")
    cnt = torch.ones((H, nB), dtype=torch.int32, device="cuda")
    ix = bsa.lvsa_block_index(T, frames.cuda(), torch.ones(T, dtype=torch.int32, device="cuda"), idx, cnt)
    _, _, grads = both(bsa, go, q, k, v, ix)
    assert bsa.get_device_status() == bsa.BSA_OK
    mask = olvsa.dense_token_mask([[t] for t in range(T)], P, N)[None] & block_mask(idx, cnt, N)
    compare(grads, go, q, k, v, d ** -0.5, mask, "all rows")
    few = np.flatnonzero(mask[0].sum(1) <= 32)              # whole groups: a frame's part in a block sees itself
    assert 0 < len(few) < N
    at = torch.from_numpy(few).cuda()
    compare_few([x[at] for x in grads], go[at], q[at], k[at], v[at], d ** -0.5, mask[:, few][:, :, few], "few")


def test_lists_that_split_the_keys(bsa):
    """With o and lse of all keys, the gradients of lists that split the keys add
    up, also where one of the lists has few keys: its D is the whole row's."""
    N, H, d = 128 + 4, 2, 64
    go, q, k, v = make(N, H, d, seed=280)
    full = torch.tensor([0, 1], dtype=torch.int32, device="cuda").expand(H, 2, 2).contiguous()
    two, one = (torch.full((H, 2), n, dtype=torch.int32, device="cuda") for n in (2, 1))
    o, lse = bsa.blocksparse_attn_fwd(q, k, v, bsa.block_index(full, two))
    parts = []
    for b in range(2):
        idx = torch.full((H, 2, 2), -1, dtype=torch.int32, device="cuda")
        idx[:, :, 0] = b
        parts.append(bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(idx, one)))
    assert bsa.get_device_status() == bsa.BSA_OK
    for i in (1, 2):                                        # every key is in one of the lists
        assert bool((parts[0][i][128:] == 0).all()) and bool((parts[1][i][:128] == 0).all())
    # dq is rounded twice: within half a step of either part; kept in 32 bits, its
    # sum is compared in `compare` as one rounding of |a + b|, so the rest is added there
    dk, dv = (parts[0][i] + parts[1][i] for i in (1, 2))
    dq = obwd.attention_back(*map(f64, (go, q, k, v)), d ** -0.5, np.ones((N, N), dtype=bool))[0]
    compare((torch.from_numpy(dq), dk, dv), go, q, k, v, d ** -0.5, np.ones((N, N), dtype=bool), "split")
    a, b = f64(parts[0][0]), f64(parts[1][0])
    whole = f64(bsa.blocksparse_attn_bwd(go, q, k, v, o, lse, bsa.block_index(full, two))[0])
    assert np.linalg.norm(a + b - whole) <= HALF * (np.linalg.norm(a) + np.linalg.norm(b) + np.linalg.norm(whole))

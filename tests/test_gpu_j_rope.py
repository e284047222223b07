"""GPU: rotation of q and k by (time, height, width), the per-head norm with the
rotation in the same pass, and its gradient, against the float64 oracle.

Tolerances, by counting roundings (u = 2^-24, float32's half step):
  * one store rounding: half a step of the output type, eps/2 * |y| (and
    tiny * eps for results below the type's normal range);
  * rotation: two table values and three operations: 4u (|a| + |b|);
  * norm: the sum of squares takes 8 + 4 additions and a product, its relative
    error is halved by the root, rsqrt is off by 2 ulps, then two products:
    under 16u of the normed value, which reaches both members of a pair:
    together under 24u (|z_a| + |z_b|);
  * gradient: g is off by 4u (|g_a| + |g_b|), the row's dot product by
    20u mean|g w xh|, r by 10u, and four operations follow: under 64u of
    r (|gw_a| + |gw_b| + |xh| mean|g w xh|);
  * weight gradient: a lane adds its token's heads (here every group has one
    token), then come at most 32 groups, 296 / 8 blocks of a slice and 16
    slices, and each term is off by 20u: under (heads + 150) u sum|g xh|.
"""
import numpy as np
import pytest
import torch

from oracle import rope as orope

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_lvsa_b200 import binding
    assert torch.cuda.is_available()
    return binding


def pairs_of(d):
    n = d // 6
    return d // 2 - 2 * n, n, n


def f64(t):
    return t.detach().cpu().double().numpy()


def tables(bsa, lens, pairs, **kw):
    return [bsa.rope_build_table(n, p, device="cuda", **kw) if p else torch.empty((n, 0, 2), device="cuda")
            for n, p in zip(lens, pairs)]


def pair_sum(x, pairing):
    """|a| + |b| of every channel's pair."""
    z = orope._complex(np.abs(x), pairing)
    return orope._real((z.real + z.imag) * (1 + 1j), pairing)


def close(got, want, slack, dtype, what):
    fi = torch.finfo(dtype)
    err = np.abs(f64(got) - want)
    bound = fi.eps / 2 * (np.abs(want) + slack) + slack + fi.tiny * fi.eps
    assert np.all(err <= bound), f"{what}: worst err/bound {(err / bound).max()}"


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def make(shape, dtype, layout, seed, scale=1.0):
    """[N, H, d] in one of the layouts a projection gives."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, H, d = shape
    if layout == "packed":
        return (randn(g, N, 3, H, d) * scale).to(dtype)[:, 1]
    if layout == "heads first":
        return (randn(g, H, N, d) * scale).to(dtype).transpose(0, 1)
    if layout == "padded":
        return (randn(g, N, H, d + 8) * scale).to(dtype)[:, :, :d]
    return (randn(g, *shape) * scale).to(dtype)


def setup(bsa, grid, tail, d, listed, start=0.0, first=(0, 0, 0), pairs=None, pairing="adjacent", seed=0):
    """(bsa_rope, oracle angles [N, d/2])"""
    pairs = pairs_of(d) if pairs is None else pairs
    lens = [f + n + 1 for f, n in zip(first, grid)]
    tabs = tables(bsa, lens, pairs, start=start)
    N = int(np.prod(grid)) + tail
    pos = orope.grid_positions(grid, first, N)
    if listed:
        pos = pos[np.random.default_rng(seed).permutation(N)]
        r = bsa.rope_axes(tabs, pos=torch.from_numpy(pos).to("cuda", torch.int32), pairing=pairing)
    else:
        r = bsa.rope_axes(tabs, grid=grid, first=first, pairing=pairing)
    ang = orope.token_angles([orope.axis_angles(n, p, start=start) for n, p in zip(lens, pairs)], pos, d)
    return r, ang


def test_table_against_double(bsa):
    for n, p, theta, start, step in [(1, 1, 10000.0, 0.0, 1.0), (126, 22, 10000.0, 0.0, 1.0),
                                     (33, 7, 256.0, 1e6, 0.25), (5, 64, 5e5, -3.0, -2.0)]:
        t = f64(bsa.rope_build_table(n, p, theta, start, step, device="cuda"))
        a = orope.axis_angles(n, p, theta, start, step)
        # angles up to 1e6 keep ~1e-9 in 64 bits, then one rounding to float32
        assert np.abs(t[..., 0] - np.cos(a)).max() <= U + 1e-8
        assert np.abs(t[..., 1] - np.sin(a)).max() <= U + 1e-8


CASES = [
    # grid, tail, H, d, dtype, pairing, layout, listed
    ((1, 1, 1), 0, 1, 64, "bf16", "adjacent", "whole", False),
    ((1, 1, 1), 3, 1, 128, "fp32", "split", "whole", False),
    ((8, 8, 8), 0, 2, 64, "bf16", "adjacent", "whole", False),
    ((3, 5, 7), 0, 12, 128, "bf16", "adjacent", "packed", False),
    ((3, 5, 7), 11, 13, 128, "fp16", "split", "padded", True),
    ((2, 30, 52), 0, 40, 128, "bf16", "split", "heads first", False),
    ((4, 9, 3), 5, 9, 64, "fp32", "adjacent", "packed", True),
    ((4, 9, 3), 0, 17, 64, "fp16", "adjacent", "heads first", False),
    ((1, 17, 1), 0, 8, 128, "fp32", "split", "whole", True),
    ((1, 1, 1), 0, 100, 128, "bf16", "adjacent", "whole", False),     # one token: its heads in several blocks
    ((2, 1, 1), 1, 33, 64, "fp32", "adjacent", "heads first", True),
]


@pytest.mark.parametrize("grid,tail,H,d,dtype,pairing,layout,listed", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_apply(bsa, grid, tail, H, d, dtype, pairing, layout, listed, inverse):
    r, ang = setup(bsa, grid, tail, d, listed, start=17.0, first=(2, 0, 1), pairing=pairing)
    x = make((ang.shape[0], H, d), TYPES[dtype], layout, 1)
    keep = x.clone()
    y = bsa.rope_apply(x, r, inverse=inverse)
    assert bsa.get_device_status() == bsa.BSA_OK
    assert torch.equal(x, keep)
    close(y, orope.turn(f64(x), -ang if inverse else ang, pairing), 4 * U * pair_sum(f64(x), pairing), x.dtype, "rope")


@pytest.mark.parametrize("grid,tail,H,d,dtype,pairing,layout,listed", CASES)
def test_norm_rope_and_gradient(bsa, grid, tail, H, d, dtype, pairing, layout, listed):
    eps = 1e-5
    dt = TYPES[dtype]
    r, ang = setup(bsa, grid, tail, d, listed, pairing=pairing)
    N, Hk = ang.shape[0], max(1, H // 2)
    q, k = make((N, H, d), dt, layout, 2, 3.0), make((N, Hk, d), dt, layout, 3, 0.5)
    g = torch.Generator(device="cuda").manual_seed(4)
    wt = torch.float32 if H % 2 else dt
    wq, wk = (1 + 0.3 * randn(g, d)).to(wt), (1 + 0.3 * randn(g, d)).to(wt)
    qo, ko = bsa.qk_norm_rope_fwd(q, k, wq, wk, r, eps=eps)
    gq, gk = make(q.shape, dt, "whole", 5), make(k.shape, dt, layout, 6)
    dq, dk, dwq, dwk = bsa.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, r, eps=eps)
    assert bsa.get_device_status() == bsa.BSA_OK
    for x, w, y, gy, dx, dw in [(q, wq, qo, gq, dq, dwq), (k, wk, ko, gk, dk, dwk)]:
        x64, w64, g64 = f64(x), f64(w), f64(gy)
        rr = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
        close(y, orope.norm_turn(x64, w64, ang, pairing, eps), 24 * U * pair_sum(x64 * rr * w64, pairing), dt, "fwd")
        rdx, rdw = orope.norm_turn_back(g64, x64, w64, ang, pairing, eps)
        gb = pair_sum(orope.turn(g64, -ang, pairing), pairing) * np.abs(w64)
        xh = np.abs(x64 * rr)
        close(dx, rdx, 64 * U * rr * (gb + xh * (gb * xh).mean(-1, keepdims=True)), dt, "dx")
        bound = (x.shape[1] + 150) * U * (pair_sum(orope.turn(g64, -ang, pairing), pairing) * xh).sum((0, 1))
        assert np.all(np.abs(f64(dw) - rdw) <= bound)


def test_norm_alone_and_queries_alone(bsa):
    x = make((37, 3, 64), torch.bfloat16, "whole", 7)
    y, none = bsa.qk_norm_rope_fwd(x, None, eps=1e-6)
    assert none is None
    zero = np.zeros((37, 32))
    close(y, orope.norm_turn(f64(x), 1.0, zero, "adjacent", 1e-6), 24 * U * np.abs(f64(y)), x.dtype, "norm")
    g = make((37, 3, 64), torch.bfloat16, "whole", 8)
    dx, dk, dw, dwk = bsa.qk_norm_rope_bwd(g, None, x, None, eps=1e-6)
    assert dk is None and dw is None and dwk is None
    ref, _ = orope.norm_turn_back(f64(g), f64(x), np.ones(64), zero, "adjacent", 1e-6)
    x64 = f64(x)
    rr = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-6)
    gb, xh = np.abs(f64(g)) * 2, np.abs(x64 * rr)
    close(dx, ref, 64 * U * rr * (gb + xh * (gb * xh).mean(-1, keepdims=True)), x.dtype, "dx")


def test_gradient_against_differences(bsa):
    """fp32 differences of the forward kernel itself: step e in one direction,
    relative error e^2 (third derivative) + rounding 2^-24 |f| / e."""
    r, ang = setup(bsa, (2, 3, 2), 0, 64, False, pairing="split")
    g = torch.Generator(device="cuda").manual_seed(9)
    x, v, gy = (randn(g, 12, 2, 64) for _ in range(3))
    w, vw = 1 + 0.2 * randn(g, 64), randn(g, 64)
    dx, _, dw, _ = bsa.qk_norm_rope_bwd(gy, None, x, None, w, None, r, eps=1e-3)
    e = 2.0 ** -8

    def f(x, w):
        return float((bsa.qk_norm_rope_fwd(x, None, w, None, r, eps=1e-3)[0].double() * gy.double()).sum())

    size = float((gy.double().abs() * 3).sum())
    got = (f(x + e * v, w) - f(x - e * v, w)) / (2 * e)
    assert abs(got - float((dx.double() * v.double()).sum())) <= size * (e * e + 8 * U / e)
    got = (f(x, w + e * vw) - f(x, w - e * vw)) / (2 * e)
    assert abs(got - float((dw.double() * vw.double()).sum())) <= size * (8 * U / e)


def test_in_place_and_unturned_parts(bsa):
    d = 128
    r, ang = setup(bsa, (2, 3, 4), 2, d, False, pairs=(5, 0, 9))          # 50 pairs stay as they are
    x = make((26, 4, d), torch.bfloat16, "packed", 10)
    x[25, 1, :] = float("inf")                                            # behind the grid: a copy
    y = bsa.rope_apply(x, r)
    assert torch.equal(y[24:], x[24:]) and torch.equal(y[:, :, 28:], x[:, :, 28:])
    z = x.clone()
    xs = x.contiguous()
    assert bsa.rope_apply(xs, r, out=xs).data_ptr() == xs.data_ptr()
    assert torch.equal(xs, y) and torch.equal(x, z)
    xs = make((26, 4, d), torch.bfloat16, "packed", 10)
    bsa.rope_apply(xs, r, out=xs)                                         # a slice of a packed tensor, in place
    assert torch.equal(xs[:24], y[:24])
    q, k = make((26, 4, d), torch.bfloat16, "whole", 11), make((26, 2, d), torch.bfloat16, "whole", 12)
    gq, gk = make(q.shape, torch.bfloat16, "whole", 13), make(k.shape, torch.bfloat16, "whole", 14)
    w = torch.ones(d, device="cuda")
    ref = bsa.qk_norm_rope_fwd(q, k, w, w, r)
    refb = bsa.qk_norm_rope_bwd(gq, gk, q, k, w, w, r)
    for out in ("x", "g"):
        q2, k2, gq2, gk2 = q.clone(), k.clone(), gq.clone(), gk.clone()
        got = bsa.qk_norm_rope_bwd(gq2, gk2, q2, k2, w, w, r, dq=q2 if out == "x" else gq2, dk=k2 if out == "x" else gk2)
        assert all(torch.equal(a, b) for a, b in zip(got, refb))
    got = bsa.qk_norm_rope_fwd(q, k, w, w, r, qo=q, ko=k)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]) and got[0] is q


def test_rows_behind_and_between_are_left(bsa):
    """A strided output: what lies between its rows keeps its values."""
    r, ang = setup(bsa, (2, 2, 2), 0, 64, False)
    x = make((8, 3, 64), torch.float16, "whole", 15)
    room = torch.full((10, 5, 72), 7.0, dtype=torch.float16, device="cuda")
    bsa.rope_apply(x, r, out=room[1:9, 1:4, :64])
    assert torch.equal(room[1:9, 1:4, :64], bsa.rope_apply(x, r))
    room[1:9, 1:4, :64] = 7.0
    assert bool((room == 7.0).all())


def test_expanded_input_and_special_rows(bsa):
    r, ang = setup(bsa, (3, 1, 1), 0, 64, False)
    one = make((1, 1, 64), torch.float32, "whole", 16)
    x = one.expand(3, 4, 64)
    assert torch.equal(bsa.rope_apply(x, r), bsa.rope_apply(x.contiguous(), r))
    x = make((3, 4, 64), torch.float32, "whole", 17)
    x[0, 0] = 0.0                                                         # zero row: stays zero, finite gradient
    x[1, 1, 5] = float("nan")                                             # a bad row stays alone
    y, _ = bsa.qk_norm_rope_fwd(x, None, None, None, r)
    assert bool((y[0, 0] == 0).all()) and bool(y[1, 1].isnan().all())
    ok = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    ok[1, 1] = False
    assert bool(y[ok].isfinite().all())
    dx = bsa.qk_norm_rope_bwd(torch.ones_like(x), None, x, None, None, None, r)[0]
    assert bool(dx[ok].isfinite().all())


def test_position_past_the_table_is_reported(bsa):
    tabs = tables(bsa, (4, 4, 4), (12, 10, 10))
    pos = torch.zeros((6, 3), dtype=torch.int32, device="cuda")
    pos[2, 1] = 4
    pos[3, 0] = -5
    r = bsa.rope_axes(tabs, pos=pos)
    x = make((6, 2, 64), torch.bfloat16, "whole", 18)
    y = bsa.rope_apply(x, r)
    assert bsa.get_device_status() == bsa.BSA_ERR_INDEX_RANGE
    assert torch.equal(y, x)                                              # position 0 turns by nothing
    assert bsa.get_device_status() == bsa.BSA_OK


def test_refusals_on_the_device(bsa):
    r, ang = setup(bsa, (2, 2, 2), 0, 64, True)
    x = make((8, 3, 64), torch.bfloat16, "whole", 19)
    with pytest.raises(ValueError):
        bsa.rope_apply(x[:7], r)                                          # pos holds 8 tokens
    with pytest.raises(ValueError):
        bsa.rope_apply(x.transpose(1, 2), r)                              # channel stride
    with pytest.raises(bsa.BsaError):
        bsa.rope_apply(x[:, :, :32].contiguous(), r)                      # d = 32
    with pytest.raises(ValueError):
        bsa.rope_apply(x, r, out=torch.empty_like(x, dtype=torch.float16))
    with pytest.raises(ValueError):
        bsa.qk_norm_rope_fwd(x, x, torch.ones(64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        bsa.qk_norm_rope_fwd(x, x, torch.ones(63, device="cuda"))
    flat = torch.zeros(8 * 3 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bsa.BsaError):                                     # 8 bytes off a 16-byte boundary
        bsa.rope_apply(flat[4:].view(8, 3, 64), r)
    with pytest.raises(bsa.BsaError):                                     # an output whose rows overlap
        bsa.rope_apply(x, r, out=flat[:64].as_strided((8, 3, 64), (0, 0, 1)))


def test_other_stream_and_graph(bsa):
    r, ang = setup(bsa, (5, 6, 7), 0, 128, False)
    q, k = make((210, 4, 128), torch.bfloat16, "whole", 20), make((210, 4, 128), torch.bfloat16, "whole", 21)
    w = torch.ones(128, device="cuda")
    gq, gk = make(q.shape, q.dtype, "whole", 22), make(q.shape, q.dtype, "whole", 23)
    ref = bsa.qk_norm_rope_bwd(gq, gk, q, k, w, w, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = bsa.qk_norm_rope_bwd(gq, gk, q, k, w, w, r, stream=s)
    raw = bsa.qk_norm_rope_bwd(gq, gk, q, k, w, w, r, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(ref, got, raw))
    # two captured graphs with workspaces of their own, replayed one after the other
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(bsa.qk_norm_rope_bwd(gq, gk, q, k, w, w, r) + bsa.qk_norm_rope_fwd(q, k, w, w, r))
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    fwd = bsa.qk_norm_rope_fwd(q, k, w, w, r)
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref + fwd))


def test_weight_gradient_repeats_bit_for_bit(bsa):
    r, ang = setup(bsa, (21, 10, 26), 0, 128, False)
    q = make((5460, 12, 128), torch.bfloat16, "whole", 24)
    g = make(q.shape, q.dtype, "whole", 25)
    w = torch.ones(128, device="cuda")
    a = bsa.qk_norm_rope_bwd(g, None, q, None, w, None, r)
    for _ in range(3):
        b = bsa.qk_norm_rope_bwd(g, None, q, None, w, None, r)
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


def test_offsets_past_32_bits(bsa):
    """Rows of a tensor whose last element lies past 2^31 elements."""
    d, ts = 64, 1 << 20
    N = 2100                                                              # 2100 * 2^20 > 2^31 elements
    room = torch.empty(((N - 1) * ts + 2 * d,), dtype=torch.bfloat16, device="cuda")
    x = room.as_strided((N, 2, d), (ts, d, 1))
    small = make((N, 2, d), torch.bfloat16, "whole", 26)
    x.copy_(small)
    r, ang = setup(bsa, (N, 1, 1), 0, d, False)
    assert torch.equal(bsa.rope_apply(x, r), bsa.rope_apply(small, r))
    bsa.rope_apply(small, r, out=x)
    assert torch.equal(x, bsa.rope_apply(small, r))

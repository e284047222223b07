"""Measured cases of the operators around the sparse attention: the rotation of
queries and keys by (time, height, width), their per-head norm with the rotation
in the same pass, the choice of key blocks by block means, the attention over the
chosen blocks, and the attention's gradient.

`run` computes a case either in plain torch operations (`own` false) or with the
calls a user makes of the framework (`own` true), on the same state."""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
THETA = 10000.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}

# the largest q (tokens x heads x channels) and the largest number of gathered
# key blocks (heads x query blocks x kept) among the listed cases: draws stay below
MOST_X = 196560 * 12 * 128
MOST_TILES = 12 * 256 * 32


def _rope(name, op, grid, H, d, dtype, pairing="adjacent", tail=0, start=0.0, listed_pos=False, packed=False):
    t, h, w = grid
    return {"name": name, "op": op, "t": t, "h": h, "w": w, "tail": tail, "H": H, "d": d, "dtype": dtype,
            "pairing": pairing, "start": start, "listed_pos": listed_pos, "packed": packed}


def _attn(name, op, N, H, d, keep, local=0, T=0, C=0):
    return {"name": name, "op": op, "N": N, "H": H, "d": d, "keep": keep, "local": local, "T": T, "C": C}


def listed():
    return [
        # the smallest call: the tiny workload's 8 frames of 8 x 8, where launch latency is all
        _rope("rope tiny", "rope", (8, 8, 8), 2, 64, "bf16"),
        # a whole 6x-horizon video of 126 frames of 30 x 52, one tensor
        _rope("rope 6x horizon", "rope", (126, 30, 52), 12, 128, "bf16"),
        # the rotation's gradient in fp32, halves paired, positions from a list, an odd number of tokens
        _rope("rope back ragged fp32", "rope_back", (23, 15, 29), 5, 128, "fp32", "split", tail=2, listed_pos=True),
        # one frame of 30 x 52 out of a packed projection: frame-by-frame use
        _rope("norm rope one frame", "norm_rope", (1, 30, 52), 12, 128, "bf16", packed=True),
        # q and k of the 6x-horizon video before its attention: the largest amount of data
        _rope("norm rope 6x horizon", "norm_rope", (126, 30, 52), 12, 128, "bf16"),
        # training at 1x horizon with 40 heads
        _rope("norm rope back 1x", "norm_rope_back", (21, 30, 52), 40, 128, "bf16"),
        # training on a small ragged fp16 batch out of a packed projection, text tokens after the grid
        _rope("norm rope back ragged", "norm_rope_back", (7, 11, 16), 3, 64, "fp16", "split", tail=5, packed=True),
        # the smallest choice of blocks: 4 blocks, 2 kept
        _attn("select tiny", "select", 512, 2, 64, 2),
        # the choice of one denoising step of the 6x-horizon video: a budget of 21 of 126 frames
        _attn("select 6x horizon", "select", 196560, 12, 128, 256, 1),
        # choice and attention of one step at 1x horizon, an eighth of the blocks kept
        _attn("select and attend 1x", "sparse", 32760, 12, 128, 32, 1),
        # gradient of the attention inside frame sets: 21 frames of 157 tokens, partial tiles everywhere
        _attn("attention back frames", "attn_back", 21 * 157, 4, 64, 0, 0, 21, 7),
        # gradient of the attention over chosen blocks at 1x horizon
        _attn("attention back 1x", "attn_back", 32760, 12, 128, 32, 1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_back", "norm_rope", "norm_rope_back", "select", "sparse", "attn_back", "attn_back"])
    d = rng.choice([64, 128])
    H = _log(rng, 1, 40)
    if "rope" in op:
        t, h, w = _log(rng, 1, 130), _log(rng, 1, 46), _log(rng, 1, 81)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = MOST_X * 2 // (SIZE[dtype] * (3 if op == "norm_rope_back" else 2))
        while t * h * w * H * d > most:
            t = max(1, t // 2)
        c = _rope("", op, (t, h, w), H, d, dtype, rng.choice(["adjacent", "split"]), rng.choice([0, 0, 1, 77]),
                  rng.choice([0.0, 0.0, 25.0, 60000.0]), rng.random() < 0.3, rng.random() < 0.5)
    elif op == "attn_back" and rng.random() < 0.5:
        T = rng.randint(1, 24)
        P = _log(rng, 1, 160)
        H = rng.randint(1, 4)
        c = _attn("", op, T * P, H, d, 0, 0, T, rng.randint(1, T))
    else:
        N = _log(rng, 1601, 196560) if op == "select" else _log(rng, 1, 32760)
        nB = -(-N // BLOCK)
        while N * H * d > MOST_X or H * nB > MOST_TILES:
            H = max(1, H // 2)
        local = rng.choice([0, 0, 1, 2])
        if op == "select":  # some blocks chosen by their scores, some left out
            keep = _log(rng, 2 * local + 2, max(2 * local + 2, nB // 2))
        else:
            keep = max(1, min(_log(rng, 1, nB), MOST_TILES // (H * nB)))
            if H * nB * max(keep, 2 * local + 1) > MOST_TILES:
                local = 0
        c = _attn("", op, N, H, d, keep, local)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs --
def _pairs(d):
    """Pairs of channels rotated by time, height and width: a third each, time takes the rest."""
    n = d // 6
    return d // 2 - 2 * n, n, n


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _table(rows, pairs, start):
    """cos and sin of every position of one axis, float32 [rows, pairs, 2], from angles in 64 bits."""
    pos = start + torch.arange(rows, device="cuda", dtype=torch.float64)
    freq = THETA ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
    ang = pos[:, None] * freq
    return torch.stack([ang.cos(), ang.sin()], -1).float()


def _positions(case, seed):
    """Token positions int64 [N, 3] (-1: behind the grid, not rotated), shuffled where the case lists them."""
    t, h, w = case["t"], case["h"], case["w"]
    n = t * h * w
    i = torch.arange(n, device="cuda")
    pos = torch.stack([i // (h * w), (i // w) % h, i % w], 1)
    if case["listed_pos"]:
        pos = pos[torch.randperm(n, generator=_gen(seed + 7), device="cuda")]
    return torch.cat([pos, pos.new_full((case["tail"], 3), -1)])


def _heads(case, g, count):
    """`count` tensors [N, H, d]: of their own, or slices of one packed projection [N, 3, H, d]."""
    N, H, d = case["t"] * case["h"] * case["w"] + case["tail"], case["H"], case["d"]
    dt = TYPES[case["dtype"]]
    gain = torch.exp(0.3 * _randn(g, d))
    if case["packed"]:
        x = (_randn(g, N, 3, H, d) * gain).to(dt)
        return [x[:, i] for i in range(count)]
    return [(_randn(g, N, H, d) * gain).to(dt) for _ in range(count)]


def _qkv(N, H, d, g, count):
    """Tokens of a video: neighbouring tokens share a part, so that blocks differ from one another."""
    out = []
    for i in range(count):
        x = _randn(g, N, H, d)
        if i < 2:
            shared = _randn(g, -(-N // 61), H, d)
            x += 0.5 * shared.repeat_interleave(61, 0)[:N]
        out.append(x.to(torch.bfloat16))
    return out


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if "rope" in case["op"]:
        s["pairs"] = _pairs(case["d"])
        s["tables"] = [_table(case[a], n, case["start"]) for a, n in zip("thw", s["pairs"])]
        s["pos"] = _positions(case, seed)
        s["pos32"] = s["pos"].to(torch.int32).contiguous()
        if case["op"] in ("rope", "rope_back"):
            s["x"], = _heads(case, g, 1)
        else:
            s["q"], s["k"] = _heads(case, g, 2)
            s["wq"], s["wk"] = (1 + 0.2 * _randn(g, case["d"]) for _ in range(2))
            if case["op"] == "norm_rope_back":
                s["gq"], s["gk"] = (_randn(g, *s["q"].shape).to(s["q"].dtype) for _ in range(2))
        return s
    N, H, d = case["N"], case["H"], case["d"]
    if case["op"] == "select":
        s["q"], s["k"] = _qkv(N, H, d, g, 2)
    else:
        s["q"], s["k"], s["v"] = _qkv(N, H, d, g, 3)
    if case["op"] == "attn_back":
        s["go"] = _randn(g, N, H, d).to(torch.bfloat16)
        if case["T"]:
            s["frames"], s["counts"] = _frame_sets(case["T"], case["C"])
            o, lse = _dense(s["q"], s["k"], s["v"], _frame_mask(s, N), d ** -0.5)
        else:
            s["idx"], s["cnt"] = _select(s["q"], s["k"], case["keep"], case["local"])
            o, lse = _gathered(s["q"], s["k"], s["v"], s["idx"], _width(case), d ** -0.5)
        s["o"], s["lse"] = o.to(torch.bfloat16), lse.contiguous()
    return s


def _frame_sets(T, C):
    """The C frames nearest to each frame (the earlier one first), ascending: int32 [T, T] padded with -1, and counts."""
    f = torch.arange(T, device="cuda")
    far = (f[None, :] - f[:, None]).abs() * 2 + (f[None, :] > f[:, None])
    near = far.argsort(1)[:, :C].sort(1).values
    frames = torch.full((T, T), -1, device="cuda", dtype=torch.int32)
    frames[:, :C] = near.to(torch.int32)
    return frames, torch.full((T,), C, device="cuda", dtype=torch.int32)


# ------------------------------------------------------------- plain forms --
def _channels(d, pairing):
    """Channel of the first and of the second member of every pair."""
    j = torch.arange(d // 2, device="cuda")
    return (2 * j, 2 * j + 1) if pairing == "adjacent" else (j, j + d // 2)


def _cos_sin(s):
    """cos and sin of every token and pair, float32 [N, 1, d/2]; tokens behind the grid are not rotated."""
    pos = s["pos"]
    cs = torch.cat([tab[pos[:, a].clamp(min=0)] for a, tab in enumerate(s["tables"])], 1)
    on = (pos[:, :1] >= 0)[:, None]
    return torch.where(on, cs[:, None, :, 0], 1.0), torch.where(on, cs[:, None, :, 1], 0.0)


def _rotate(x, cos, sin, pairing):
    a, b = _channels(x.shape[-1], pairing)
    y = torch.empty_like(x)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _norm_rope(x, w, cos, sin, pairing):
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return _rotate(x * r * w, cos, sin, pairing)


def _norm_rope_back(g, x, w, cos, sin, pairing):
    g = _rotate(g.float(), cos, -sin, pairing)
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = x * r
    dw = (g * xh).sum((0, 1))
    g = g * w
    return r * (g - xh * (g * xh).mean(-1, keepdim=True)), dw


def _blocks(x, dtype):
    """[N, H, d] -> [H, blocks, 128, d], zeros behind the last token."""
    N, H, d = x.shape
    nB = -(-N // BLOCK)
    y = torch.zeros((nB * BLOCK, H, d), dtype=dtype, device=x.device)
    y[:N] = x
    return y.view(nB, BLOCK, H, d).permute(2, 0, 1, 3)


def _select(q, k, keep, local):
    """Key blocks of the largest mean score per query block (own neighbourhood first); scores in 64 bits: a border decides."""
    N, H, _ = q.shape
    nB = -(-N // BLOCK)
    b = torch.arange(nB, device=q.device)
    rows = (N - b * BLOCK).clamp(max=BLOCK).double()[:, None]
    mq, mk = (_blocks(x, torch.float64).sum(2) / rows for x in (q, k))
    score = mq @ mk.transpose(1, 2)
    near = (b[:, None] - b[None, :]).abs() <= local
    score.masked_fill_(near, math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices
    cnt = near.sum(1).clamp(min=min(keep, nB))
    kept = torch.where(b[None, None, :] < cnt[None, :, None], order, nB).sort(dim=2).values
    return torch.where(kept < nB, kept, -1).to(torch.int32), cnt.to(torch.int32).expand(H, nB).contiguous()


def _width(case):
    """The longest list of kept blocks."""
    return min(-(-case["N"] // BLOCK), max(case["keep"], 2 * case["local"] + 1))


def _gather(xb, idx):
    H, nB, K = idx.shape
    at = torch.arange(H, device=idx.device)[:, None, None]
    return xb[at, idx.clamp(min=0).long()].reshape(H, nB, K * BLOCK, xb.shape[-1])


def _scores(qb, kg, idx, N, scale):
    """Scores of every query block against its gathered keys, -inf where there is no key."""
    pos = idx.long()[..., None] * BLOCK + torch.arange(BLOCK, device=idx.device)
    on = ((idx[..., None] >= 0) & (pos < N)).flatten(2)[:, :, None]
    return (qb @ kg.transpose(2, 3)).mul_(scale).masked_fill_(~on, -math.inf)


def _softmax(sc):
    m = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (sc - m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = (m + l.log()).squeeze(-1)
    return torch.where(l > 0, p / l, 0.0), lse


def _rows(xb, N):
    """[H, blocks, 128, d] -> [N, H, d]."""
    H, nB, _, d = xb.shape
    return xb.permute(1, 2, 0, 3).reshape(nB * BLOCK, H, d)[:N]


def _gathered(q, k, v, idx, width, scale):
    N, H, d = q.shape
    idx = idx[:, :, :width]
    sc = _scores(_blocks(q, torch.float32), _gather(_blocks(k, torch.float32), idx), idx, N, scale)
    p, lse = _softmax(sc)
    return _rows(p @ _gather(_blocks(v, torch.float32), idx), N), lse.flatten(1)[:, :N]


def _gathered_back(s, scale):
    q, k, v = s["q"], s["k"], s["v"]
    N, H, d = q.shape
    idx = s["idx"][:, :, :_width(s["case"])]
    qb, gb = _blocks(q, torch.float32), _blocks(s["go"], torch.float32)
    kg = _gather(_blocks(k, torch.float32), idx)
    p, _ = _softmax(_scores(qb, kg, idx, N, scale))
    vg = _gather(_blocks(v, torch.float32), idx)
    dp = gb @ vg.transpose(2, 3)
    nB, K = idx.shape[1:]
    at = (torch.arange(H, device=q.device)[:, None, None] * nB + idx.clamp(min=0)).flatten()

    def back(x):
        to = torch.zeros((H * nB, BLOCK * d), device=q.device)
        return _rows(to.index_add_(0, at, x.reshape(H * nB * K, BLOCK * d)).view(H, nB, BLOCK, d), N)

    dv = back(p.transpose(2, 3) @ gb)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    return _rows(ds @ kg, N), back(ds.transpose(2, 3) @ qb), dv


def _frame_mask(s, N):
    """bool [N, N]: the key's frame is in the query's frame set."""
    T = s["frames"].shape[0]
    on = torch.zeros((T, T + 1), dtype=torch.bool, device="cuda")
    on.scatter_(1, torch.where(s["frames"] < 0, T, s["frames"]).long(), True)
    f = torch.arange(N, device="cuda") // (N // T)
    return on[f][:, f]


def _dense(q, k, v, mask, scale):
    q, k, v = (x.float().transpose(0, 1) for x in (q, k, v))
    p, lse = _softmax((q @ k.transpose(1, 2) * scale).masked_fill_(~mask, -math.inf))
    return (p @ v).transpose(0, 1), lse


def _dense_back(s, mask, scale):
    q, k, v, go = (s[n].float().transpose(0, 1) for n in ("q", "k", "v", "go"))
    p, _ = _softmax((q @ k.transpose(1, 2) * scale).masked_fill_(~mask, -math.inf))
    dp = go @ v.transpose(1, 2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
    return tuple(x.transpose(0, 1) for x in (ds @ k, ds.transpose(1, 2) @ q, p.transpose(1, 2) @ go))


def _plain(s):
    c = s["case"]
    if "rope" in c["op"]:
        cos, sin = _cos_sin(s)
        if c["op"] in ("rope", "rope_back"):
            return _rotate(s["x"].float(), cos, sin if c["op"] == "rope" else -sin, c["pairing"]).to(s["x"].dtype)
        if c["op"] == "norm_rope":
            return tuple(_norm_rope(s[n], s["w" + n], cos, sin, c["pairing"]).to(s[n].dtype) for n in "qk")
        dq, dwq = _norm_rope_back(s["gq"], s["q"], s["wq"], cos, sin, c["pairing"])
        dk, dwk = _norm_rope_back(s["gk"], s["k"], s["wk"], cos, sin, c["pairing"])
        return dq.to(s["q"].dtype), dk.to(s["k"].dtype), dwq, dwk
    scale = c["d"] ** -0.5
    if c["op"] == "select":
        return _select(s["q"], s["k"], c["keep"], c["local"])
    if c["op"] == "sparse":
        idx, cnt = _select(s["q"], s["k"], c["keep"], c["local"])
        o, lse = _gathered(s["q"], s["k"], s["v"], idx, _width(c), scale)
        return o.to(torch.bfloat16), lse, idx, cnt
    grads = _dense_back(s, _frame_mask(s, c["N"]), scale) if c["T"] else _gathered_back(s, scale)
    return tuple(x.to(torch.bfloat16) for x in grads)


# --------------------------------------------------- the framework's calls --
def _own(s):
    from block_sparse_attention_lvsa_b200 import binding as bsa

    c = s["case"]
    if "rope" in c["op"]:
        where = {"pos": s["pos32"]} if c["listed_pos"] else {"grid": (c["t"], c["h"], c["w"])}
        rope = bsa.rope_axes(s["tables"], pairing=c["pairing"], **where)
        if c["op"] in ("rope", "rope_back"):
            return bsa.rope_apply(s["x"], rope, inverse=c["op"] == "rope_back")
        if c["op"] == "norm_rope":
            return bsa.qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], rope, eps=EPS)
        return bsa.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], rope, eps=EPS)
    if c["op"] == "select":
        return bsa.blockmean_select(s["q"], s["k"], c["keep"], local=c["local"])
    if c["op"] == "sparse":
        idx, cnt = bsa.blockmean_select(s["q"], s["k"], c["keep"], local=c["local"])
        o, lse = bsa.blocksparse_attn_fwd(s["q"], s["k"], s["v"], bsa.block_index(idx, cnt))
        return o, lse, idx, cnt
    index = bsa.lvsa_index(c["T"], s["frames"], s["counts"]) if c["T"] else bsa.block_index(s["idx"], s["cnt"])
    return bsa.blocksparse_attn_bwd(s["go"], s["q"], s["k"], s["v"], s["o"], s["lse"], index)


def run(state):
    return _own(state) if own else _plain(state)


def _tiles(case):
    """Kept pairs of tokens over all heads (block lists: whole tiles), for the operation counts."""
    if case["T"]:
        P = case["N"] // case["T"]
        return case["H"] * case["T"] * P * case["C"] * P
    return case["H"] * -(-case["N"] // BLOCK) * _width(case) * BLOCK * BLOCK


def work(case):
    op, H, d = case["op"], case["H"], case["d"]
    if "rope" in op:
        N = case["t"] * case["h"] * case["w"] + case["tail"]
        n = N * H * d
        size = SIZE[case["dtype"]]
        if op in ("rope", "rope_back"):
            return {"bytes": 2 * n * size, "flops": 3 * n}
        if op == "norm_rope":
            return {"bytes": 4 * n * size, "flops": 2 * 7 * n}
        return {"bytes": 6 * n * size, "flops": 2 * 14 * n}
    N = case["N"]
    nB = -(-N // BLOCK)
    n = N * H * d
    if op == "select":
        return {"bytes": 4 * n + 4 * H * nB * (nB + 1), "flops": 2 * n + 2 * H * nB * nB * d}
    if op == "sparse":
        return {"bytes": 8 * n + 4 * H * N + 4 * H * nB * (nB + 1), "flops": 2 * n + 2 * H * nB * nB * d + 4 * d * _tiles(case)}
    return {"bytes": 16 * n + 4 * H * N, "flops": 10 * d * _tiles(case)}


# --------------------------------------------- definitions, in 64 bits -------
def _turn(x, case, pos, sign):
    """x [N, H, d] in 64 bits with every pair of token n turned by sign * angle, as complex numbers."""
    d = case["d"]
    ang = []
    for a, pairs in enumerate(_pairs(d)):
        f = torch.tensor([THETA ** (-j / pairs) for j in range(pairs)], dtype=torch.float64, device="cuda")
        ang.append(torch.outer(pos[:, a].double() + case["start"], f))
    ang = torch.cat(ang, 1) * (pos[:, :1] >= 0)
    turn = torch.polar(torch.ones_like(ang), sign * ang)[:, None]
    if case["pairing"] == "adjacent":
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:2], d // 2, 2).contiguous()) * turn).flatten(2)
    z = torch.complex(x[..., : d // 2], x[..., d // 2:]) * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_rope(case, s):
    pos = s["pos"]
    if case["op"] == "rope":
        return _turn(s["x"].double(), case, pos, 1.0)
    if case["op"] == "rope_back":
        return _turn(s["x"].double(), case, pos, -1.0)
    out, dws = [], []
    for n in "qk":
        x, w = s[n].double(), s["w" + n].double()
        norm = torch.sqrt(torch.einsum("nhd,nhd->nh", x, x) / case["d"] + EPS)[..., None]
        if case["op"] == "norm_rope":
            out.append(_turn(x / norm * w, case, pos, 1.0))
            continue
        g = _turn(s["g" + n].double(), case, pos, -1.0)
        dws.append(torch.einsum("nhd,nhd->d", g, x / norm))
        gw = g * w
        out.append(gw / norm - x * (torch.einsum("nhd,nhd->nh", gw, x)[..., None] / (case["d"] * norm ** 3)))
    return tuple(out + dws)


def _exact_select(case, s):
    """idx and cnt by rank: a block is kept if fewer than cnt blocks come before it."""
    N, H, d = s["q"].shape
    nB = -(-N // BLOCK)
    idx = torch.full((H, nB, nB), -1, dtype=torch.int32, device="cuda")
    b = torch.arange(nB, device="cuda")
    near = (b[:, None] - b[None, :]).abs() <= case["local"]
    cnt = torch.maximum(near.sum(1), torch.full_like(b, min(case["keep"], nB)))
    size = torch.bincount(torch.arange(N, device="cuda") // BLOCK, minlength=nB).double()[:, None]
    for h in range(H):
        mq, mk = (torch.zeros((nB, d), dtype=torch.float64, device="cuda").index_add_(
            0, torch.arange(N, device="cuda") // BLOCK, s[n][:, h].double()) / size for n in "qk")
        sc = torch.where(near, math.inf, mq @ mk.T)
        order = torch.argsort(-sc, dim=1, stable=True)
        rank = torch.empty_like(order).scatter_(1, order, b.expand(nB, nB))
        keep = rank < cnt[:, None]
        put = keep.cumsum(1) - 1
        at = keep.nonzero(as_tuple=True)
        idx[h, at[0], put[at]] = at[1].to(torch.int32)
    return idx, cnt.to(torch.int32).expand(H, nB).contiguous()


def _exact_attend(case, s, idx, cnt):
    """(o, lse) or the gradients, one head and one run of query blocks after another."""
    N, H, d = s["q"].shape
    nB = -(-N // BLOCK)
    scale = d ** -0.5
    back = case["op"] == "attn_back"
    out = [torch.zeros((N, H, d), dtype=torch.float64, device="cuda") for _ in range(3 if back else 1)]
    lse = torch.zeros((H, N), dtype=torch.float64, device="cuda")
    frame = torch.arange(N, device="cuda") // (N // case["T"]) if case["T"] else None
    if case["T"]:
        allowed = torch.zeros((case["T"], case["T"]), dtype=torch.bool, device="cuda")
        for t in range(case["T"]):
            allowed[t, s["frames"][t, : case["C"]].long()] = True
    for h in range(H):
        q, k, v = (s[n][:, h].double() for n in "qkv")
        if not case["T"]:
            lists = [row[:n] for row, n in zip(idx[h].tolist(), cnt[h].tolist())]
        for i in range(nB):
            r = slice(i * BLOCK, min(N, (i + 1) * BLOCK))
            if case["T"]:
                keys, on = slice(0, N), allowed[frame[r]][:, frame]
            else:
                keys = torch.cat([torch.arange(j * BLOCK, min(N, (j + 1) * BLOCK)) for j in lists[i]]).cuda()
                on = None
            sc = q[r] @ k[keys].T * scale
            if on is not None:
                sc = torch.where(on, sc, -math.inf)
            top = torch.logsumexp(sc, 1, keepdim=True)
            p = torch.exp(sc - top)
            if not back:
                out[0][r, h], lse[h, r] = p @ v[keys], top[:, 0]
                continue
            go = s["go"][r, h].double()
            ds = go @ v[keys].T
            ds = p * (ds - torch.einsum("ij,ij->i", p, ds)[:, None]) * scale
            out[0][r, h] = ds @ k[keys]
            out[1][keys, h] += ds.T @ q[r]
            out[2][keys, h] += p.T @ go
    return tuple(out) if back else (out[0], lse)


def exact(case, seed):
    s = prepare(case, seed)
    if "rope" in case["op"]:
        return _exact_rope(case, s)
    if case["op"] == "select":
        return _exact_select(case, s)
    if case["op"] == "sparse":
        idx, cnt = _exact_select(case, s)
        return (*_exact_attend(case, s, idx, cnt), idx, cnt)
    if case["T"]:
        return _exact_attend(case, s, None, None)
    return _exact_attend(case, s, s["idx"], s["cnt"])

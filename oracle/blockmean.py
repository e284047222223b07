"""Key blocks chosen by the mean score of their tile (oracle; test
infrastructure only).

Per head, query block i and key block j of `block` tokens (the last may be
short): s(i, j) = <mean of q over i, mean of k over j>, the mean of the
tile's scores.  Row i keeps every j with |i - j| <= local, then the largest s
(equal scores: the lower j first) until it holds max(min(keep, nB), size of
the neighbourhood) blocks.  Scores are exact fractions: no rounding decides."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def block_sums(x, block):
    """[nB] lists of [H][d] exact sums of x [N, H, d]."""
    N, H, d = x.shape
    nB = -(-N // block)
    return [[[sum((Fraction(float(v)) for v in x[b * block:(b + 1) * block, h, c]), Fraction(0)) for c in range(d)]
             for h in range(H)] for b in range(nB)]


def keep_row(scores, i, keep, local):
    """Ascending kept blocks of row i given its scores."""
    nB = len(scores)
    own = [j for j in range(nB) if abs(i - j) <= local]
    rest = sorted((j for j in range(nB) if abs(i - j) > local), key=lambda j: (-scores[j], j))
    return sorted(own + rest[:max(0, min(keep, nB) - len(own))])


def select_exact(q, k, keep, local, block=128):
    """lists[h][i] for small inputs, in exact fractions."""
    N, H, d = q.shape
    sq, sk = block_sums(q, block), block_sums(k, block)
    nB = len(sq)
    rows = [min(block, N - b * block) for b in range(nB)]
    out = []
    for h in range(H):
        out.append([])
        for i in range(nB):
            s = [sum((a * b for a, b in zip(sq[i][h], sk[j][h])), Fraction(0)) / rows[j] for j in range(nB)]
            out[h].append(keep_row(s, i, keep, local))
    return out


def select(q, k, keep, local, block=128):
    """(idx [H, nB, nB] int32 padded with -1, cnt [H, nB]) in float64."""
    N, H, d = q.shape
    nB = -(-N // block)
    pad = nB * block - N
    rows = np.full(nB, block, dtype=np.float64)
    rows[-1] -= pad
    m = [np.pad(x, ((0, pad), (0, 0), (0, 0))).reshape(nB, block, H, d).sum(1) / rows[:, None, None] for x in (q, k)]
    idx = np.full((H, nB, nB), -1, dtype=np.int32)
    cnt = np.zeros((H, nB), dtype=np.int32)
    for h in range(H):
        s = m[0][:, h] @ m[1][:, h].T
        s = np.where(np.isnan(s), -np.inf, s)
        for i in range(nB):
            kept = keep_row(list(s[i]), i, keep, local)
            idx[h, i, :len(kept)], cnt[h, i] = kept, len(kept)
    return idx, cnt

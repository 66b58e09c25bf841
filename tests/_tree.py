"""The operators of a tree decode step in 64 bits, on the CPU, straight from
their definitions (include/oasis.h), and the error bounds of the GPU's.

Rotation.  An angle is off by at most 2^-23 of a turn (its 32 bits become an
fp32 number of half turns: 2^-25 half turns; cos and sin add a few units of
2^-24): cos and sin by ROT = 2 pi 2^-24 + 2^-22 < 2^-20.  A turned entry is two
products and a sum in fp32: off by at most (ROT + 3 * 2^-24) (|a| + |b|) * scale,
then rounded once.

Tree attention.
* x = log2(e) * scale * q.k: products of split queries, summed in fp32, at most
  500 roundings or truncations of 2^-23 of A = scale log2(e) sum |q_i k_i|; a
  split query entry is off by at most 2^-19 of its row's largest, so x by 2^-19
  of B = scale log2(e) max|q| sum |k_i|.
* 2^x: two units of 2^-23; the difference of x and the maximum, 2^-23 A.
* Weights are rounded to fp16 (2^-11), those under 2^-21 of the largest by at
  most 2^-32 of it; values, in units of the largest scale 448 * 2^e of the
  request's tokens, by at most 2^-39 of that.
"""
import math

import numpy as np
import torch

from tests import _q8 as Q

D, B = 128, 16
ROT = 2.0 ** -20


def rotate(x, positions, rope):
    """(turned, bound of fp32's error) [T][H][128] in 64 bits; angles exact to 2^-64 of a turn."""
    x = x.double().cpu().numpy()
    pos = positions.cpu().reshape(-1, x.shape[0]).numpy()
    half, scale = rope.rot_dim // 2, float(rope.scale) or 1.0
    y, bound = x.copy(), np.zeros_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if rope.interleaved else (i, i + half)
        w = np.zeros(x.shape[0])
        for t in range(x.shape[0]):
            w[t] = angle(int(pos[rope.axis[i], t]), rope.frequency[i])
        c, s = np.cos(w)[:, None], np.sin(w)[:, None]
        y[:, :, a] = scale * (x[:, :, a] * c - x[:, :, b] * s)
        y[:, :, b] = scale * (x[:, :, a] * s + x[:, :, b] * c)
        with np.errstate(invalid="ignore"):
            e = (ROT + 3 * 2.0 ** -24) * scale * (np.abs(x[:, :, a]) + np.abs(x[:, :, b]))
        bound[:, :, a], bound[:, :, b] = e, e
    return y, bound


# 2 pi as an integer over 2^200 (from Machin's series, in whole numbers)
def _two_pi():
    one = 1 << 240

    def atan_inv(n):
        total, term, k = 0, one // n, 0
        while term:
            total += term // (2 * k + 1) * (-1) ** k
            term //= n * n
            k += 1
        return total
    return (8 * (4 * atan_inv(5) - atan_inv(239))) >> 40


TWO_PI = _two_pi()


def angle(position, frequency):
    """position * frequency modulo 2 pi, in [-pi, pi], from whole numbers."""
    from fractions import Fraction
    f = Fraction(frequency) * position
    turn = Fraction(TWO_PI, 1 << 200)
    return float(f - round(f / turn) * turn)


def words_of(parents):
    """Plain: node i sees itself and what its parent sees."""
    out = []
    for i, p in enumerate(parents):
        out.append((1 << i) | (out[p] if p >= 0 else 0))
    return out


def random_tree(N, g, back=6):
    return [max(-1, i - 1 - int(torch.randint(0, back, (1,), generator=g))) for i in range(N)]


def signed(words):
    """64-bit words as int64."""
    return torch.tensor([[w - (1 << 64) if w >> 63 else w for w in row] for row in words], dtype=torch.int64)


def attention(q, words, sizes, pages, table, lens, scale=None, out=None):
    """(o, bound, is_node) of oasis_q8_tree_attn; words: whole numbers [R][N]."""
    R, N, Hq, _ = q.shape
    H = pages.shape[1]
    G = Hq // H
    scale = scale or 1.0 / math.sqrt(D)
    qn = q.double().cpu().numpy()
    o = np.zeros((R, N, Hq, D))
    bound = np.zeros_like(o)
    node = np.zeros((R, N), dtype=bool)
    for r in range(R):
        n = N if sizes is None else min(max(int(sizes[r]), 0), N)
        node[r, :n] = True
        L = max(0, int(lens[r]))
        if L < n:
            continue
        k, v, at, E = Q.tokens_and_scales(pages, table[r], L)
        for i in range(n):
            see = np.array([t < L - n or bool(int(words[r][i]) >> (t - (L - n)) & 1) for t in at.tolist()], dtype=bool)
            if not see.any():
                continue
            for hq in range(Hq):
                h = hq // G
                kk, vv = k[h, see], v[h, see]
                x = kk @ qn[r, i, hq] * scale
                A = (np.abs(kk) @ np.abs(qn[r, i, hq])).max() * scale * math.log2(math.e)
                Bq = np.abs(kk).sum(1).max() * np.abs(qn[r, i, hq]).max() * scale * math.log2(math.e)
                p = np.exp(x - x.max())
                l = p.sum()
                o[r, i, hq] = p @ vv / l
                e = 2.0 ** -11 + math.log(2) * (501 * 2.0 ** -23 * A + 2.0 ** -19 * Bq) + 2.0 ** -20
                U = 448 * E[h].max()
                bound[r, i, hq] = 2 * e * (p @ np.abs(vv)) / l + (see.sum() * 2.0 ** -32 + 2.0 ** -39) * U
    bound += Q.HALF[out] * np.abs(o) * 1.01 + 1e-30 if out is not None else 0.0
    return o, bound, node


def keep(pages, table, lens, sizes, N, nodes, n_keep):
    """oasis_q8_keep on numpy pages."""
    new = pages.copy()
    for r in range(len(lens)):
        n = N if sizes is None else min(max(int(sizes[r]), 0), N)
        base = int(lens[r]) - n
        if int(lens[r]) <= 0 or base < 0:
            continue
        for i in range(min(max(int(n_keep[r]), 0), min(nodes.shape[1], n))):
            x = int(nodes[r, i])
            if not 0 <= x < n:
                continue
            (a, s), (b, d) = divmod(base + x, B), divmod(base + i, B)
            p, w = int(table[r, a]), int(table[r, b])
            if not (0 <= p < pages.shape[0] and 0 <= w < pages.shape[0]):
                continue
            dim = np.arange(D)
            new[w][:, Q.key_at(d, dim)] = pages[p][:, Q.key_at(s, dim)]
            new[w][:, Q.value_at(d, dim)] = pages[p][:, Q.value_at(s, dim)]
            new[w][:, [4096 + d, 4112 + d]] = pages[p][:, [4096 + s, 4112 + s]]
    return new


def logprobs(x, tokens, k):
    """(logprobs, entropy, ids, top) in 64 bits of a float tensor [rows][V]."""
    x = x.double().cpu().numpy()
    rows, V = x.shape
    lp, H = np.full(rows, np.nan), np.full(rows, np.nan)
    ids, top = np.full((rows, k), -1), np.full((rows, k), -np.inf)
    for r in range(rows):
        m = x[r].max()
        order = np.lexsort((np.arange(V), -x[r]))[:k]
        ids[r, :len(order)] = order
        if not np.isfinite(m):
            top[r, :len(order)] = np.nan
            if tokens is not None and tokens[r] >= V:
                lp[r] = -np.inf
            continue
        y = x[r] - m
        e = np.exp(y)
        S = e.sum()
        H[r] = math.log(S) - np.where(e > 0, e * np.where(e > 0, y, 0), 0).sum() / S
        top[r, :len(order)] = y[order] - math.log(S)
        if tokens is not None:
            lp[r] = y[tokens[r]] - math.log(S) if 0 <= tokens[r] < V else -np.inf
    return lp, H, ids, top

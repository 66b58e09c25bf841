"""The decode operators over the 8-bit cache in 64 bits, on the CPU, straight
from their definitions (include/oasis.h), and the error bounds of the GPU's.

Bounds.  A rounding to a type is off by at most half its step,
torch.finfo(t).eps / 2 of the value.  The attention kernels
* form x = log2(e) * scale * q.k in fp32: at most 2 * 130 roundings or
  truncations of 2^-23 of the sum A of the terms' absolute values,
* take 2^x (two units of 2^-23, and the logarithm's rounding at most 2^-23 |x|
  <= 2^-23 A),
* round the weights to fp16 (8-bit pages) or bf16 (prefix) before the second
  product, and sum at most N terms in fp32.
* round weights under 2^-28 of the largest weighted one by at most 2^-39 of it
  (fp16's least step is 2^-24, the largest weight 2^14): with E the value scale
  448 * 2^e of the token whose p * 2^e is largest, a token adds at most
  2^-39 * 448 * 2^e * p_there <= 2^-39 E to the numerator's sum p v, which is
  divided by l >= p_there; N tokens add at most 2^-39 N E to the output.
The weights' common relative error e = 2^-11 (2^-8) + ln 2 * 270 * 2^-23 * A +
2^-20 enters numerator and denominator: |o - o'| <= 2 e * sum p |v| / l, plus
2^-39 N E and the output's own rounding.
"""
import math

import numpy as np
import torch

D, B, UNIT = 128, 16, 4128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def e4m3_table():
    """The 256 codes' values, NaN for 0x7f and 0xff."""
    c = np.arange(256)
    ex, man = (c >> 3) & 15, c & 7
    v = np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >> 7, -v, v)


TABLE = e4m3_table()


def quantise(x):
    """(codes uint8, exponents int) of rows of 128 values (any float tensor), by search over the
    table: nearest value, ties to the even code."""
    x = x.double().cpu().numpy()
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = fin.max(-1)
    e = np.full(a.shape, -100, dtype=np.int64)
    for k in range(-100, 121):          # least e with a <= 448 * 2^e
        e = np.where(a > 448.0 * 2.0 ** k, np.minimum(k + 1, 120), e)
    with np.errstate(over="ignore", invalid="ignore"):
        y = x * 2.0 ** (-e[..., None].astype(np.float64))
        pos = TABLE[:127]               # codes 0..126 in order of value
        m = np.minimum(np.abs(y), 448.0)
        m = np.where(np.isnan(m), 0.0, m)
        hi = np.searchsorted(pos, m).clip(0, 126)
        lo = np.maximum(hi - 1, 0)
        dl, dh = m - pos[lo], pos[hi] - m
        c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = c | (np.signbit(x).astype(np.int64) << 7)
    nan = np.isnan(x)
    return np.where(nan, 0x7F, c).astype(np.uint8), e, nan


def key_at(j, i):
    return D * j + (i ^ (64 * (j & 1)))


def value_at(j, i):
    return 2048 + 16 * i + j


def write(pages, k, v, slots):
    """Codes into pages (numpy uint8 [P][H][4128]) as oasis_q8_write; returns a mask of the bytes
    that hold a NaN code (its sign is free)."""
    kc, ke, kn = quantise(k)
    vc, ve, vn = quantise(v)
    free = np.zeros(pages.shape, dtype=bool)
    i = np.arange(D)
    for t, slot in enumerate(slots.tolist()):
        if slot < 0 or slot >= pages.shape[0] * B:
            continue
        p, j = slot // B, slot % B
        pages[p][:, key_at(j, i)] = kc[t]
        pages[p][:, value_at(j, i)] = vc[t]
        free[p][:, key_at(j, i)] = kn[t]
        free[p][:, value_at(j, i)] = vn[t]
        pages[p][:, 4096 + j] = ke[t] + 127
        pages[p][:, 4112 + j] = ve[t] + 127
    return free


def tokens(pages, row, n):
    """(keys, values) [H][n][128] fp64 of one request's first n tokens; tokens of bad pages are
    left out (a third result names the tokens that are there)."""
    return tokens_and_scales(pages, row, n)[:3]


def tokens_and_scales(pages, row, n):
    """`tokens` and the values' scales 2^e [H][n]."""
    P, H = pages.shape[:2]
    K, V, at, E = [], [], [], []
    i = np.arange(D)
    for t in range(n):
        p, j = int(row[t // B]), t % B
        if p < 0 or p >= P:
            continue
        u = pages[p]
        K.append(TABLE[u[:, key_at(j, i)]] * 2.0 ** (u[:, 4096 + j].astype(np.float64) - 127)[:, None])
        V.append(TABLE[u[:, value_at(j, i)]] * 2.0 ** (u[:, 4112 + j].astype(np.float64) - 127)[:, None])
        E.append(2.0 ** (u[:, 4112 + j].astype(np.float64) - 127))
        at.append(t)
    if not K:
        z = np.zeros((H, 0, D))
        return z, z, np.zeros(0, dtype=np.int64), np.zeros((H, 0))
    return np.stack(K, 1), np.stack(V, 1), np.asarray(at), np.stack(E, 1)


def attention(q, pages, table, lens, causal, scale=None, prefix=None, p_half=2.0 ** -11, out=None):
    """(o, bound) [S][R][Hq][128] fp64: the attention and how far a kernel's may be from it.
    `prefix` = (keys, values) [H][P][128] fp64."""
    S, R, Hq, _ = q.shape
    H = pages.shape[1]
    G = Hq // H
    scale = scale or 1.0 / math.sqrt(D)
    qn = q.double().cpu().numpy()
    o = np.zeros((S, R, Hq, D))
    bound = np.zeros_like(o)
    for r in range(R):
        n = max(0, int(lens[r]))
        k, v, at, E = tokens_and_scales(pages, table[r], n)
        for s in range(S):
            see = at < (n - (S - 1 - s) if causal else n)
            kk, vv = k[:, see], v[:, see]
            if prefix is not None:
                kk, vv = np.concatenate([prefix[0], kk], 1), np.concatenate([prefix[1], vv], 1)
            if kk.shape[1] == 0:
                continue
            for hq in range(Hq):
                h = hq // G
                x = kk[h] @ qn[s, r, hq] * scale
                A = (np.abs(kk[h]) @ np.abs(qn[s, r, hq])).max() * scale * math.log2(math.e)
                p = np.exp(x - x.max())
                l = p.sum()
                o[s, r, hq] = p @ vv[h] / l
                e = p_half + math.log(2) * 270 * 2.0 ** -23 * A + 2.0 ** -20
                bound[s, r, hq] = 2 * e * (p @ np.abs(vv[h])) / l
                if see.any():
                    w = p[-int(see.sum()):] * E[h, see]
                    bound[s, r, hq] += 2.0 ** -39 * see.sum() * 448 * E[h, see][w.argmax()]
    bound += HALF[out] * np.abs(o) * 1.01 + 1e-30 if out is not None else 0.0
    return o, bound


def verify(target, draft, x, ua, us, n_drafts=None):
    """(tokens, n_accept) from the definition in fp64."""
    R, n1, V = target.shape
    n = n1 - 1
    p = target.double().cpu().numpy()
    q = draft.double().cpu().numpy() if draft is not None else None
    x, ua, us = x.cpu().numpy(), ua.double().cpu().numpy(), us.double().cpu().numpy()
    out = np.full((R, n + 1), -1, dtype=np.int64)
    acc = np.zeros(R, dtype=np.int64)
    for r in range(R):
        m = n if n_drafts is None else min(max(int(n_drafts[r]), 0), n)
        if any(not 0 <= x[r, i] < V for i in range(m)):
            acc[r] = -1
            continue
        k = 0
        positive = lambda a: np.where(a > 0, a, 0.0)  # noqa: E731  (NaN and negative entries count as 0)
        while k < m and ua[r, k] * (positive(q[r, k, x[r, k]]) if q is not None else 1.0) < positive(p[r, k, x[r, k]]):
            out[r, k] = x[r, k]
            k += 1
        acc[r] = k
        w = p[r, k]
        if k < m:
            d = q[r, k] if q is not None else (np.arange(V) == x[r, k]) * max(1.0, p[r, k, x[r, k]])
            if np.isposinf(d).any():
                continue
            left = np.maximum(positive(w) - positive(d), 0.0)
            if left.sum() > 0 or np.isposinf(w).any():
                w = left
        c = np.cumsum(positive(w))
        if c[-1] > 0 and np.isfinite(c[-1]):
            j = int(np.searchsorted(c, us[r] * c[-1], side="right"))
            out[r, k] = min(j, int(np.nonzero(positive(w))[0][-1]))
    return out, acc


def table_of(lens, num_pages, max_blocks, g, low=0):
    """A page table [R][max_blocks] int32 with distinct random pages >= low, -1 past each
    request's blocks."""
    nb = [-(-max(0, int(n)) // B) for n in lens]
    order = (torch.randperm(num_pages - low, generator=g) + low).to(torch.int32)
    t = torch.full((len(nb), max_blocks), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(nb):
        t[r, :n] = order[at:at + n]
        at += n
    assert at <= num_pages - low
    return t


def slots_of(table, r, lo, hi):
    """Slots of tokens [lo, hi) of request r."""
    t = torch.arange(lo, hi)
    return table[r, t // B].long() * B + t % B

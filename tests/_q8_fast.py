"""tests/_q8.py's attention for long contexts and large batches: the same
definition and bound in 64-bit torch operations, a request and KV head at a
time, on the device that the pages are on."""
import math

import torch

from tests import _q8 as Q


def units(pages, row, n, h):
    """Keys, values [n][128] and the values' scales [n] in 64 bits of a request's first n tokens,
    head h; `row` its table entries, all of them in the pool."""
    dev = pages.device
    t = torch.arange(n, device=dev)
    j = t % 16
    b = pages[row[t // 16].long(), h]                                  # [n][4128]
    i = torch.arange(128, device=dev)
    table = torch.from_numpy(Q.TABLE).to(dev)
    k = table[b.gather(1, 128 * j[:, None] + (i ^ (64 * (j[:, None] & 1)))).long()]
    v = table[b.gather(1, 2048 + 16 * i + j[:, None]).long()]
    ke = b.gather(1, (4096 + j)[:, None]).double() - 127
    ve = b.gather(1, (4112 + j)[:, None]).double() - 127
    return k * torch.exp2(ke), v * torch.exp2(ve), torch.exp2(ve[:, 0])


def attention(q, pages, table, lens, causal, out, scale=None, prefix=None, p_half=2.0 ** -11):
    """(o, bound) as numpy [S][R][Hq][128]; prefix = (keys, values) [H][P][128] in 64 bits on the
    pages' device."""
    S, R, Hq, _ = q.shape
    H, dev = pages.shape[1], pages.device
    G = Hq // H
    scale = scale or 1.0 / math.sqrt(128)
    q64 = q.double().to(dev)
    table = table.to(dev)
    o = torch.zeros(S, R, Hq, 128, dtype=torch.float64, device=dev)
    bound = torch.zeros_like(o)
    P = 0 if prefix is None else prefix[0].shape[1]
    for r in range(R):
        n = max(0, int(lens[r]))
        for h in range(H):
            k, v, E = units(pages, table[r], n, h)
            if P:
                k, v = torch.cat([prefix[0][h], k]), torch.cat([prefix[1][h], v])
                E = torch.cat([torch.zeros(P, dtype=torch.float64, device=dev), E])
            if k.shape[0] == 0:
                continue
            x = q64[:, r, h * G:(h + 1) * G].reshape(S * G, 128)
            less = torch.arange(S - 1, -1, -1, device=dev).repeat_interleave(G) if causal else torch.zeros(S * G, device=dev)
            pos = torch.arange(k.shape[0], device=dev) - P
            see = (pos < 0) | (pos < (n - less)[:, None])              # [S*G][tokens]
            s = torch.where(see, x @ k.T * scale, -math.inf)
            m = s.amax(1, keepdim=True)
            p = torch.where(see, torch.exp(s - torch.where(torch.isinf(m), 0.0, m)), 0.0)
            l = p.sum(1, keepdim=True)
            A = torch.where(see, x.abs() @ k.abs().T, 0.0).amax(1, keepdim=True) * scale * math.log2(math.e)
            e = p_half + math.log(2) * 270 * 2.0 ** -23 * A + 2.0 ** -20
            w = p * E
            at = w[:, P:].argmax(1) + P if n else None
            extra = 2.0 ** -39 * see[:, P:].sum(1) * 448 * E[at] if n else 0.0
            some = l > 0
            oo = torch.where(some, p @ v / l, 0.0)
            bb = torch.where(some, 2 * e * (p @ v.abs()) / l + (extra[:, None] if n else 0.0), 0.0)
            o[:, r, h * G:(h + 1) * G] = oo.view(S, G, 128)
            bound[:, r, h * G:(h + 1) * G] = bb.view(S, G, 128)
    bound += Q.HALF[out] * o.abs() * 1.01 + 1e-30
    return o.cpu().numpy(), bound.cpu().numpy()

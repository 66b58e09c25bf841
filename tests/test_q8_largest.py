"""The largest sizes that the header allows, one at a time: the longest context
and prefix, the most requests, the longest rows and most drafts, tokens far
apart in memory."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _q8_fast as F
from tests.test_q8 import BF, FP, HF, close, dev, gen  # noqa: F401
from tests.test_verify_drafts import draw, go

pytestmark = pytest.mark.gpu


def random_pages(P, H):
    """Pages of finite codes under 1 (0x38) and exponents of a few powers of two."""
    g = torch.Generator(device="cuda")
    g.manual_seed(P)
    pages = torch.randint(0, 0x38, (P, H, Q.UNIT), generator=g, dtype=torch.uint8, device="cuda")
    pages[..., :4096] |= torch.randint(0, 2, (P, H, 4096), generator=g, dtype=torch.uint8, device="cuda") << 7
    pages[..., 4096:] = torch.randint(125, 129, (P, H, 32), generator=g, dtype=torch.uint8, device="cuda")
    return pages


@pytest.mark.parametrize("S,G,ragged", [(1, 4, False), (4, 4, True)])
def test_longest_context(dev, S, G, ragged):  # noqa: F811
    """131072 blocks, 2097152 tokens, in parts and in one cluster; a second, short request beside it."""
    blocks = 131072
    lens = [blocks * 16 - 3, 40] if ragged else [blocks * 16]
    pages = random_pages(blocks, 1)
    c = ob.Q8Cache(ob.make_q8_config(blocks, blocks, G, 1, out_fp32=True), pages=pages)
    table = torch.randperm(blocks, generator=gen(1)).to(torch.int32).repeat(len(lens), 1)
    q = (2 * torch.randn(S, len(lens), G, 128, generator=gen(2))).to(BF)
    out = torch.zeros(q.shape, dtype=FP, device=dev)
    t, m = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    o, b = F.attention(q, pages, table, lens, True, FP)
    assert c.oasis_q8_attn_workspace(len(lens), S) > 0
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=dev)):
        out.zero_()
        c.oasis_q8_attn(q.cuda(), t, m, out, causal=True, workspace=ws)
        assert c.oasis_q8_sync() == 0
        close(out, o, b)


def test_longest_prefix(dev):  # noqa: F811
    """131072 blocks of one KV head behind which two requests have a few tokens."""
    blocks, S, R, G = 131072, 2, 2, 4
    plen = blocks * 16 - 5
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    kv = torch.randn(1, blocks, 2, 16, 128, generator=g, device=dev).to(BF)
    pages = random_pages(4, 1)
    c = ob.Q8Cache(ob.make_q8_config(4, 2, G, 1, out_fp32=True), pages=pages)
    lens, table = [20, 0], torch.tensor([[1, 3], [0, 0]], dtype=torch.int32)
    q = torch.randn(S, R, G, 128, generator=gen(4)).to(BF)
    out = torch.zeros(q.shape, dtype=FP, device=dev)
    c.oasis_prefix_attn(q.cuda(), kv, plen, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), out,
                        c.prefix_workspace(R, S, plen), causal=True)
    assert c.oasis_q8_sync() == 0
    ref = tuple(kv[:, :, i].reshape(1, -1, 128)[:, :plen].double() for i in (0, 1))
    o, b = F.attention(q, pages, table, lens, True, FP, prefix=ref, p_half=2.0 ** -8)
    close(out, o, b)


@pytest.mark.parametrize("plen", [0, 300])
def test_most_requests(dev, plen):  # noqa: F811
    """65535 requests of up to two blocks: every one of them gets its own output (single tokens'
    outputs are their values), read back and attended to, with and without a prefix."""
    R, P = 65535, 500
    pages = random_pages(P, 1)
    c = ob.Q8Cache(ob.make_q8_config(P, 2, 1, 1, out_fp32=True), pages=pages)
    g = gen(5)
    table = torch.randint(0, P, (R, 2), generator=g).to(torch.int32)
    lens = torch.randint(0, 33, (R,), generator=g).to(torch.int32)
    lens[-1] = 17
    q = torch.randn(1, R, 1, 128, generator=g).to(BF)
    out = torch.full(q.shape, 9.0, dtype=FP, device=dev)
    kv = torch.randn(1, 20, 2, 16, 128, generator=g).to(BF).cuda()
    if plen:
        c.oasis_prefix_attn(q.cuda(), kv, plen, table.cuda(), lens.cuda(), out, c.prefix_workspace(R, 1, plen))
    else:
        c.oasis_q8_attn(q.cuda(), table.cuda(), lens.cuda(), out)
    back = torch.full((R, 1, 2, 2, 16, 128), 9.0, dtype=FP, device=dev)
    c.oasis_q8_read(table.cuda(), lens.cuda(), back)
    assert c.oasis_q8_sync() == 0
    # all requests at once, in 64 bits, from the units of the whole pool
    tok = torch.arange(P * 16, device=dev)
    k, v, E = F.units(pages, torch.arange(P, device=dev), P * 16, 0)
    at = (table.cuda().long()[:, :, None] * 16 + torch.arange(16, device=dev)).view(R, 32)
    there = torch.arange(32, device=dev) < lens.cuda()[:, None]
    want = torch.where(there[:, :, None], k[at], 9.0)
    assert torch.equal(back[:, 0, :, 0].reshape(R, 32, 128).double(), want)
    want = torch.where(there[:, :, None], v[at], 9.0)
    assert torch.equal(back[:, 0, :, 1].reshape(R, 32, 128).double(), want)
    del want, back
    x = torch.einsum("rd,rtd->rt", q[0, :, 0].double().cuda(), k[at])
    a = torch.einsum("rd,rtd->rt", q[0, :, 0].double().cuda().abs(), k[at].abs())
    s = torch.where(there, x / 128 ** 0.5, -torch.inf)
    A = torch.where(there, a, 0.0).amax(1)
    vals, vabs = v[at], v[at].abs()
    p_half, pv = 2.0 ** -11, None
    if plen:
        pk, pv = (kv[0, :, i].reshape(-1, 128)[:plen].double() for i in (0, 1))
        s = torch.cat([s, q[0, :, 0].double().cuda() @ pk.T / 128 ** 0.5], 1)
        A = torch.maximum(A, (q[0, :, 0].double().cuda().abs() @ pk.abs().T).amax(1))
        p_half = 2.0 ** -8
    top = s.amax(1, keepdim=True)
    w = torch.where(torch.isinf(s), 0.0, torch.exp(s - torch.where(torch.isinf(top), 0.0, top)))
    l = w.sum(1, keepdim=True)
    o = torch.einsum("rt,rtd->rd", w[:, :32], vals)
    m = torch.einsum("rt,rtd->rd", w[:, :32], vabs)
    if plen:
        o, m = o + w[:, 32:] @ pv, m + w[:, 32:] @ pv.abs()
    o, m = (torch.where(l > 0, y / l, 0.0) for y in (o, m))
    e = p_half + 0.6932 * 270 * 2.0 ** -23 * A * 1.4427 / 128 ** 0.5 + 2.0 ** -20
    b = 2 * e[:, None] * m + 2.0 ** -39 * 32 * 448 * 2 + 2.0 ** -24 * o.abs() * 1.01 + 1e-30
    close(out[0, :, 0], o.cpu().numpy(), b.cpu().numpy())


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("R,n,V", [(2, 1, 1 << 20), (1, 0, (1 << 20) - 1), (1, 2, 1 << 18), (1, 1, (1 << 18) + 1), (5, 64, 2000)])
def test_longest_rows_and_most_drafts(dev, dtype, R, n, V):  # noqa: F811
    p, q, x, ua, us = draw(R, n, V, gen(V + n), dtype)
    if n == 64:
        ua[:4] *= 0.0                                     # all of them accepted, but for one
        ua[1, 63] = 1.0
        q[1, 63, x[1, 63].long()] = 1.0
    for d in (q, None):
        wt, wa = Q.verify(p, d, x, ua, us)
        tok, acc = go(p, d, x, ua, us)
        assert np.array_equal(acc, wa) and np.array_equal(tok, wt)
        if n == 64:
            assert wa[0] == 64 and wa[1] == 63 or d is None


def test_most_verified_requests(dev):  # noqa: F811
    """2^20 requests over a vocabulary of seven: against the definition for all of them at once."""
    R, V = 1 << 20, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    p = torch.rand(R, 2, V, generator=g, device=dev)
    q = torch.rand(R, 1, V, generator=g, device=dev)
    x = torch.randint(0, V, (R, 1), generator=g, device=dev).int()
    ua, us = torch.rand(R, 1, generator=g, device=dev), torch.rand(R, generator=g, device=dev)
    tok, acc = go(p, q, x, ua, us)
    P, D = p.double(), q.double()
    yes = ua[:, 0].double() * D[:, 0].gather(1, x.long())[:, 0] < P[:, 0].gather(1, x.long())[:, 0]
    w = torch.where(yes[:, None], P[:, 1], (P[:, 0] - D[:, 0]).clamp(min=0))
    w = torch.where(w.sum(1, keepdim=True) > 0, w, P[:, 0])
    c = w.cumsum(1)
    j = (c <= us.double()[:, None] * c[:, -1:]).sum(1).cpu().numpy()
    yes = yes.cpu().numpy()
    assert np.array_equal(acc, yes.astype(np.int32))
    assert np.array_equal(tok[np.arange(R), yes.astype(int)], j)
    assert np.array_equal(tok[yes, 0], x.cpu().numpy()[yes, 0]) and (tok[~yes, 1] == -1).all()


def test_tokens_far_apart(dev):  # noqa: F811
    """Tokens' keys and values in rows of 1.5 MB: offsets past 2^32 bytes, 2^31 elements."""
    T, H, wide = 2900, 2, 6144 * 128
    x = torch.empty(T, wide, dtype=BF, device=dev)
    assert (T - 1) * wide > 1 << 31
    at = [0, wide - H * 128]
    k, v = (x[:, a:a + H * 128].view(T, H, 128) for a in at)
    g = gen(10)
    kc, vc = (torch.randn(2, T, H, 128, generator=g) * torch.exp2(2 * torch.randn(2, T, H, 1, generator=g))).to(BF)
    k.copy_(kc), v.copy_(vc)
    P = -(-T // 16) + 1
    c = ob.Q8Cache(ob.make_q8_config(P, 1, H, H))
    slots = torch.arange(T) + 5
    want = np.zeros((P, H, Q.UNIT), dtype=np.uint8)
    Q.write(want, kc, vc, slots)
    c.oasis_q8_write(k, v, slots.cuda())
    assert c.oasis_q8_sync() == 0
    assert np.array_equal(c.pages.cpu().numpy(), want)

"""Forms of the attention kernels over the 8-bit cache that only some sizes
reach, against the definition in 64 bits: one and two warps a CTA, more than
32 parts or shares of one axis, two row tiles behind a prefix of several key
tiles, and maxima that move between tiles, parts and shares."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _q8_fast as F
from tests.test_q8 import BF, FP, HF, close, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def levels(k, g, high=40.0):
    """Give keys [..., tokens, 128] (cast in place) score levels along the context that queries of
    `steep` pick: dim 0 climbs, dim 1 falls, dim 2 is drawn anew every 100 tokens."""
    n = k.shape[-2]
    t = torch.linspace(-1, 1, n)
    k[..., 0], k[..., 1] = t * high, -t * high
    k[..., 2] = (2 * torch.rand(-(-n // 100), generator=g) - 1).repeat_interleave(100)[:n] * high
    return k


def steep(q):
    """Queries [..., 128] whose rows follow one of the levels each (or none), as base-2 logarithms
    of about the levels' size."""
    rows = q.reshape(-1, 128)
    rows[:, :3] = 0
    for i in range(3):
        rows[i::4, i] = 128 ** 0.5 / 1.44
    return q


def run(c, q, table, lens, causal, ws=None):
    out = torch.full(q.shape, 5.0, dtype=FP if c.cfg.out_fp32 else q.dtype, device="cuda")
    t, m = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    c.oasis_q8_attn(q.cuda(), t, m, out, causal=causal, workspace=ws)
    assert c.oasis_q8_sync() == 0
    return out


def check(c, q, table, lens, causal, out, **kw):
    o, b = F.attention(q, c.pages, table, lens, causal, out.dtype, **kw)
    close(out, o, b)


def cache(lens, blocks, Hq, Hkv, g, fp32=True, shape_keys=None):
    """A cache with its pages written (values of uneven sizes) and a table in random order, blocks of
    one request in the order of its context."""
    nb = [-(-n // 16) for n in lens]
    P = sum(nb) + 3
    c = ob.Q8Cache(ob.make_q8_config(P, blocks, Hq, Hkv, out_fp32=fp32))
    table = Q.table_of(lens, P, blocks, g)
    for r, n in enumerate(lens):
        if n == 0:
            continue
        k = torch.randn(Hkv, n, 128, generator=g)
        v = torch.randn(n, Hkv, 128, generator=g) * torch.exp2(torch.randn(n, Hkv, 1, generator=g))
        if shape_keys:
            k = shape_keys(k)
        k = k.transpose(0, 1).contiguous()
        c.oasis_q8_write(k.cuda(), v.cuda(), Q.slots_of(table, r, 0, n).cuda())
    assert c.oasis_q8_sync() == 0
    return c, table


def ragged(R, most, g):
    lens = torch.randint(1, most + 1, (R,), generator=g).tolist()
    lens[0], lens[R // 2], lens[-1] = most, 0, 1
    return lens


# Pairs (request, KV head) past what the card holds in CTAs of four warps, over tables of few blocks.
@pytest.mark.parametrize("R,Hkv,blocks,S,G", [
    (64, 8, 8, 1, 1), (64, 8, 8, 2, 4), (64, 8, 16, 1, 8),          # one warp, one column tile
    (64, 8, 20, 1, 1), (60, 8, 32, 2, 4), (30, 16, 17, 1, 5),       # two warps
    (44, 8, 20, 4, 4), (20, 16, 32, 3, 5), (44, 8, 20, 4, 8),       # two warps, two column tiles (twice)
    (64, 8, 40, 1, 4), (44, 8, 36, 4, 4)], ids=str)                 # four
@pytest.mark.parametrize("dtype,fp32", [(BF, True), (HF, False), (BF, False), (HF, True)])
def test_many_short_contexts(dev, R, Hkv, blocks, S, G, dtype, fp32):  # noqa: F811
    g = gen(R + blocks + S)
    lens = ragged(R, 16 * blocks, g)
    c, table = cache(lens, blocks, G * Hkv, Hkv, g, fp32)
    assert c.oasis_q8_attn_workspace(R, S) == 0
    q = (2 * torch.randn(S, R, G * Hkv, 128, generator=g)).to(dtype)
    for causal in {False, S > 1}:
        check(c, q, table, lens, causal, run(c, q, table, lens, causal))


@pytest.mark.parametrize("R,Hkv,S,G", [(64, 8, 1, 4), (64, 8, 2, 4), (129, 2, 4, 4)])
@pytest.mark.parametrize("plen", [0, 600])
def test_clusters_of_which_short_requests_take_a_part(dev, R, Hkv, S, G, plen):  # noqa: F811
    """More clusters than the card holds at once: a request takes as many of a cluster's CTAs as have
    six groups a warp, the others leave (the grid's last one too, behind a prefix)."""
    g = gen(R + S + plen)
    lens = torch.randint(0, 300, (R,), generator=g).tolist()
    lens[1:8] = [8192, 0, 1600, 3100, 1536, 1537, 6000]
    lens[-2:] = [8191, 1]
    if plen:
        c, table, lens, kv, ref, q = prefix_case(R, S, G, Hkv, plen, 8192, g, lens=lens)
        out = run_prefix(c, q, kv, plen, table, lens, S > 1)
        return check(c, q, table, lens, S > 1, out, prefix=ref, p_half=2.0 ** -8)
    c, table = cache(lens, 512, G * Hkv, Hkv, g)
    if c.oasis_q8_attn_workspace(R, S):
        pytest.fail("these sizes are cut into parts")
    q = (2 * torch.randn(S, R, G * Hkv, 128, generator=g)).to(BF)
    check(c, q, table, lens, S > 1, run(c, q, table, lens, S > 1))


@pytest.mark.parametrize("S,G,causal", [(1, 4, False), (4, 4, True), (2, 2, True), (1, 8, False), (4, 8, True)])
def test_more_than_32_parts_of_one_request(dev, S, G, causal):  # noqa: F811
    """45,003 tokens of one KV head in parts of 1024, joined 32 at a time, with scores that climb,
    fall and jump along the context, so that the maximum of the joined parts moves."""
    g = gen(80 + S)
    n, blocks = 45003, 2900
    c, table = cache([n], blocks, G, 1, g, shape_keys=lambda k: levels(k, g))
    w = c.oasis_q8_attn_workspace(1, S)
    assert w > 0
    q = steep(torch.randn(S, 1, G, 128, generator=g)).to(BF)
    out = run(c, q, table, [n], causal)
    check(c, q, table, [n], causal, out)
    whole = run(c, q, table, [n], causal, torch.empty(0, dtype=torch.uint8, device=dev))
    check(c, q, table, [n], causal, whole)
    assert torch.equal(out, run(c, q, table, [n], causal))


@pytest.mark.parametrize("S,G", [(1, 4), (4, 4)])
def test_parts_longer_than_the_least(dev, S, G):  # noqa: F811
    """So many tokens that a part is longer than it has to be: one request of 70,001 of eight heads,
    and a batch of unequal ones behind it."""
    g = gen(90)
    for lens in ([70001], [40000, 7, 0, 30001, 16000]):
        blocks = 4400
        c, table = cache(lens, blocks, 8 * G, 8, g, shape_keys=lambda k: levels(k, g))
        assert c.oasis_q8_attn_workspace(len(lens), S) > 0
        q = steep(torch.randn(S, len(lens), 8 * G, 128, generator=g)).to(HF)
        check(c, q, table, lens, True, run(c, q, table, lens, True))


# ------------------------------------------------------------------ prefix
def prefix_case(R, S, G, Hkv, plen, most, g, fp32=True, blocks_more=1, lens=None):
    lens = lens or (ragged(R, most, g) if R > 2 else [most, 0][:R])
    c, table = cache(lens, max(1, -(-most // 16)), G * Hkv, Hkv, g, fp32)
    nb = -(-plen // 16) + blocks_more
    kv = torch.randn(Hkv, 2, nb * 16, 128, generator=g)
    kv[:, 0, :plen] = levels(kv[:, 0, :plen], g)
    kv = kv.to(BF)
    ref = tuple(kv[:, i, :plen].double().cuda() for i in (0, 1))
    kv[:, :, plen:] = float("nan")                       # behind the prefix: anything
    kv[:, :, plen + 1::2] = float("inf")
    kv = kv.view(Hkv, 2, nb, 16, 128).transpose(1, 2).contiguous().cuda()
    q = steep(torch.randn(S, R, G * Hkv, 128, generator=g)).to(BF)
    return c, table, lens, kv, ref, q


def run_prefix(c, q, kv, plen, table, lens, causal):
    out = torch.full(q.shape, 5.0, dtype=FP if c.cfg.out_fp32 else q.dtype, device="cuda")
    ws = c.prefix_workspace(q.shape[1], q.shape[0], plen)
    ws.fill_(255)
    c.oasis_prefix_attn(q.cuda(), kv, plen, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), out, ws,
                        causal=causal)
    assert c.oasis_q8_sync() == 0
    return out


@pytest.mark.parametrize("R,S,G,Hkv,plen,most,fp32", [
    (40, 4, 4, 8, 4025, 40, True),      # 640 rows a head, six shares of five or six key tiles, the last one partial
    (40, 4, 4, 8, 4096, 40, False),
    (65, 2, 1, 16, 4500, 33, True),     # 130 rows: the second tile of two rows
    (20, 4, 4, 8, 8191, 100, True),     # 320 rows, the second CTA's second tile empty
    (32, 1, 4, 16, 7700, 20, True),     # 128 rows: one tile
    (3, 1, 5, 16, 7001, 30, False),     # fifteen rows
    (128, 1, 4, 8, 3333, 64, True)])
def test_prefix_of_several_key_tiles_a_share(dev, R, S, G, Hkv, plen, most, fp32):  # noqa: F811
    """The ring's stages are used again and again, and rows' maxima grow by more than 2^8 between the
    key tiles of a share (levels climb, fall and jump by tens), so outputs are rescaled."""
    g = gen(R + plen)
    c, table, lens, kv, ref, q = prefix_case(R, S, G, Hkv, plen, most, g, fp32)
    out = run_prefix(c, q, kv, plen, table, lens, S > 1)
    check(c, q, table, lens, S > 1, out, prefix=ref, p_half=2.0 ** -8)
    assert torch.equal(out, run_prefix(c, q, kv, plen, table, lens, S > 1))


@pytest.mark.parametrize("R,S,G,plen", [(1, 1, 4, 9000), (2, 4, 8, 5000), (40, 4, 4, 9000)])
def test_prefix_in_more_than_32_shares(dev, R, S, G, plen):  # noqa: F811
    """One KV head: 40 to 71 shares of one or two key tiles, joined 32 at a time."""
    g = gen(R + plen + S)
    c, table, lens, kv, ref, q = prefix_case(R, S, G, 1, plen, 50, g)
    out = run_prefix(c, q, kv, plen, table, lens, True)
    check(c, q, table, lens, True, out, prefix=ref, p_half=2.0 ** -8)


# ------------------------------------------------------------------ scales
@pytest.mark.parametrize("amp,spread,qamp", [(1.0, 6.0, 1.0), (1e-20, 3.0, 1e20), (1e18, 2.0, 1e-18), (1.0, 0.0, 30.0),
                                             (1.0, 12.0, 4.0)])
@pytest.mark.parametrize("blocks", [20, 1024])
def test_values_of_very_different_sizes(dev, amp, spread, qamp, blocks):  # noqa: F811
    """Token sizes many powers of two apart, within the derived bound of each output alone: small
    weights are kept to 2^-39 of the largest weighted one."""
    g = gen(int(spread) + blocks)
    lens = [300, 77]
    P = 40
    c = ob.Q8Cache(ob.make_q8_config(P, blocks, 8, 2, out_fp32=True))
    k = amp * torch.randn(P * 16, 2, 128, generator=g) * torch.exp2(spread * torch.randn(P * 16, 2, 1, generator=g)).clamp(max=4)
    v = amp * torch.randn(P * 16, 2, 128, generator=g) * torch.exp2(spread * torch.randn(P * 16, 2, 1, generator=g))
    v[::7] = 0
    c.oasis_q8_write(k.cuda(), v.cuda(), torch.arange(P * 16).cuda())
    table = Q.table_of(lens, P, blocks, g)
    q = (qamp * torch.randn(2, 2, 8, 128, generator=g)).to(BF)
    assert (c.oasis_q8_attn_workspace(2, 2) > 0) == (blocks == 1024)
    check(c, q, table, lens, False, run(c, q, table, lens, False))

"""Attention of trees where it could go wrong for its size or its surroundings:
waits that run out, the longest context, many requests, the ends of the
exponents' range, another handle's scratch, and the calls beside it at their
largest."""
import math

import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import BF, FP, HF, cache_of, dev, gen  # noqa: F401
from tests.test_q8_largest import random_pages
from tests.test_tree_attn import case, check, go, i32

pytestmark = pytest.mark.gpu


def test_waits_that_run_out(dev):  # noqa: F811
    """With a limit of a clock tick the kernel ends and says so; afterwards the same bits as before."""
    for R, N, lens, dtype in ((1, 5, [300], BF), (3, 64, [2000, 64, 700], BF), (2, 40, [900, 500], HF)):
        s = case(R, N, 8, 2, lens, gen(N), dtype)
        go(s)
        assert s["c"].oasis_q8_sync() == 0
        before = s["out"].clone()
        s["c"].oasis_q8_set_wait_limit(1)
        go(s)
        with pytest.raises(ob.OasisError) as e:
            s["c"].oasis_q8_sync()
        assert e.value.status == ob.OASIS_EDEVICE and "0x2" in str(e.value)
        s["c"].oasis_q8_set_wait_limit(0)
        s["out"].fill_(7.0)
        go(s)
        assert s["c"].oasis_q8_sync() == 0
        assert torch.equal(s["out"], before)


def test_longest_context(dev):  # noqa: F811
    """131072 blocks, 2097152 tokens, a chain of three nodes at their end."""
    blocks, N, G = 131072, 3, 4
    n = blocks * 16 - 5
    pages = random_pages(blocks, 1)
    c = ob.Q8Cache(ob.make_q8_config(blocks, blocks, G, 1, out_fp32=True), pages=pages)
    table = torch.randperm(blocks, generator=gen(1)).to(torch.int32)[None].cuda()
    q = (2 * torch.randn(1, N, G, 128, generator=gen(2))).to(BF).cuda()
    out = torch.empty(1, N, G, 128, device=dev)
    words = torch.tensor([[1, 3, 7]], device=dev)
    c.oasis_q8_tree_attn(q, words, table, i32([n]), out)
    assert c.oasis_q8_sync() == 0
    units = torch.empty(1, 1, blocks, 2, 16, 128, device=dev)
    c.oasis_q8_read(table, i32([n]), units)
    k, v = units[0, 0].unbind(1)
    k, v = k.reshape(-1, 128)[:n], v.reshape(-1, 128)[:n]
    scale, log2e = 1 / math.sqrt(128), math.log2(math.e)
    U = 448 * 2.0
    for i in range(N):
        m = n - N + 1 + i
        x = torch.cat([q[0, i].double() @ part.double().T for part in k[:m].split(1 << 18)], 1) * scale
        p = (x - x.max(1, keepdim=True).values).exp()
        l = p.sum(1, keepdim=True)
        o = sum(pp @ vv.double() for pp, vv in zip(p.split(1 << 18, 1), v[:m].split(1 << 18))) / l
        av = sum(pp @ vv.double().abs() for pp, vv in zip(p.split(1 << 18, 1), v[:m].split(1 << 18))) / l
        top = k[:m].abs().max().item() * q[0, i].double().abs() @ torch.ones(128, dtype=torch.float64, device=dev)
        A = (top * scale * log2e)[:, None]
        # As in the definition's bound; and sums of up to 2^10 terms a share, 2^8 shares, each fp32.
        e = 2.0 ** -11 + math.log(2) * (501 * 2.0 ** -23 + 2.0 ** -19 * 128) * A + 2.0 ** -20 + 2 * 2.0 ** -13
        bound = 2 * e * av + (m * 2.0 ** -32 + 2.0 ** -39) * U + 1e-30
        off = (out[0, i].double() - o).abs()
        assert (off <= bound).all(), (off / bound).max()
        assert off.max() < 0.02                          # (the bound is wide; this is two roundings of weights)


def test_many_requests(dev):  # noqa: F811
    """More requests than a warp, and than a CTA has threads, some without nodes, some without tokens."""
    g = gen(3)
    R, N = 1100, 2
    lens = [int(torch.randint(0, 40, (1,), generator=g)) for _ in range(R)]
    sizes = [min(r % 4, n) for r, n in enumerate(lens)]
    s = case(R, N, 2, 1, lens, g, sizes=sizes, fp32=True)
    lens[700] = s["lens"][700] = 0
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)


@pytest.mark.parametrize("R", [31, 32, 33, 64, 65])
def test_requests_around_a_warp(dev, R):  # noqa: F811
    s = case(R, 3, 2, 2, [3 + 37 * (r % 5) for r in range(R)], gen(R))
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)


@pytest.mark.parametrize("up", [-125, -100, 60, 110])
def test_queries_at_the_ends_of_the_range(dev, up):  # noqa: F811
    """Queries of 2^up against keys of 2^-up (as far as exponents go) have the scores of common ones."""
    s = case(1, 6, 4, 2, [150], gen(4), fp32=True, amp=1.0)
    down = min(max(-up, -100), 110)
    q = s["q"].double()
    s["q"] = (q * 2.0 ** up).to(BF)
    s["pages"][..., 4096:4112] = (s["pages"][..., 4096:4112].astype(np.int64) + down).clip(1, 245).astype(np.uint8)
    s["c"].pages.copy_(torch.from_numpy(s["pages"]))
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)
    assert torch.isfinite(s["out"]).all()


def test_scratch(dev):  # noqa: F811
    """Scratch of the caller's: the same bits as with the class's own, whatever was in it; too little is
    refused; bytes past the size asked for are left alone."""
    s = case(2, 20, 8, 2, [900, 300], gen(5))
    go(s)
    want = s["out"].clone()
    need = s["c"].oasis_q8_tree_workspace(2, 20)
    assert need > 0
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device=dev)
    s["out"].zero_()
    go(s, workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(s["out"], want) and (ws[need:] == 255).all()
    s["out"].zero_()
    go(s, workspace=ws[:need])                            # a used one
    assert torch.equal(s["out"], want)
    with pytest.raises((ob.OasisError, ValueError)):
        go(s, workspace=ws[:need - 256])


def test_sides_of_a_step_at_once(dev):  # noqa: F811
    """Append into one handle's pages while another's trees are attended, each on a stream of its own."""
    a, b = case(4, 30, 8, 2, [700, 900, 40, 1500], gen(6)), case(1, 4, 8, 2, [90], gen(7))
    go(a)
    want = a["out"].clone()
    g = gen(8)
    n = 1000
    c = cache_of(70, 70, 8, 2)
    plain = cache_of(70, 70, 8, 2)
    k, v, q = (torch.randn(n, h, 128, generator=g).to(BF).cuda() for h in (2, 2, 8))
    slots = torch.randperm(70 * 16, generator=g)[:n].cuda()
    pos = torch.arange(n).cuda()
    rope = ob.make_rope(64)
    q_out, q_one = torch.empty_like(q), torch.empty_like(q)
    plain.oasis_q8_append(rope, q, k, v, pos, slots, q_one)
    x = (a["q"].cuda(), T.signed(a["words"]).cuda(), a["table"].cuda(), i32(a["lens"]))
    outs = [torch.empty_like(a["out"]) for _ in range(6)]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for o in outs:
        with torch.cuda.stream(one):
            a["c"].oasis_q8_tree_attn(*x, o)
        with torch.cuda.stream(two):
            c.oasis_q8_append(rope, q, k, v, pos, slots, q_out)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert torch.equal(q_out, q_one) and torch.equal(c.pages, plain.pages)
    assert a["c"].oasis_q8_sync() == 0 and c.oasis_q8_sync() == 0
    go(b)
    check(b)


def test_append_of_many_tokens(dev):  # noqa: F811
    """A prompt's 70001 tokens, in order and turned from far positions, as in two halves."""
    n, H = 70001, 2
    blocks = -(-n // 16)
    one, two = cache_of(blocks, blocks, 4, H), cache_of(blocks, blocks, 4, H)
    k, v = (torch.randn(n, H, 128, generator=gen(9)).to(HF).cuda() for _ in range(2))
    pos = (torch.arange(n) + (1 << 31)).cuda()
    slots = torch.arange(n).cuda()
    rope = ob.make_rope(128)
    one.oasis_q8_append(rope, None, k, v, pos, slots, None)
    h = 33333
    two.oasis_q8_append(rope, None, k[:h], v[:h], pos[:h], slots[:h], None)
    two.oasis_q8_append(rope, None, k[h:], v[h:], pos[h:], slots[h:], None)
    assert one.oasis_q8_sync() == 0 and two.oasis_q8_sync() == 0
    assert torch.equal(one.pages, two.pages)


def test_logprobs_of_the_longest_rows(dev):  # noqa: F811
    """2^20 entries a row, far apart in memory, one that is all -inf but two; and 70000 short rows."""
    V, stride = 1 << 20, (1 << 20) + 24
    flat = torch.empty(5 * stride, dtype=BF, device=dev)
    x = flat.as_strided((5, V), (stride, 1))
    x.copy_(3 * torch.randn(5, V, generator=gen(10)))
    x[3] = -math.inf
    x[3, 77], x[3, V - 1] = 1.0, 2.0
    tok = i32([5, V - 1, 0, 77, 1000])
    lp, en = torch.empty(2, 5, device=dev)
    ids, top = torch.empty(5, 32, dtype=torch.int32, device=dev), torch.empty(5, 32, device=dev)
    ob.oasis_token_logprobs(x, tok, logprobs=lp, entropy=en, top_ids=ids, top_logprobs=top)
    y = x.double()
    want = y.log_softmax(1)
    p = want.exp()
    H = -(p * want.masked_fill(p == 0, 0.0)).sum(1)
    # Sums of up to 2^10 fp32 terms a thread, and 2^5 of those joined: 2^-13 relative.
    assert (lp.double() - want.gather(1, tok.long()[:, None])[:, 0]).abs().max() < 2 ** -12
    assert (en.double() - H).abs().max() < 2 ** -12 * (1 + H.max())
    assert torch.equal(ids[3, :2].cpu(), torch.tensor([V - 1, 77], dtype=torch.int32))
    for r in (0, 1, 2, 4):
        key = y[r].cpu().numpy()
        order = np.lexsort((np.arange(V), -key))[:32]
        assert ids[r].tolist() == order.tolist()
    rows = 70000
    z = torch.randn(rows, 40, generator=gen(11)).cuda()
    lp, ids, top = torch.empty(rows, device=dev), torch.empty(rows, 3, dtype=torch.int32, device=dev), torch.empty(rows, 3, device=dev)
    tok = torch.randint(0, 40, (rows,), generator=gen(12)).int().cuda()
    ob.oasis_token_logprobs(z, tok, logprobs=lp, top_ids=ids, top_logprobs=top)
    want = z.double().log_softmax(1)
    assert (lp.double() - want.gather(1, tok.long()[:, None])[:, 0]).abs().max() < 2 ** -18
    assert torch.equal(ids.long(), want.topk(3).indices)

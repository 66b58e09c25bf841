"""Attention of trees of drafted tokens on the GPU against the 64-bit
definition, within derived bounds."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import BF, FP, HF, cache_of, dev, fill, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def case(R, N, Hq, Hkv, lens, g, dtype=BF, sizes=None, fp32=False, amp=2.0, spread=1.0, extra=0, words=None, **kw):
    """A cache with random pages, queries, and random trees."""
    blocks = max(1, max(-(-n // 16) for n in lens)) + extra
    P = sum(-(-max(n, 0) // 16) for n in lens) + 2
    c = cache_of(P, blocks, Hq, Hkv, out_fp32=fp32, **kw)
    pages = fill(c, g, spread)
    table = Q.table_of(lens, P, blocks, g)
    q = (amp * torch.randn(R, N, Hq, 128, generator=g)).to(dtype)
    if words is None:
        words = [T.words_of(T.random_tree(N, g)) for _ in range(R)]
    out = torch.full(q.shape, 7.0, dtype=FP if fp32 else dtype, device="cuda")
    return dict(c=c, pages=pages, table=table, q=q, words=words, out=out, lens=lens, sizes=sizes)


def go(s, **kw):
    s["c"].oasis_q8_tree_attn(s["q"].cuda(), T.signed(s["words"]).cuda(), s["table"].cuda(), i32(s["lens"]), s["out"],
                              tree_size=None if s["sizes"] is None else i32(s["sizes"]), **kw)


def check(s, scale=None):
    o, bound, node = T.attention(s["q"], s["words"], s["sizes"], s["pages"], s["table"], s["lens"], scale, s["out"].dtype)
    got = s["out"].double().cpu().numpy()
    assert (got[~node] == 7.0).all()                     # rows past a tree: as they were
    off = np.abs(got - o)[node]
    assert (off <= bound[node]).all(), (off / bound[node]).max()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("R,N,Hq,Hkv,lens", [
    (1, 1, 1, 1, [1]), (1, 1, 8, 1, [129]), (2, 2, 2, 2, [2, 40]), (1, 16, 32, 8, [700]),
    (3, 5, 24, 8, [300, 0, 21]), (2, 64, 4, 1, [64, 500]), (2, 13, 28, 4, [127, 142]),
    (1, 33, 4, 1, [1000]), (2, 64, 8, 1, [65, 400]), (2, 32, 8, 2, [128, 256]), (1, 64, 10, 2, [333])])
def test_tree(dev, dtype, R, N, Hq, Hkv, lens):  # noqa: F811
    s = case(R, N, Hq, Hkv, lens, gen(N * 10 + R), dtype)
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)


@pytest.mark.parametrize("before", [0, 1, 63, 64, 100, 112, 127, 128, 129, 240, 255, 256])
@pytest.mark.parametrize("N", [3, 20])
def test_where_the_tree_begins(dev, before, N):  # noqa: F811
    """Around the ends of blocks and of tiles of tokens."""
    s = case(1, N, 4, 2, [before + N], gen(before), fp32=True)
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)


@pytest.mark.parametrize("G,N", [(1, 40), (2, 64), (3, 43), (4, 32), (4, 33), (5, 51), (8, 16), (8, 33), (8, 64), (7, 37)])
def test_heads_and_rows(dev, G, N):  # noqa: F811
    """Rows a KV head up to and past 128 and 256, fp32 outputs, several heads."""
    s = case(2, N, 3 * G, 3, [N + 200, N + 31], gen(G * 64 + N), fp32=True)
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)


@pytest.mark.parametrize("seed", range(6))
def test_ragged(dev, seed):  # noqa: F811
    """Lengths and tree sizes of all kinds side by side, a table wider than needed."""
    g = gen(50 + seed)
    r = lambda n: int(torch.randint(0, n, (1,), generator=g))  # noqa: E731
    R, N, G, Hkv = 1 + r(9), 1 + r(40), 1 + r(6), 1 + r(3)
    sizes = [r(N + 3) - 1 for _ in range(R)]
    lens = [0 if r(5) == 0 else max(min(max(n, 0), N), 1) + [0, r(30), r(1500)][r(3)] for n in sizes]
    s = case(R, N, G * Hkv, Hkv, lens, g, [BF, HF][seed % 2], sizes=sizes, fp32=seed > 3, extra=r(40))
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)


def test_words_of_any_kind(dev):  # noqa: F811
    """Nothing seen, everything seen, later nodes seen, bits past the tree, with and without a
    context before the tree."""
    N = 11
    some = (1 << 64) - 1
    words = [[0, some, 1 << 10, some ^ 1, 1 << 11, 1 << 63, 5, 1, 2, 0x7FF, 0x400]] * 2
    s = case(2, N, 8, 2, [N, N + 40], gen(1), words=words)
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    check(s)
    assert (s["out"][0, 0] == 0).all() and (s["out"][0, 4] == 0).all() and (s["out"][0, 5] == 0).all()


def test_masked_nodes_may_hold_anything(dev):  # noqa: F811
    """NaN keys and values of nodes that a query does not see, and bytes behind the last token,
    leave its output as it is; those that see them get NaN (a value's in its own dims alone)."""
    N, n = 9, 150
    s = case(1, N, 8, 2, [n + N], gen(2), extra=2, words=[[1 << i for i in range(N)]])
    pages = s["pages"]
    go(s)
    clean = s["out"].clone()

    def at(node):
        t = n + node
        return int(s["table"][0, t // 16]), t % 16
    p, j = at(3)
    pages[p][:, Q.key_at(j, np.arange(128))] = 0x7F       # node 3: its whole key
    p, j = at(5)
    pages[p][0, Q.value_at(j, 17)] = 0xFF                 # node 5: one dim of a value of head 0
    p, _ = at(N - 1)
    for j in range((n + N) % 16, 16):                     # behind the end
        pages[p][:, Q.key_at(j, np.arange(128))] = 0x7F
        pages[p][:, Q.value_at(j, np.arange(128))] = 0x7F
        pages[p][:, [4096 + j, 4112 + j]] = 255
    s["c"].pages.copy_(torch.from_numpy(pages))
    go(s)
    nan = torch.isnan(s["out"][0].float()).cpu()
    want = torch.zeros_like(nan)
    want[3] = True
    want[5, :4, 17] = True
    assert torch.equal(nan, want)
    same = ~want
    assert torch.equal(s["out"][0].cpu()[same], clean[0].cpu()[same])
    assert s["c"].oasis_q8_sync() == 0


def test_context_nan_reaches_all(dev):  # noqa: F811
    s = case(1, 4, 4, 1, [200], gen(3))
    p = int(s["table"][0, 3])
    s["pages"][p][0, Q.value_at(5, 9)] = 0x7F
    s["c"].pages.copy_(torch.from_numpy(s["pages"]))
    go(s)
    nan = torch.isnan(s["out"][0].float()).cpu()
    assert nan[:, :, 9].all() and int(nan.sum()) == 16


@pytest.mark.parametrize("dtype", [BF, HF])
def test_query_with_nan_or_infinity(dev, dtype):  # noqa: F811
    """Its own rows give NaN, no other."""
    s = case(1, 6, 8, 2, [90], gen(4), dtype)
    go(s)
    clean = s["out"].clone()
    s["q"][0, 2, 3, 5], s["q"][0, 4, 7, 100] = float("nan"), float("inf")
    go(s)
    want = torch.zeros(6, 8, dtype=torch.bool)
    want[2, 3] = want[4, 7] = True
    assert torch.equal(torch.isnan(s["out"][0].float()).all(-1).cpu(), want)
    assert torch.equal(s["out"][0][~want], clean[0][~want])


@pytest.mark.parametrize("spread", [12.0, 30.0])
def test_scales_far_apart(dev, spread):  # noqa: F811
    """Keys and values whose tokens' sizes differ by many powers of two; scores stay small."""
    s = case(1, 12, 8, 2, [400], gen(5), fp32=True, amp=2.0 ** -20, spread=spread / 3)
    go(s)
    check(s)


def test_large_and_tiny_queries(dev):  # noqa: F811
    for amp, fp32 in ((30.0, True), (2.0 ** -14, False), (0.0, True)):
        s = case(1, 10, 8, 2, [300], gen(6), HF, amp=amp, fp32=fp32)
        go(s)
        check(s)
    s = case(1, 10, 8, 2, [300], gen(6), BF, amp=2.0 ** 60, fp32=True, softmax_scale=2.0 ** -62)
    go(s)
    check(s, 2.0 ** -62)


def test_bad_pages_and_lengths(dev):  # noqa: F811
    """A bad block is left out; a length below the tree's or past the table raises the bit."""
    s = case(2, 5, 4, 2, [100, 60], gen(7))
    s["table"][0, 2], s["table"][1, 3] = -1, 10000
    go(s)
    with pytest.raises(ob.OasisError, match="0x1"):
        s["c"].oasis_q8_sync()
    check(s)
    s = case(3, 5, 4, 2, [100, 4, 0], gen(8))
    go(s)
    with pytest.raises(ob.OasisError, match="0x1"):
        s["c"].oasis_q8_sync()
    check(s)
    assert (s["out"][1:] == 0).all()
    s["lens"] = [10 ** 9, 80, -7]
    s["table"][:] = s["table"][0]
    go(s)
    with pytest.raises(ob.OasisError, match="0x1"):
        s["c"].oasis_q8_sync()
    assert (s["out"][2] == 0).all()


def test_streams_and_graphs(dev):  # noqa: F811
    """Two calls on two streams, captured and replayed over new inputs: the same bits as one by one."""
    a, b = case(2, 12, 8, 2, [900, 40], gen(9)), case(3, 64, 8, 2, [64, 300, 5000], gen(10))
    t = [(s["q"].cuda(), T.signed(s["words"]).cuda(), s["table"].cuda(), i32(s["lens"])) for s in (a, b)]
    want = []
    for s, x in zip((a, b), t):
        s["c"].oasis_q8_tree_attn(*x, s["out"])
        want.append(s["out"].clone())
        s["out"].zero_()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=one):
        two.wait_stream(one)
        a["c"].oasis_q8_tree_attn(*t[0], a["out"], stream=one)
        with torch.cuda.stream(two):
            b["c"].oasis_q8_tree_attn(*t[1], b["out"], stream=two)
        one.wait_stream(two)
    for k in range(3):
        if k == 2:
            for x in t:
                x[0].mul_(-1)
        g.replay()
        torch.cuda.synchronize()
        if k < 2:
            assert torch.equal(a["out"], want[0]) and torch.equal(b["out"], want[1])
    got = a["out"].clone(), b["out"].clone()
    for s, x in zip((a, b), t):
        s["c"].oasis_q8_tree_attn(*x, s["out"])
    assert torch.equal(a["out"], got[0]) and torch.equal(b["out"], got[1])
    assert a["c"].oasis_q8_sync() == 0 and b["c"].oasis_q8_sync() == 0


def test_back_to_back(dev):  # noqa: F811
    """Forty calls of several sizes without a wait between, beside the attention over a shared prefix
    (both take tensor memory): the same bits as one by one."""
    cases = [case(R, N, 8, 2, lens, gen(20 + N)) for R, N, lens in ((1, 8, [600]), (4, 50, [80, 2000, 50, 900]), (2, 30, [30, 31]))]
    t = [(s["q"].cuda(), T.signed(s["words"]).cuda(), s["table"].cuda(), i32(s["lens"])) for s in cases]
    want = []
    for s, x in zip(cases, t):
        s["c"].oasis_q8_tree_attn(*x, s["out"])
        torch.cuda.synchronize()
        want.append(s["out"].clone())
    c = cases[0]["c"]
    kv = torch.randn(2, 64, 2, 16, 128, device=dev).to(BF)
    q, po = torch.randn(2, 1, 8, 128, device=dev).to(BF), torch.empty(2, 1, 8, 128, dtype=BF, device=dev)
    ws = c.prefix_workspace(1, 2, 1000)
    outs = []
    for _ in range(40):
        for s, x in zip(cases, t):
            o = torch.empty_like(s["out"])
            s["c"].oasis_q8_tree_attn(*x, o)
            outs.append(o)
        c.oasis_prefix_attn(q, kv, 1000, t[0][2], t[0][3], po, ws)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 3])
    assert c.oasis_q8_sync() == 0


def test_refusals(dev):  # noqa: F811
    s = case(2, 5, 4, 2, [100, 60], gen(12))
    good = dict(q=s["q"].cuda(), tree=T.signed(s["words"]).cuda(), page_table=s["table"].cuda(), seq_len=i32([100, 60]),
                out=s["out"])
    c = s["c"]
    c.oasis_q8_tree_attn(**good)
    z = torch.zeros
    for change in (dict(q=good["q"].float()), dict(q=good["q"][:, :4]), dict(q=good["q"].transpose(0, 1)),
                   dict(out=good["out"].float()), dict(tree=good["tree"].int()), dict(tree=good["tree"][:, :4]),
                   dict(tree=good["tree"].cpu()), dict(page_table=good["page_table"][:, :2]),
                   dict(seq_len=good["seq_len"].long()), dict(tree_size=i32([1])), dict(q=good["q"][0])):
        with pytest.raises(ValueError):
            c.oasis_q8_tree_attn(**{**good, **change})
    big = z(2, 65, 4, 128, dtype=BF, device=dev)
    with pytest.raises(ob.OasisError, match="num_nodes"):
        c.oasis_q8_tree_attn(**{**good, "q": big, "out": big.clone(), "tree": z(2, 65, dtype=torch.int64, device=dev)})
    none = z(2, 0, 4, 128, dtype=BF, device=dev)
    with pytest.raises(ob.OasisError, match="num_nodes"):
        c.oasis_q8_tree_attn(**{**good, "q": none, "out": none.clone(), "tree": z(2, 0, dtype=torch.int64, device=dev)})
    n = c.oasis_q8_tree_workspace(2, 5)
    if n:
        with pytest.raises(ob.OasisError, match="workspace"):
            c.oasis_q8_tree_attn(**good, workspace=z(n - 256, dtype=torch.uint8, device=dev))
    with pytest.raises(ob.OasisError):
        c.oasis_q8_tree_workspace(2, 65)
    empty = z(0, 5, 4, 128, dtype=BF, device=dev)
    c.oasis_q8_tree_attn(empty, z(0, 5, dtype=torch.int64, device=dev), z(0, c.cfg.max_blocks, dtype=torch.int32, device=dev),
                         z(0, dtype=torch.int32, device=dev), empty.clone())
    assert c.oasis_q8_sync() == 0


def test_chain_is_causal_attention(dev):  # noqa: F811
    """A tree that is a chain gives what oasis_q8_attn gives its causal queries, within both bounds."""
    g = gen(30)
    s = case(3, 4, 8, 2, [500, 4, 77], g, fp32=True, words=[[1, 3, 7, 15]] * 3)
    go(s)
    q = s["q"].transpose(0, 1).contiguous().cuda()
    out = torch.empty(4, 3, 8, 128, device=dev)
    s["c"].oasis_q8_attn(q, s["table"].cuda(), i32(s["lens"]), out, causal=True)
    o, b = Q.attention(s["q"].transpose(0, 1), s["pages"], s["table"], s["lens"], True, out=FP)
    _, b2, _ = T.attention(s["q"], s["words"], None, s["pages"], s["table"], s["lens"], out=FP)
    off = (out.transpose(0, 1) - s["out"]).abs().double().cpu().numpy()
    assert (off <= b.transpose(1, 0, 2, 3) + b2).all()

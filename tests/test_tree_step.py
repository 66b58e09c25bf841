"""A run of the tree step's operators together: append, attend, look at the
logits, keep a path, and go on decoding; captured and not."""
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import BF, FP, cache_of, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def test_tree_steps_leave_what_plain_steps_would(dev):  # noqa: F811
    """Three steps of trees: after each, the pages' tokens are those of the paths that the
    logits chose, as if they had been appended one by one, and the attention of the kept nodes
    is the causal attention over them."""
    g = gen(1)
    R, N, Hq, Hkv, V = 3, 12, 8, 2, 500
    c, plain = cache_of(40, 8, Hq, Hkv, out_fp32=True), cache_of(40, 8, Hq, Hkv, out_fp32=True)
    table = torch.randperm(40, generator=g)[:R * 8].view(R, 8).to(torch.int32)
    d_table = table.cuda()
    rope = ob.make_rope(128, base=10000.0)
    lens = torch.tensor([14, 0, 30])
    for r in range(R):                                            # the context so far
        n = int(lens[r])
        if n:
            k, v = torch.randn(2, n, Hkv, 128, generator=g).to(BF).cuda()
            for x in (c, plain):
                x.oasis_q8_append(rope, None, k, v, torch.arange(n).cuda(), Q.slots_of(table, r, 0, n).cuda(), None)
    for step in range(3):
        parents = [T.random_tree(N, g) for _ in range(R)]
        depth = torch.zeros(R, N, dtype=torch.int64)
        for r in range(R):
            for i, p in enumerate(parents[r]):
                depth[r, i] = depth[r, p] + 1 if p >= 0 else 0
        q, k, v = (torch.randn(R * N, h, 128, generator=g).to(BF).cuda() for h in (Hq, Hkv, Hkv))
        pos = (lens[:, None] + depth).flatten()
        slots = torch.cat([Q.slots_of(table, r, int(lens[r]), int(lens[r]) + N) for r in range(R)])
        turned = torch.empty_like(q)
        c.oasis_q8_append(rope, q, k, v, pos.cuda(), slots.cuda(), turned)
        seq = i32(lens + N)
        out = torch.empty(R, N, Hq, 128, device=dev)
        c.oasis_q8_tree_attn(turned.view(R, N, Hq, 128), ob.tree_words(parents).cuda(), d_table, seq, out)
        # a made-up model: every node's logits choose one of its children, where it has any
        logits = torch.randn(R, N + 1, V, generator=g)
        drafted = torch.stack([torch.randperm(V, generator=g)[:N] for _ in range(R)])
        for r in range(R):
            for i in range(-1, N):
                kids = [j for j in range(N) if parents[r][j] == i]
                if kids:
                    logits[r, i + 1, drafted[r, kids[step % len(kids)]]] = 20.0
        ids = torch.empty(R, N + 1, 1, dtype=torch.int32, device=dev)
        ob.oasis_token_logprobs(logits.cuda(), top_ids=ids, top_logprobs=torch.empty(R, N + 1, 1, device=dev))
        best = ids.squeeze(-1).cpu()
        paths = []
        for r in range(R):
            path, at = [], -1
            while True:
                nxt = [j for j in range(N) if parents[r][j] == at and int(drafted[r, j]) == int(best[r, at + 1])]
                if not nxt:
                    break
                path.append(nxt[0])
                at = nxt[0]
            assert path
            paths.append(path)
        c.oasis_q8_keep(d_table, seq, i32([p + [0] * (N - len(p)) for p in paths]), i32([len(p) for p in paths]), N)
        # one by one: the same path appended as consecutive tokens
        for r, p in enumerate(paths):
            rows = r * N + torch.tensor(p)
            n = int(lens[r])
            one = torch.empty(len(p), Hq, 128, dtype=BF, device=dev)
            plain.oasis_q8_append(rope, q[rows], k[rows], v[rows], (n + torch.arange(len(p))).cuda(),
                                  Q.slots_of(table, r, n, n + len(p)).cuda(), one)
            assert torch.equal(one, turned[rows])
            lens[r] = n + len(p)
        a, b = (torch.zeros(R, Hkv, 8, 2, 16, 128, device=dev) for _ in range(2))
        c.oasis_q8_read(d_table, i32(lens), a)
        plain.oasis_q8_read(d_table, i32(lens), b)
        assert torch.equal(a, b) and a.abs().sum() > 0
        # the kept nodes' outputs are causal attention over the kept tokens
        pages = c.pages.cpu().numpy()
        for r, p in enumerate(paths):
            for i, node in enumerate(p[:3]):
                L = int(lens[r]) - len(p) + i + 1
                one = turned[r * N + node].view(1, 1, Hq, 128).cpu()
                o, bound = Q.attention(one, pages, table[r:r + 1], [L], False, out=FP)
                off = (out[r, node].double().cpu().numpy() - o[0, 0])
                _, wide, _ = T.attention(one, [[1]], None, pages, table[r:r + 1], [L], out=FP)
                assert (abs(off) <= bound[0, 0] + wide[0, 0]).all()
    assert c.oasis_q8_sync() == 0 and plain.oasis_q8_sync() == 0


def test_a_captured_step(dev):  # noqa: F811
    """All four calls in one graph, replayed with new inputs, against the calls one by one."""
    g = gen(2)
    R, N, Hq, Hkv, V = 2, 20, 8, 2, 3000
    one, two = cache_of(30, 12, Hq, Hkv), cache_of(30, 12, Hq, Hkv)
    fill = torch.randint(0, 120, one.pages.shape, generator=g, dtype=torch.uint8).cuda()
    table = torch.randperm(30, generator=g)[:24].view(R, 12).to(torch.int32).cuda()
    words = ob.tree_words([T.random_tree(N, g) for _ in range(R)]).cuda()
    lens, rope = i32([150, 41]), ob.make_rope(64, sections=(8, 12, 12))
    qkv = torch.empty(R * N, Hq + 2 * Hkv, 128, dtype=BF, device=dev)
    pos, slots = torch.empty(3, R * N, dtype=torch.int64, device=dev), torch.cat(
        [Q.slots_of(table.cpu(), r, int(lens[r]) - N, int(lens[r])) for r in range(R)]).cuda()
    logits, tokens = torch.empty(R, N, V, device=dev), torch.zeros(R, N, dtype=torch.int32, device=dev)
    nodes, keep = i32([[0, 2, 5], [1, 7, 19]]), i32([3, 2])

    def step(c, o):
        c.oasis_q8_append(rope, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], pos, slots, o["turned"])
        c.oasis_q8_tree_attn(o["turned"].view(R, N, Hq, 128), words, table, lens, o["out"])
        ob.oasis_token_logprobs(logits, tokens, o["lp"], o["H"], o["ids"], o["top"])
        c.oasis_q8_keep(table, lens, nodes, keep, N)
    new = lambda: dict(turned=torch.empty(R * N, Hq, 128, dtype=BF, device=dev), out=torch.empty(R, N, Hq, 128, dtype=BF, device=dev),  # noqa: E731,E501
                       lp=torch.empty(R, N, device=dev), H=torch.empty(R, N, device=dev),
                       ids=torch.empty(R, N, 6, dtype=torch.int32, device=dev), top=torch.empty(R, N, 6, device=dev))
    a, b = new(), new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(one, a)
    for k in range(3):
        for c in (one, two):
            c.pages.copy_(fill)
        qkv.normal_()
        pos.random_(0, 10 ** 5)
        logits.normal_()
        tokens.random_(-1, V)
        for x, y in zip(a.values(), b.values()):
            x.zero_(), y.zero_()
        graph.replay()
        step(two, b)
        torch.cuda.synchronize()
        for n in a:
            assert torch.equal(a[n], b[n]), n
        assert torch.equal(one.pages, two.pages)
    assert one.oasis_q8_sync() == 0 and two.oasis_q8_sync() == 0

"""A tree step over a pool of pages that begins 16 bytes past a 32-byte
boundary, and with as many requests as a call takes."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import BF, HF, FP, cache_of, dev, gen  # noqa: F401
from tests.test_tree_attn import case, check, go, i32

pytestmark = pytest.mark.gpu


def shifted(cfg, by):
    """A handle whose pages begin `by` bytes into a larger buffer, and that buffer."""
    n = ob.oasis_q8_query_sizes(cfg).pages_bytes
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    first = -buf.data_ptr() % 256 + by
    pages = buf[first:first + n].view(cfg.num_pages, cfg.num_kv_heads, Q.UNIT)
    return ob.Q8Cache(cfg, pages=pages), buf, first, n


@pytest.mark.parametrize("by", [16, 48, 112])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_step_over_shifted_pages(dev, by, dtype):  # noqa: F811
    """Append, attend, keep: the same bytes and bits as over an aligned pool, and nothing around it."""
    R, N, Hq, Hkv, blocks = 3, 20, 8, 2, 8
    g = gen(by)
    cfg = ob.make_q8_config(R * blocks, blocks, Hq, Hkv)
    a = ob.Q8Cache(cfg)
    b, buf, first, n = shifted(cfg, by)
    a.pages.copy_(torch.randint(0, 127, a.pages.shape, generator=g, dtype=torch.uint8))
    b.pages.copy_(a.pages)
    table = torch.randperm(R * blocks, generator=g).to(torch.int32).view(R, blocks)
    rope = ob.make_rope(64)
    x = torch.randn(R * 128, Hq + 2 * Hkv, 128, generator=g).to(dtype).cuda()
    t = torch.arange(128)
    slots = (table[:, t // 16].long() * 16 + t % 16).flatten().cuda()
    words = T.signed([T.words_of(T.random_tree(N, g)) for _ in range(R)]).cuda()
    lens, nodes = i32([100, 128, 61]), i32([[0, 3, 7, 19], [5, 4, 3, 2], [0, 1, 2, 18]])
    outs = []
    for c in (a, b):
        q = torch.empty(R * 128, Hq, 128, dtype=dtype, device=dev)
        c.oasis_q8_append(rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], torch.arange(R * 128).cuda(), slots, q)
        out = torch.empty(R, N, Hq, 128, dtype=dtype, device=dev)
        c.oasis_q8_tree_attn(q[:R * N].view(R, N, Hq, 128), words, table.cuda(), lens, out)
        c.oasis_q8_keep(table.cuda(), lens, nodes, i32([4, 4, 3]), num_nodes=N)
        assert c.oasis_q8_sync() == 0
        outs.append((q, out))
    assert torch.isfinite(outs[0][1].float()).all()
    assert all(torch.equal(p, q) for p, q in zip(*outs)) and torch.equal(a.pages, b.pages)
    assert (buf[:first] == 0xA5).all() and (buf[first + n:] == 0xA5).all()


def test_the_most_requests(dev):  # noqa: F811
    """65535 requests of one or two nodes over 1 to 24 tokens, some empty: each as in a call of its own
    neighbours, and a sample against the definition."""
    R, N, g = 65535, 2, gen(5)
    P = 4096
    c = cache_of(P, 2, 2, 1, out_fp32=True)
    k, v = (torch.randn(P * 16, 1, 128, generator=g).to(BF).cuda() for _ in range(2))
    c.oasis_q8_write(k, v, torch.arange(P * 16).cuda())
    table = torch.randint(0, P, (R, 2), generator=g, dtype=torch.int32)
    lens = torch.randint(2, 25, (R,), generator=g, dtype=torch.int32)
    lens[::97] = 0
    sizes = torch.randint(0, 3, (R,), generator=g, dtype=torch.int32)
    q = torch.randn(R, N, 2, 128, generator=g).to(BF)
    words = torch.tensor([[1, 3]]).repeat(R, 1)
    words[::5, 1] = 2
    dv = (q.cuda(), words.cuda(), table.cuda(), lens.cuda())
    out = torch.full((R, N, 2, 128), 7.0, device=dev)
    c.oasis_q8_tree_attn(*dv, out, tree_size=sizes.cuda())
    assert c.oasis_q8_sync() == 0
    for lo in (0, 20000, 65000):                          # other shares of the work: other roundings of sums alone
        part = torch.full((535, N, 2, 128), 7.0, device=dev)
        s = slice(lo, lo + 535)
        c.oasis_q8_tree_attn(*(x[s] for x in dv), part, tree_size=sizes[s].cuda())
        assert (part - out[s]).abs().max() < 2.0 ** -9
    pages = c.pages.cpu().numpy()
    some = [0, 1, 2, 96, 97, 12345, 32767, 32768, 65533, 65534] + list(range(40000, 40060))
    o, bound, node = T.attention(q[some], words[some].tolist(), sizes[some], pages, table[some], lens[some], None, FP)
    got = out[some].double().cpu().numpy()
    assert (got[~node] == 7.0).all()
    assert (np.abs(got - o)[node] <= bound[node]).all()


def test_results_repeat(dev):  # noqa: F811
    """The same call gives the same bits, whatever runs beside it and whatever the scratch held."""
    s = case(5, 40, 8, 2, [3000, 40, 777, 129, 2000], gen(6))
    go(s)
    want = s["out"].clone()
    x = torch.randn(4096, 4096, device=dev)
    side = torch.cuda.Stream()
    for _ in range(30):
        with torch.cuda.stream(side):
            x.mul_(1.0)
        s["out"].fill_(7.0)
        go(s, workspace=torch.randint(0, 255, (s["c"].oasis_q8_tree_workspace(5, 40),), dtype=torch.uint8, device=dev))
        assert torch.equal(s["out"], want)
    check(s)

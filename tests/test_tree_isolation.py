"""Attention of trees where nodes' values are many powers of two above the
others': a row's precision is that of the tokens it sees, whatever the nodes
that it does not see hold."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _tree as T
from tests.test_q8 import BF, HF, dev, gen  # noqa: F401
from tests.test_tree_attn import case, go

pytestmark = pytest.mark.gpu


def value_exponents(s, r, node, n):
    """(page, byte) of the value exponents of one of n nodes."""
    t = s["lens"][r] - n + node
    return int(s["table"][r, t // 16]), 4112 + t % 16


def against(s, pages, rows):
    """The rows' outputs are those over `pages`, within the bound that those give."""
    o, bound, _ = T.attention(s["q"], s["words"], s["sizes"], pages, s["table"], s["lens"], None, s["out"].dtype)
    got = s["out"].double().cpu().numpy()
    for r, i in rows:
        off = np.abs(got[r, i] - o[r, i])
        assert (off <= bound[r, i]).all(), (r, i, (off / bound[r, i]).max())


def row_of(s, pages, r, i, N):
    """(o, bound) [Hq][128] of one row alone."""
    q = torch.zeros(1, N, *s["q"].shape[2:], dtype=s["q"].dtype)
    q[0, i] = s["q"][r, i]
    words = [[0] * N]
    words[0][i] = s["words"][r][i]
    o, bound, _ = T.attention(q, words, None, pages, s["table"][r:r + 1], [s["lens"][r]], None, s["out"].dtype)
    return o[0, i], bound[0, i]


@pytest.mark.parametrize("up", [-110, 1, 7, 20, 21, 22, 40, 100])
@pytest.mark.parametrize("dtype,N,G,before", [(BF, 9, 4, 150), (HF, 9, 4, 150), (BF, 64, 4, 200), (BF, 20, 2, 0), (BF, 40, 1, 100),
                                              (HF, 64, 2, 100), (BF, 64, 1, 70), (BF, 12, 4, 3000)])
def test_one_large_node(dev, up, dtype, N, G, before):  # noqa: F811
    """One node's value is 2^up of what it was; only some see it (itself and every fourth node)."""
    Hkv, big = 2, N // 2
    seen_by = [i for i in range(N) if i == big or i % 4 == 3]
    words = [sum(1 << j for j in range(N) if (j != big and (i + j) % 3 != 0) or j == i) | (int(i in seen_by) << big) for i in range(N)]
    s = case(1, N, G * Hkv, Hkv, [before + N], gen(N + before), dtype, fp32=True, spread=0.3, words=[words])
    plain = s["pages"].copy()
    page, byte = value_exponents(s, 0, big, N)
    s["pages"][page][:, byte] = np.clip(s["pages"][page][:, byte].astype(int) + up, 27, 247).astype(np.uint8)
    s["c"].pages.copy_(torch.from_numpy(s["pages"]))
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    against(s, plain, [(0, i) for i in range(N) if i not in seen_by])
    o, bound, _ = T.attention(s["q"], s["words"], None, s["pages"], s["table"], s["lens"], None, s["out"].dtype)
    off = np.abs(s["out"].double().cpu().numpy() - o)
    assert (off <= bound).all(), (off / bound).max()


@pytest.mark.parametrize("before", [0, 90, 128, 500])
def test_every_node_of_another_size(dev, before):  # noqa: F811
    """Nodes that see the context and themselves, each 2^9 of the one before: all keep their own bits."""
    N, Hkv = 24, 2
    s = case(2, N, 4 * Hkv, Hkv, [before + N, before + N], gen(before), fp32=True, spread=0.0,
             words=[[1 << i for i in range(N)], [1 << (N - 1 - i) for i in range(N)]])
    if before == 0:
        s["words"][1] = [3 << max(i - 1, 0) for i in range(N)]
    for r in range(2):
        for i in range(N):
            page, byte = value_exponents(s, r, i, N)
            s["pages"][page][:, byte] = np.clip(s["pages"][page][:, byte].astype(int) + 9 * (i - N // 2), 27, 247).astype(np.uint8)
    s["c"].pages.copy_(torch.from_numpy(s["pages"]))
    go(s)
    assert s["c"].oasis_q8_sync() == 0
    got = s["out"].double().cpu().numpy()
    for r in range(2):
        for i in range(N):                               # over pages whose other nodes have the least exponent
            pages = s["pages"].copy()
            for j in range(N):
                if not s["words"][r][i] >> j & 1:
                    page, byte = value_exponents(s, r, j, N)
                    pages[page][:, byte] = 27
            o, bound = row_of(s, pages, r, i, N)
            off = np.abs(got[r, i] - o)
            assert (off <= bound).all(), (r, i, (off / bound).max())


def test_wide_context_around_a_bad_page(dev):  # noqa: F811
    """A block that is left out makes its tile one that is looked at token by token; the context's
    values there are up to 2^60 apart."""
    s = case(2, 6, 8, 2, [400, 150], gen(17), fp32=True, amp=0.5, spread=8.0)
    s["table"][0, 3], s["table"][1, 1] = -1, 10000
    go(s)
    with pytest.raises(ob.OasisError, match="0x1"):
        s["c"].oasis_q8_sync()
    o, bound, _ = T.attention(s["q"], s["words"], None, s["pages"], s["table"], s["lens"], None, s["out"].dtype)
    off = np.abs(s["out"].double().cpu().numpy() - o)
    assert (off <= bound).all(), (off / bound).max()

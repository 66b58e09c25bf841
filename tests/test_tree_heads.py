"""Trees over very many heads: a query of a late node is more than 2^31
elements behind the first one's."""
import numpy as np
import pytest
import torch

from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import BF, HF, FP, cache_of, dev, gen  # noqa: F401
from tests.test_tree_attn import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF])
def test_queries_past_31_bits(dev, dtype):  # noqa: F811
    """64 nodes x 280000 query heads, 35000 KV heads; a few heads against the definition."""
    N, Hkv, G, n = 64, 35000, 8, 70
    g = torch.Generator(device="cuda").manual_seed(3)
    c = cache_of(6, 5, Hkv * G, Hkv)
    k, v = (torch.randn(n, Hkv, 128, generator=g, device=dev).to(BF) for _ in range(2))
    table = torch.tensor([[3, 0, 5, 1, 4]], dtype=torch.int32)
    t = torch.arange(n)
    c.oasis_q8_write(k, v, (table[0, t // 16].long() * 16 + t % 16).cuda())
    q = torch.empty(1, N, Hkv * G, 128, dtype=dtype, device=dev)
    for i in range(N):
        q[0, i] = torch.randn(Hkv * G, 128, generator=g, device=dev)
    assert (N - 1) * Hkv * G * 128 > 1 << 31
    words = [T.words_of(T.random_tree(N, gen(4)))]
    out = torch.full_like(q, 7.0)
    c.oasis_q8_tree_attn(q, T.signed(words).cuda(), table.cuda(), i32([n]), out)
    assert c.oasis_q8_sync() == 0
    for h in (0, 1, 16789, 17500, 33288, 33289, 34998, 34999):
        pages = c.pages[:, h:h + 1].cpu().numpy()
        rows = slice(h * G, (h + 1) * G)
        o, bound, _ = T.attention(q[:, :, rows].cpu(), words, None, pages, table, [n], None, dtype)
        off = np.abs(out[:, :, rows].double().cpu().numpy() - o)
        assert (off <= bound).all(), (h, (off / bound).max())

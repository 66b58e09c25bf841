"""Keeping nodes of a tree on the GPU, byte for byte."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import cache_of, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("R,N,M,Hkv,kind,seed", [
    (1, 1, 1, 1, "path", 0), (1, 16, 16, 8, "path", 1), (3, 64, 64, 2, "path", 2), (5, 33, 7, 3, "any", 3),
    (4, 64, 64, 1, "same", 4), (6, 20, 20, 4, "reversed", 5), (130, 9, 9, 2, "path", 6), (4, 64, 64, 1, "all", 7)])
@pytest.mark.parametrize("sized", [False, True])
def test_keep(dev, R, N, M, Hkv, kind, seed, sized):  # noqa: F811
    g = gen(seed)
    r = lambda n: int(torch.randint(0, n, (1,), generator=g))  # noqa: E731
    lens = [N + r(60) for _ in range(R)]
    sizes = [r(N + 3) - 1 for _ in range(R)] if sized else None
    blocks = max(-(-n // 16) for n in lens)
    c = cache_of(R * blocks + 2, blocks, Hkv, Hkv)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8))
    old = c.pages.cpu().numpy()
    table = Q.table_of(lens, R * blocks + 2, blocks, g)
    n_of = [N if sizes is None else min(max(s, 0), N) for s in sizes or [0] * R]
    if kind == "reversed":
        nodes = [[max(n - 1 - i, 0) for i in range(M)] for n in n_of]
    elif kind == "same":
        nodes = [[max(n - 1, 0)] * M for n in n_of]
    elif kind == "any":
        nodes = [[r(max(n, 1)) for _ in range(M)] for n in n_of]
    else:
        nodes = [sorted(torch.randperm(max(n, 1), generator=g)[:M].tolist()) for n in n_of]
        nodes = [x + [0] * (M - len(x)) for x in nodes]
    keep = [M if kind in ("all", "same", "reversed") else r(M + 2) - 1 for _ in range(R)]
    if kind in ("path", "all"):
        keep = [min(k, n) for k, n in zip(keep, n_of)]
    want = T.keep(old, table.numpy(), lens, sizes, N, np.array(nodes), keep)
    c.oasis_q8_keep(table.cuda(), i32(lens), i32(nodes), i32(keep), N, tree_size=i32(sizes) if sized else None)
    assert c.oasis_q8_sync() == 0
    assert np.array_equal(c.pages.cpu().numpy(), want)


def test_bad_nodes_pages_and_lengths(dev):  # noqa: F811
    """Each raises its bit; the others' moves are made."""
    g = gen(11)
    c = cache_of(10, 2, 2, 2)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8))
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32)

    def go(lens, nodes, keep, table=table):
        old = c.pages.cpu().numpy()
        want = T.keep(old, table.numpy(), lens, None, 4, np.array(nodes), keep)
        c.oasis_q8_keep(table.cuda(), i32(lens), i32(nodes), i32(keep), 4)
        with pytest.raises(ob.OasisError) as e:
            c.oasis_q8_sync()
        assert np.array_equal(c.pages.cpu().numpy(), want) and (want != old).any()
        return str(e.value)
    assert "0x4" in go([20, 18, 32], [[1, 4], [2, -1], [3, 3]], [2, 2, 2])
    bad = table.clone()
    bad[0, 1], bad[1, 0] = 10, -1
    assert "0x1" in go([18, 18, 32], [[1, 3], [2, 3], [3, 1]], [2, 2, 2], bad)
    c.oasis_q8_keep(table.cuda(), i32([0, -5, 20]), i32([[1, 2]] * 3), i32([2, 2, 0]), 4)
    assert c.oasis_q8_sync() == 0


@pytest.mark.parametrize("length", [3, 33])
def test_length_that_cannot_be(dev, length):  # noqa: F811
    """Fewer tokens than nodes, more than the table holds: nothing moves and the bit is raised."""
    c = cache_of(4, 2, 2, 2)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=gen(1), dtype=torch.uint8))
    old = c.pages.clone()
    c.oasis_q8_keep(i32([[0, 1]]), i32([length]), i32([[1, 2]]), i32([2]), 4)
    with pytest.raises(ob.OasisError, match="0x1"):
        c.oasis_q8_sync()
    assert torch.equal(c.pages, old)


def test_refusals(dev):  # noqa: F811
    c = cache_of(4, 2, 2, 2)
    good = dict(page_table=i32([[0, 1]]), seq_len=i32([20]), nodes=i32([[0, 1]]), keep=i32([2]), num_nodes=4)
    c.oasis_q8_keep(**good)
    for change in (dict(page_table=i32([[0]])), dict(nodes=i32([0, 1])), dict(keep=i32([[2]])), dict(nodes=i32([[0, 1]]).long()),
                   dict(keep=torch.tensor([2], dtype=torch.int32)), dict(tree_size=i32([1, 2])), dict(nodes=i32([[0, 1]] * 2))):
        with pytest.raises(ValueError):
            c.oasis_q8_keep(**{**good, **change})
    for change in (dict(num_nodes=0), dict(num_nodes=65), dict(nodes=torch.zeros(1, 65, dtype=torch.int32, device=dev))):
        with pytest.raises(ob.OasisError, match="EINVAL"):
            c.oasis_q8_keep(**{**good, **change})
    assert c.oasis_q8_sync() == 0

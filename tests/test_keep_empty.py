"""Keeping nodes of requests that have none: what raises and what does not."""
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests.test_keep import i32
from tests.test_q8 import cache_of, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("length,keep,raises", [(0, 2, False), (-1, 2, False), (-2 ** 31, 64, False), (1, 1, True), (3, 2, True),
                                                (3, 0, False), (3, -5, False), (33, 1, True), (33, 0, False), (2 ** 31 - 1, 1, True)])
def test_lengths(dev, length, keep, raises):  # noqa: F811
    """A length of 0 or less is an empty request; one that cannot be raises BAD_BLOCK_ID where a node is
    to be kept.  Nothing moves."""
    c = cache_of(4, 2, 2, 2)
    c.pages.copy_(torch.randint(0, 256, c.pages.shape, generator=gen(1), dtype=torch.uint8))
    old = c.pages.clone()
    c.oasis_q8_keep(i32([[0, 1]]), i32([length]), i32([[1, 2]]), i32([keep]), 4)
    if raises:
        with pytest.raises(ob.OasisError, match="0x1"):
            c.oasis_q8_sync()
    else:
        assert c.oasis_q8_sync() == 0
    assert torch.equal(c.pages, old)

"""The rotation's angle, to what oasis_q8_append promises: 2^-27 of a turn for
positions up to 2^32.

Bound.  cos and sin: 2 pi 2^-27 for the angle, and a unit in the last place of
fp32 below 1, 2^-24.  A turned entry: both times (|a| + |b|) scale, and one
rounding each of the scaled factor, the product and the sum, 3 * 2^-24."""
import math

import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _tree as T
from tests.test_q8 import cache_of, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu
ROT = 2 * math.pi * 2.0 ** -27 + 2.0 ** -24


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("positions", ["near", "far", "largest", "quarters"])
def test_angle(dev, interleaved, positions):  # noqa: F811
    n, g = 96, gen(7)
    pos = {"near": torch.arange(n), "far": torch.randint(0, 1 << 32, (n,), generator=g),
           "largest": (1 << 32) - torch.arange(n), "quarters": torch.arange(n)}[positions]
    f = [10000.0 ** (-i / 64) for i in range(64)]
    if positions == "quarters":                           # quarters and eighths of a turn, and next to them
        f = [(math.pi / 4) * (1 + s * 2.0 ** -p) for p in range(20, 52) for s in (-1, 1)]
    rope = ob.make_rope(128, frequency=f, interleaved=interleaved)
    c = cache_of(7, 7, 2, 1)
    q = torch.randn(n, 2, 128, generator=g)
    q[:, 1, :] = 0.0
    q[:, 1, 0::2 if interleaved else 1] = 1.0             # cos and sin themselves
    if not interleaved:
        q[:, 1, 64:] = 0.0
    out = torch.empty(n, 2, 128, device=dev)
    k = torch.zeros(n, 1, 128, device=dev)
    c.oasis_q8_append(rope, q.cuda(), k, k, pos.cuda(), torch.full((n,), -1).cuda(), out)
    assert c.oasis_q8_sync() == 0
    y, loose = T.rotate(q, pos, rope)
    bound = loose * ((ROT + 3 * 2.0 ** -24) / (T.ROT + 3 * 2.0 ** -24))
    off = np.abs(out.double().cpu().numpy() - y)
    assert (off <= bound).all(), (off - bound).max()

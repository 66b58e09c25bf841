"""Log probabilities of many rows of the longest kind, where one CTA of 128
threads adds up a row of 2^20 entries.

Rows of equal entries behind 256 equal peaks, one at least for each thread: a
thread's weights are then all the same number w, and the roundings of a plain
running sum of them have one sign over long stretches (7e-6 of S in all).
Bound, in units of u = 2^-24 of S: w itself 4 (the exponential) + 2.2 * 0.69 *
|y| = 17 at |y| = 10.9, nine in a group of entries, two for a running sum that
carries its rounding along, 5 + 3 where threads and warps are joined, their two
factors 5 each: 50 u = 3.0e-6, and 3 u for the logarithm: under the 2^-19 + 2^-21
of 6.5 = 5.0e-6 that is asked."""
import math

import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests.test_q8 import BF, FP, HF, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_a_peak_over_many_equal_entries(dev, dtype):  # noqa: F811
    V, rows = 1 << 20, 640
    x = torch.zeros(rows, V, dtype=dtype, device=dev)
    up = torch.linspace(6.5, 7.5, rows, device=dev).to(dtype)              # as many different weights
    x[:, :1024:4] = up[:, None]
    at = 4 * torch.randint(0, 256, (rows,), generator=gen(1)).cuda()
    lp, en, low = (torch.empty(rows, device=dev) for _ in range(3))
    ob.oasis_token_logprobs(x, at.int(), logprobs=lp, entropy=en)
    ob.oasis_token_logprobs(x, at.int() + 1, logprobs=low)
    a = up.double()
    lse = torch.log((V - 256) + 256 * a.exp())
    for got, want, depth in ((lp, a - lse, 0), (low, -lse, a)):
        off = (got.double() - want).abs() - (2.0 ** -19 + 2.0 ** -21 * want.abs() + 2.0 ** -22 * depth)
        assert off.max() <= 0, (got.double() - want).abs().max()
    # H = lse - 256 p a: both terms have the sums' errors.
    H = lse - 256 * a * (a - lse).exp()
    assert ((en.double() - H).abs() <= 2.0 ** -18 * (1 + H)).all(), (en.double() - H).abs().max()


@pytest.mark.parametrize("down", [False, True])
def test_rising_rows(dev, down):  # noqa: F811
    """A maximum that rises, or falls, a little with every entry."""
    V, rows = 1 << 20, 600
    x = torch.linspace(-9, 9, V, device=dev)
    x = (x.flip(0) if down else x).expand(rows, V).contiguous()
    lp, en = torch.empty(2, rows, device=dev)
    tok = torch.arange(rows, device=dev).int() * 1700
    ob.oasis_token_logprobs(x, tok, logprobs=lp, entropy=en)
    want = x[:1].double().log_softmax(1)[0]
    H = -(want.exp() * want).sum()
    w = want[tok.long()]
    # As above, and 20 u where the maximum is raised (some five times a factor's 5 u counts).
    assert ((lp.double() - w).abs() <= 2.0 ** -18 + 2.0 ** -21 * w.abs() + 2.0 ** -22 * 18).all(), (lp.double() - w).abs().max()
    assert ((en.double() - H).abs() <= 2.0 ** -17 * (1 + H)).all()
    assert math.isfinite(en.sum().item())

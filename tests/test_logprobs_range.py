"""Log probabilities of rows whose entries are as large as their type allows:
masks of the type's lowest value, entries near its largest, and rows that are
far from 0 throughout.

Bound: an entry's difference from the largest is one rounding (2^-24 of it),
its product with log2 e another and the constant's own 2^-26, so a weight is off
by 2^-22 + 2^-23 |y|, and what is held to as for common rows applies at any
magnitude: 2^-19 + 2^-21 of the value + 2^-22 of the difference."""
import math

import numpy as np
import pytest
import torch

from tests import _tree as T
from tests.test_logprobs import go
from tests.test_q8 import BF, FP, HF, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def check(x, tokens, k, got):
    with np.errstate(over="ignore"):
        lp, H, ids, top = (a.astype(np.float32).astype(float) if a.dtype == float else a for a in T.logprobs(x, tokens, k))

    def near(a, b, depth):
        with np.errstate(invalid="ignore"):
            ok = (a == b) | (np.abs(a - b) <= 2.0 ** -19 + 2.0 ** -21 * np.abs(b) + 2.0 ** -22 * depth)
        assert ok.all(), (a[~ok], b[~ok])
    near(got["logprobs"], lp, -lp)
    near(got["entropy"], H, 0)
    assert np.array_equal(got["top_ids"], ids)
    near(got["top_logprobs"], top, -top)


def row(kind, V, dtype, g):
    big, i = torch.finfo(dtype).max, torch.arange(V).double()
    x = 3 * torch.randn(V, generator=g, dtype=torch.float64)
    few = torch.rand(V, generator=g) < 5 / V
    few[V // 2] = True
    return {"lowest": torch.full((V,), -big, dtype=torch.float64), "largest": torch.full((V,), big, dtype=torch.float64),
            "masked": torch.where(few, x, -big), "half masked": torch.where(i % 2 == 0, x, -big),
            "one largest": torch.where(i == V // 3, big, x), "both ends": torch.where(i % 3 == 0, big, -big),
            "masks of both kinds": torch.where(few, x, torch.where(i % 2 == 0, -big, -math.inf)),
            "one finite": torch.where(i == V // 2, -big, -math.inf),
            "1e10": 1e10 + 1000 * x, "-1e10": -1e10 + 1000 * x, "-1e30": torch.full((V,), -1e30, dtype=torch.float64),
            "spread 1e30": 1e30 * x, "1e7": 1e7 + x, "-3e4": -3e4 + x, "2e9 and below": 2e9 - 1e3 * i}[kind]


KINDS = ["lowest", "largest", "masked", "half masked", "one largest", "both ends", "masks of both kinds", "one finite",
         "1e10", "-1e10", "-1e30", "spread 1e30", "1e7", "-3e4", "2e9 and below"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_large_entries(dev, kind, dtype):  # noqa: F811
    g = gen(len(kind))
    big = torch.finfo(dtype).max
    for V in (1, 7, 1000, 40003):
        x = row(kind, V, dtype, g)
        x = torch.where(x.abs() < math.inf, x.clamp(-big, big), x).to(dtype).repeat(3, 1)
        tokens = [V // 2, 0, min(V - 1, V // 3)]
        for k in (1, 20):
            check(x, tokens, k, go(x.cuda(), tokens, k))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_side_by_side(dev, dtype):  # noqa: F811
    """More rows than clusters run at once, of every kind; a wrong one must not reach its neighbours."""
    V, g = 5001, gen(4)
    big = torch.finfo(dtype).max
    x = torch.stack([row(KINDS[r % len(KINDS)], V, dtype, g) for r in range(700)])
    x = torch.where(x.abs() < math.inf, x.clamp(-big, big), x).to(dtype)
    tokens = [(r * 37) % V for r in range(700)]
    check(x, tokens, 5, go(x.cuda(), tokens, 5))


def test_infinity_beside_the_largest(dev):  # noqa: F811
    """+infinity and NaN still give NaN where the rest is at the ends of the range."""
    x = torch.full((3, 3000), -torch.finfo(FP).max)
    x[0, 5], x[1, 2999], x[2, 17] = math.inf, math.nan, torch.finfo(FP).max
    got = go(x.cuda(), [5, 5, 17], 2)
    for n in ("logprobs", "entropy", "top_logprobs"):
        assert np.isnan(got[n][:2]).all(), n
    assert got["logprobs"][2] == 0 and got["entropy"][2] == 0 and got["top_ids"][2].tolist() == [17, 0]

"""Draft verification of batches over rows of many entries, where a warp takes
segments of 1024 entries: aligned rows and rows of any alignment, with a
draft's row to subtract and with certain drafts, in all three types."""
import numpy as np
import pytest
import torch

from tests import _q8 as Q
from tests.test_verify_drafts import BF, FP, HF, dev, draw, gen, go  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("R,n,V", [(300, 1, 9001), (300, 2, 9004), (280, 3, 9216), (20, 2, 151936), (17, 1, 151939)])
def test_batches_of_long_rows(dev, dtype, R, n, V):  # noqa: F811
    """R rows of more than 152 * 16 segments together: one to eight CTAs a request."""
    assert R * -(-V // 1024) >= 152 * 16
    p, q, x, ua, us = draw(R, n, V, gen(R + V + n), dtype)
    us[:3] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5])
    ua[3], ua[4:20] = 0.0, 1.0                            # all accepted; mostly refused
    for d in (q, None):
        wt, wa = Q.verify(p, d, x, ua, us)
        tok, acc = go(p, d, x, ua, us)
        assert np.array_equal(acc, wa) and np.array_equal(tok, wt)
        assert len(set(wa.tolist())) > 1 or d is None


@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_long_rows_in_padded_and_offset_memory(dev, dtype):  # noqa: F811
    """Rows that begin at any element, with NaN between them."""
    R, n, V, pad, off = 270, 1, 9300, 5, 3
    p, q, x, ua, us = draw(R, n, V, gen(8), dtype)

    def place(t):
        m = t.shape[1]
        buf = torch.full((R * m * (V + pad) + off,), float("nan"), dtype=dtype, device="cuda")
        v = buf.as_strided((R, m, V), (m * (V + pad), V + pad, 1), off)
        v.copy_(t)
        return v
    wt, wa = Q.verify(p, q, x, ua, us)
    tok, acc = go(place(p), place(q), x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_long_rows_with_little_left(dev, dtype):  # noqa: F811
    """Equal rows but for one entry in the last segment, equal rows altogether (p itself is drawn
    from), rows of zeros, and a threshold on the border between two segments."""
    R, V = 300, 9100
    p, _, x, ua, us = draw(R, 1, V, gen(9), dtype)
    q = p[:, :1].clone()
    ua[:] = 1.0                                            # refused: u q < p does not hold
    p[0:100, 0, V - 1] += 0.25
    x[0:100] = 5                                           # (not the entry that is left)
    p[100:110] = 0
    q[110:120] = 0                                         # the draft was impossible: accepted
    p[120:130, 0], q[120:130, 0] = 0, 1
    p[120:130, 0, 1023], p[120:130, 0, 1024], p[120:130, 0, 9000] = 0.5, 0.25, 0.25
    q[120:130, 0, 1023:1025], q[120:130, 0, 9000] = 0, 0
    x[120:130] = 7
    us[120:130] = torch.tensor([0.0, 0.25, 0.49, 0.5, 0.51, 0.74, 0.75, 0.76, 0.99, 1.0 - 2.0 ** -24])
    wt, wa = Q.verify(p, q, x, ua, us)
    assert (wt[0:100, 0] == V - 1).all() and (wt[100:110, 0] == -1).all() and set(wt[120:130, 0]) == {1023, 1024, 9000}
    tok, acc = go(p, q, x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)

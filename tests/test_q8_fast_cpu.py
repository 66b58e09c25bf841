"""The vectorised 64-bit attention of the tests against the plain one."""
import numpy as np
import pytest
import torch

from tests import _q8 as Q
from tests import _q8_fast as F


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("plen", [0, 50])
def test_same_outputs_and_bounds(causal, plen):
    g = torch.Generator()
    g.manual_seed(3)
    lens, H, Hq, S = [40, 0, 2, 17], 2, 6, 4
    P = 8
    x = torch.randn(2, P * 16, H, 128, generator=g) * torch.exp2(2 * torch.randn(2, P * 16, H, 1, generator=g))
    pages = np.zeros((P, H, Q.UNIT), dtype=np.uint8)
    Q.write(pages, x[0], x[1], torch.arange(P * 16))
    table = Q.table_of(lens, P, 4, g)
    q = torch.randn(S, 4, Hq, 128, generator=g).to(torch.bfloat16)
    pre = torch.randn(2, H, plen, 128, generator=g, dtype=torch.float64)
    a = dict(prefix=tuple(pre), p_half=2.0 ** -8) if plen else {}
    b = dict(prefix=tuple(pre.numpy()), p_half=2.0 ** -8) if plen else {}
    o, e = F.attention(q, torch.from_numpy(pages), table, lens, causal, torch.bfloat16, **a)
    o2, e2 = Q.attention(q, pages, table.numpy(), lens, causal, out=torch.bfloat16, **b)
    assert np.allclose(o, o2, rtol=1e-12, atol=1e-13)
    assert np.allclose(e, e2, rtol=1e-9, atol=0)

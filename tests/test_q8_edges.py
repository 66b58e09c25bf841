"""The 8-bit cache where its documentation's limits lie: the least alignment
of what is lent, and the ends of the number range."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests.test_q8 import BF, FP, HF, attend, close, dev, gen, prefix_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("off", [16, 48, 32])
def test_pages_lent_at_any_multiple_of_sixteen_bytes(dev, dtype, off):  # noqa: F811
    """Pages are 16-byte aligned and no more (a slice of a larger arena): whole blocks, parts of
    blocks and single tokens are written where they belong, read back and attended to, and the
    bytes on both sides of the pool stay."""
    g = gen(60 + off)
    P, H, T = 24, 8, 330
    arena = torch.full((off + P * H * Q.UNIT + 64,), 0xA5, dtype=torch.uint8, device=dev)
    pages = arena[off:off + P * H * Q.UNIT].view(P, H, Q.UNIT)
    assert pages.data_ptr() % 64 == off
    c = ob.Q8Cache(ob.make_q8_config(P, 12, 16, H, out_fp32=True), pages=pages)
    slots = torch.cat([torch.arange(16, 16 + 300), torch.arange(340, 340 + 27), torch.tensor([2, 9, 383])])
    assert len(slots) == T and T * H * 2 >= 152 * 32      # sixteen tokens a warp
    x = (torch.randn(T, 2 * H, 128, generator=g) * torch.exp2(3 * torch.randn(T, 2 * H, 1, generator=g))).to(dtype)
    want = np.full(pages.shape, 0xA5, dtype=np.uint8)
    Q.write(want, x[:, :H], x[:, H:], slots)
    k, v = x.cuda()[:, :H], x.cuda()[:, H:]
    c.oasis_q8_write(k, v, slots.cuda())
    assert c.oasis_q8_sync() == 0
    assert np.array_equal(pages.cpu().numpy(), want)
    pages.fill_(0xA5)
    for i in range(0, T, 30):                             # and a token a warp
        c.oasis_q8_write(k[i:i + 30], v[i:i + 30], slots[i:i + 30].cuda())
    assert c.oasis_q8_sync() == 0
    assert np.array_equal(pages.cpu().numpy(), want)
    lens = [130, 77]
    table = Q.table_of(lens, 15, 12, g) + 1               # whole blocks of the first run
    q = torch.randn(2, 2, 16, 128, generator=g).to(BF)
    out = attend(c, q.cuda(), table, lens, True)
    back = torch.zeros(2, H, 12, 2, 16, 128, dtype=FP, device=dev)
    c.oasis_q8_read(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), back)
    assert c.oasis_q8_sync() == 0
    o, b = Q.attention(q, want, table.numpy(), lens, True, out=FP)
    close(out, o, b)
    for r, n in enumerate(lens):
        kk, vv, _ = Q.tokens(want, table[r].tolist(), n)
        got = back[r].permute(0, 2, 1, 3, 4).reshape(H, 2, -1, 128)[:, :, :n].double().cpu().numpy()
        assert np.array_equal(got[:, 0], kk) and np.array_equal(got[:, 1], vv)
    assert (arena[:off] == 0xA5).all() and (arena[off + P * H * Q.UNIT:] == 0xA5).all()

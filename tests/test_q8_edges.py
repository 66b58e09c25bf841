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


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_the_largest_values_come_back_finite(dev, dtype):  # noqa: F811
    """A row's largest value can round up to the power of two past the type's range: it is read, and
    attended to, as the type's largest value, within 2^-4 of what was written (half a step of e4m3;
    the type's own rounding of the output is less than the 2^-8 that the largest value is nearer)."""
    top = torch.finfo(dtype).max
    x = torch.zeros(32, 1, 128, dtype=torch.float64)
    x[:, 0, 0] = torch.linspace(0.5, 1.0, 32, dtype=torch.float64) * top
    x[:, 0, 1] = -x[:, 0, 0].flip(0)
    x[:, 0, 2] = top
    x[7, 0, 3], x[8, 0, 3], x[9, 0, 4] = float("inf"), float("-inf"), float("nan")
    x = x.to(dtype)
    c = ob.Q8Cache(ob.make_q8_config(2, 1, 2, 1, out_fp32=dtype == FP))
    k = torch.zeros_like(x)
    k[:, 0, :] = 1.0
    c.oasis_q8_write(k.cuda(), x.cuda(), torch.arange(32).cuda())
    out = torch.zeros(2, 1, 1, 2, 16, 128, dtype=dtype, device=dev)
    c.oasis_q8_read(torch.tensor([[0], [1]], dtype=torch.int32).cuda(), torch.full((2,), 16, dtype=torch.int32).cuda(), out)
    back = out[:, 0, 0, 1].reshape(32, 128).double().cpu()
    want = x[:, 0].double()

    def near(got, want):
        fin = torch.isfinite(want)
        assert torch.isfinite(got[fin]).all() and torch.isnan(got[torch.isnan(want)]).all()
        assert ((got - want).abs()[fin] <= 2.0 ** -4 * want.abs()[fin]).all()
    near(back, want)
    # infinities were written as the code of 448 * 2^e, past the type's range: 114688 in fp16
    far = float("inf") if dtype == HF else top
    assert back[7, 3] == far and back[8, 3] == -far
    # one token a request: its value is the output
    qt = HF if dtype == HF else BF
    for t in range(0, 32, 16):
        pages = torch.full((2, 1), t // 16, dtype=torch.int32)
        q = torch.ones(1, 2, 2, 128, dtype=qt).cuda()
        got = attend(c, q, pages, [1, 0], False).double().cpu()
        near(got[0, 0, 0].view(1, -1), want[t:t + 1])
        assert (got[0, 1] == 0).all()
    assert c.oasis_q8_sync() == 0


@pytest.mark.parametrize("lens,blocks", [([500, 33], 32), ([900], 512), ([700, 0, 3000], 1024)],
                         ids=["one CTA", "cluster", "parts"])
@pytest.mark.parametrize("S,G,fp32", [(1, 4, True), (4, 4, True), (2, 2, False)])
def test_values_whose_sum_passes_the_range(dev, lens, blocks, S, G, fp32):  # noqa: F811
    """Outputs are averages: values near the end of fp32's range give finite ones although their
    sum is not."""
    g = gen(71 + S)
    c = ob.Q8Cache(ob.make_q8_config(sum(-(-n // 16) for n in lens), blocks, 2 * G, 2, out_fp32=fp32))
    P = c.cfg.num_pages
    k = torch.randn(P * 16, 2, 128, generator=g)
    v = (2 * torch.rand(P * 16, 2, 128, generator=g) - 1) * (0.93 * 2.0 ** 127)
    v[:, :, :8] = v[:1, :, :8]                            # the same in every token
    c.oasis_q8_write(k.cuda(), v.cuda(), torch.arange(P * 16).cuda())
    pages = c.pages.cpu().numpy()
    table = Q.table_of(lens, P, blocks, g)
    q = (0.5 * torch.randn(S, len(lens), 2 * G, 128, generator=g)).to(BF)
    o, b = Q.attention(q, pages, table.numpy(), lens, True, out=FP if fp32 else BF)
    assert np.abs(o).max() < 0.97 * 2.0 ** 127
    t, m = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    out = torch.zeros(q.shape, dtype=FP if fp32 else BF, device=dev)
    n = c.oasis_q8_attn_workspace(len(lens), S)
    assert (n > 0) == (blocks == 1024)
    for ws in ([torch.empty(n, dtype=torch.uint8, device=dev)] if n else []) + [torch.empty(0, dtype=torch.uint8, device=dev)]:
        out.zero_()
        c.oasis_q8_attn(q.cuda(), t, m, out, causal=True, workspace=ws)
        close(out, o, b)
    assert c.oasis_q8_sync() == 0


def test_handles_on_the_same_pages_with_tables_of_other_widths(dev):  # noqa: F811
    """A second handle with fewer blocks a row, on the same pages: each writes what the other reads,
    and both attend within the bound over tables of their own width."""
    g = gen(91)
    lens = [100, 33, 0, 160]
    wide = ob.Q8Cache(ob.make_q8_config(40, 4096, 16, 4, out_fp32=True))
    narrow = ob.Q8Cache(ob.make_q8_config(40, 10, 16, 4, out_fp32=True), pages=wide.pages)
    k, v = torch.randn(2, 640, 4, 128, generator=g)
    wide.oasis_q8_write(k[:300].cuda(), v[:300].cuda(), torch.arange(300).cuda())
    narrow.oasis_q8_write(k[300:].cuda(), v[300:].cuda(), torch.arange(300, 640).cuda())
    t = Q.table_of(lens, 40, 10, g)
    t_wide = torch.full((4, 4096), -1, dtype=torch.int32)
    t_wide[:, :10] = t
    q = torch.randn(2, 4, 16, 128, generator=g).to(BF)
    o, b = Q.attention(q, wide.pages.cpu().numpy(), t.numpy(), lens, True, out=FP)
    close(attend(wide, q.cuda(), t_wide, lens, True), o, b)
    close(attend(narrow, q.cuda(), t, lens, True), o, b)
    m = torch.tensor(lens, dtype=torch.int32).cuda()
    a, c = (torch.zeros(4, 4, 10, 2, 16, 128, dtype=BF, device=dev) for _ in range(2))
    wide.oasis_q8_read(t_wide.cuda(), m, a)
    narrow.oasis_q8_read(t.cuda(), m, c)
    assert wide.oasis_q8_sync() == 0 and narrow.oasis_q8_sync() == 0
    assert torch.equal(a, c)


def test_fp16_rounds_wider_values_as_ever(dev):  # noqa: F811
    """Values of a wider type past fp16's range are read, and attended to, as fp16 rounds them."""
    x = torch.zeros(16, 1, 128)
    x[0, 0, :8] = torch.tensor([1e6, -1e6, 65536.0, -65536.0, 73728.0, 3e38, 40000.0, 65504.0])
    c = ob.Q8Cache(ob.make_q8_config(1, 1, 1, 1))
    c.oasis_q8_write(torch.ones_like(x).cuda(), x.cuda(), torch.arange(16).cuda())
    x[0, 0, 5] = 0
    y = x.clone()
    c2 = ob.Q8Cache(ob.make_q8_config(1, 1, 1, 1))
    c2.oasis_q8_write(torch.ones_like(y).cuda(), y.cuda(), torch.arange(16).cuda())
    for h in (c, c2):
        t, m = torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
        wide, half = (torch.zeros(1, 1, 1, 2, 16, 128, dtype=d, device=dev) for d in (FP, HF))
        h.oasis_q8_read(t, m, wide)
        h.oasis_q8_read(t, m, half)
        v = wide[0, 0, 0, 1, 0].cpu()
        want = torch.where(v.abs() == 65536, v.sign() * 65504, v).to(HF)
        assert torch.equal(half[0, 0, 0, 1, 0].cpu(), want) and torch.isinf(want).any()
        q = torch.ones(1, 1, 1, 128, dtype=HF, device=dev)
        out = torch.zeros_like(q)
        h.oasis_q8_attn(q, t, m, out)
        assert torch.equal(out[0, 0, 0].cpu(), want)
        assert h.oasis_q8_sync() == 0

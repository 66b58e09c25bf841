"""The 8-bit paged cache on the GPU against the 64-bit definitions: writing
and reading exactly, attention within derived bounds, device errors, streams,
graphs, and a speculative decode loop through all the calls."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    return torch.device("cuda", 0)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def cache_of(num_pages, max_blocks, Hq, Hkv, **kw):
    return ob.Q8Cache(ob.make_q8_config(num_pages, max_blocks, Hq, Hkv, **kw))


def fill(c, g, spread=2.0, amp=1.0):
    """Random pages: every slot written through the library; returns them as numpy."""
    P, H = c.cfg.num_pages, c.cfg.num_kv_heads
    k, v = (amp * torch.randn(P * 16, H, 128, generator=g) *
            torch.exp2(spread * torch.randn(P * 16, H, 1, generator=g)) for _ in range(2))
    c.oasis_q8_write(k.cuda(), v.cuda(), torch.arange(P * 16).cuda())
    c.oasis_q8_sync()
    return c.pages.cpu().numpy()


# ---------------------------------------------------------------- write
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("T,Hkv,mode", [(1, 1, "random"), (16, 2, "block"), (17, 3, "block"),
                                        (50, 8, "offset"), (161, 2, "block"), (200, 1, "random"),
                                        (96, 4, "reversed"), (64, 2, "holes")])
def test_write(dev, dtype, T, Hkv, mode):
    g = gen(T * 7 + Hkv)
    P = T // 16 + 4
    c = cache_of(P, 1, Hkv, Hkv)
    old = torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8)
    c.pages.copy_(old)
    x = torch.randn(T, 2 * Hkv + 1, 128, generator=g) * torch.exp2(3 * torch.randn(T, 2 * Hkv + 1, 1, generator=g))
    x[:, :, 5] *= (torch.rand(T, 2 * Hkv + 1, generator=g) < 0.3)
    x = x.to(dtype)
    k, v = x.cuda()[:, :Hkv], x.cuda()[:, Hkv + 1:]      # slices of a wider projection
    if mode == "block":
        slots = torch.arange(T) + 16
    elif mode == "offset":
        slots = torch.arange(T) + 5
    elif mode == "reversed":
        slots = torch.arange(T).flip(0) + 16
    else:
        slots = torch.randperm(P * 16, generator=g)[:T]
    if mode == "holes":
        slots = torch.arange(T) + 16
        slots[torch.rand(T, generator=g) < 0.3] = -1
    want = old.numpy().copy()
    Q.write(want, x[:, :Hkv], x[:, Hkv + 1:], slots)
    c.oasis_q8_write(k, v, slots.cuda())
    c.oasis_q8_sync()
    assert np.array_equal(c.pages.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("seed", range(6))
def test_write_mixed_runs(dev, dtype, seed):
    """Runs of any length from anywhere in a block, single tokens, whole blocks across the places
    where a warp's tokens end, holes, and slots past the pool: 700 and more tokens of 8 heads."""
    g = gen(100 + seed)
    r = lambda n: int(torch.randint(0, n, (1,), generator=g))  # noqa: E731
    P, at, slots = 260, 0, []
    while len(slots) < 700 + seed:
        at += r(20)                                   # where the next run begins
        n = [1, 1 + r(5), 16, 15, 17, 1 + r(60), 16 * (1 + r(4))][r(7)]
        if r(3) == 0:
            at = -(-at // 16) * 16
        slots += range(at, at + n)
        at += n
        if r(4) == 0:
            slots += [-1] * (1 + r(3))
    order = list(range(len(slots)))
    if seed % 2:                                      # whole runs in another order
        cut = sorted(r(len(slots)) for _ in range(6))
        parts = [order[a:b] for a, b in zip([0] + cut, cut + [len(order)])]
        order = [i for k in torch.randperm(len(parts), generator=g).tolist() for i in parts[k]]
    slots = torch.tensor([slots[i] for i in order])
    slots = torch.where(slots >= P * 16, torch.full_like(slots, -1), slots)
    T, H = len(slots), 8
    c = cache_of(P, 1, H, H)
    old = torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8)
    c.pages.copy_(old)
    x = (torch.randn(T, H, 128, generator=g) * torch.exp2(3 * torch.randn(T, H, 1, generator=g))).to(dtype)
    if seed == 2:                                     # values that do not set a scale
        x[::7, :, 3], x[::11, ::2, 9] = float("inf"), float("nan")
    y = x.flip(0).contiguous()
    want = old.numpy().copy()
    free = Q.write(want, x, y, slots)
    c.oasis_q8_write(x.cuda(), y.cuda(), slots.cuda())
    assert c.oasis_q8_sync() == 0
    got = c.pages.cpu().numpy()
    assert np.array_equal(got[~free], want[~free]) and (got[free] & 127 == 127).all()
    if seed == 0:                                     # the last run past the pool: a bit, the rest written
        slots[-40:] = torch.arange(40) + P * 16 - 8
        c.pages.copy_(old)
        want = old.numpy().copy()
        Q.write(want, x, y, slots)
        c.oasis_q8_write(x.cuda(), y.cuda(), slots.cuda())
        with pytest.raises(ob.OasisError):
            c.oasis_q8_sync()
        assert np.array_equal(c.pages.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_write_special_values(dev, dtype):
    rows = [[0.0], [-0.0], [float("inf")], [float("-inf"), 2.0], [float("nan"), -3.0],
            [float("nan"), float("inf"), 448.0], [torch.finfo(dtype).max], [torch.finfo(dtype).tiny],
            [1e-44], [448.0, 1.0625], [464.0, 1.1875], [448.5], [-57344.0, 3e-5], [1.0, -1.0]]
    x = torch.zeros(32, 1, 128)
    for t, r in enumerate(rows):
        x[t, 0, 3:3 + len(r)] = torch.tensor(r)
    x[20:] = torch.randn(12, 1, 128, generator=gen(0)) * 1e-6
    x = x.to(dtype)
    c = cache_of(2, 1, 1, 1)
    want = np.zeros((2, 1, Q.UNIT), dtype=np.uint8)
    free = Q.write(want, x, x.flip(0), torch.arange(32))
    c.oasis_q8_write(x.cuda(), x.flip(0).contiguous().cuda(), torch.arange(32).cuda())
    c.oasis_q8_sync()
    got = c.pages.cpu().numpy()
    assert np.array_equal(got[~free], want[~free])
    assert (got[free] & 127 == 127).all()


def test_write_bad_slots_raise_a_bit(dev):
    c = cache_of(4, 1, 2, 2)
    x = torch.randn(5, 2, 128, generator=gen(1), dtype=FP)
    for slots in (torch.tensor([0, 64, 2, -1, 3]), torch.tensor([0, 1 << 40, 2, -1, 3])):
        want = np.zeros((4, 2, Q.UNIT), dtype=np.uint8)
        Q.write(want, x, x, slots)
        c.pages.zero_()
        c.oasis_q8_write(x.cuda(), x.cuda(), slots.cuda())
        with pytest.raises(ob.OasisError) as e:
            c.oasis_q8_sync()
        assert e.value.status == ob.OASIS_EDEVICE and "0x4" in str(e.value)
        assert c.oasis_q8_sync() == 0
        assert np.array_equal(c.pages.cpu().numpy(), want)


def test_write_nothing_and_broadcast(dev):
    c = cache_of(4, 1, 2, 2)
    e = torch.empty(0, 2, 128, dtype=BF, device=dev)
    c.oasis_q8_write(e, e, torch.empty(0, dtype=torch.int64, device=dev))
    x = torch.randn(1, 2, 128, generator=gen(2), dtype=FP)
    b = x.cuda().expand(40, 2, 128)
    c.oasis_q8_write(b, b, torch.arange(40).cuda())
    c.oasis_q8_sync()
    want = np.zeros((4, 2, Q.UNIT), dtype=np.uint8)
    Q.write(want, x.expand(40, 2, 128), x.expand(40, 2, 128), torch.arange(40))
    assert np.array_equal(c.pages.cpu().numpy(), want)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("lens,Hkv", [([1], 1), ([16, 0, 17], 2), ([100, 33, 15, 64], 8), ([0], 3)])
def test_read(dev, dtype, lens, Hkv):
    g = gen(sum(lens) + Hkv)
    nb = max(1, max(-(-n // 16) for n in lens))
    c = cache_of(sum(-(-n // 16) for n in lens) + 2, nb + 1, Hkv, Hkv)
    pages = fill(c, g)
    table = Q.table_of(lens, c.cfg.num_pages, nb + 1, g)
    out = torch.full((len(lens), Hkv, nb, 2, 16, 128), 7.0, dtype=dtype, device=dev)
    c.oasis_q8_read(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), out)
    c.oasis_q8_sync()
    want = torch.full(out.shape, 7.0, dtype=torch.float64)
    for r, n in enumerate(lens):
        k, v, _ = Q.tokens(pages, table[r].tolist(), n)
        for t in range(n):
            want[r, :, t // 16, 0, t % 16] = torch.from_numpy(k[:, t])
            want[r, :, t // 16, 1, t % 16] = torch.from_numpy(v[:, t])
    if dtype != HF:      # four significant bits and an exponent: exact
        assert torch.equal(out.double().cpu(), want)
    assert torch.equal(out.cpu(), want.float().to(dtype))


def test_read_gives_back_values_that_fit(dev):
    """Values of four significant bits close to their row's maximum survive unchanged."""
    g = gen(3)
    x = (torch.randint(8, 16, (48, 2, 128), generator=g) * 2.0 ** torch.randint(-3, 4, (48, 2, 128), generator=g)).to(BF)
    x *= (torch.randint(0, 2, x.shape, generator=g) * 2 - 1).to(BF)
    c = cache_of(3, 3, 2, 2)
    c.oasis_q8_write(x.cuda(), x.cuda(), torch.arange(48).cuda())
    out = torch.zeros(1, 2, 3, 2, 16, 128, dtype=BF, device=dev)
    c.oasis_q8_read(torch.arange(3, dtype=torch.int32).view(1, 3).cuda(),
                    torch.tensor([48], dtype=torch.int32).cuda(), out)
    c.oasis_q8_sync()
    want = x.view(3, 16, 2, 128).permute(2, 0, 1, 3)
    assert torch.equal(out[0, :, :, 0].cpu(), want) and torch.equal(out[0, :, :, 1].cpu(), want)


def test_read_bad_table_and_length(dev):
    c = cache_of(6, 3, 2, 2)
    pages = fill(c, gen(4))
    table = torch.tensor([[0, 6, 2], [1, -1, 3], [4, 5, 0]], dtype=torch.int32)
    lens = torch.tensor([40, 40, 70], dtype=torch.int32)      # 70 > 3 * 16
    out = torch.full((3, 2, 3, 2, 16, 128), 9.0, dtype=FP, device=dev)
    c.oasis_q8_read(table.cuda(), lens.cuda(), out)
    with pytest.raises(ob.OasisError) as e:
        c.oasis_q8_sync()
    assert "0x1" in str(e.value)
    got = out.cpu()
    assert (got[0, :, 1] == 9).all() and (got[1, :, 1] == 9).all()
    assert (got[0, :, 2, :, 8:] == 9).all()
    k, v, at = Q.tokens(pages, table[2].tolist(), 48)
    assert np.array_equal(got[2, :, :, 0].reshape(2, 48, 128).double().numpy(), k)
    # a shorter output than the contexts: what fits is written, the bit is raised
    small = torch.full((3, 2, 1, 2, 16, 128), 9.0, dtype=FP, device=dev)
    c.oasis_q8_read(torch.zeros_like(table).cuda(), torch.tensor([16, 17, 3], dtype=torch.int32).cuda(), small)
    with pytest.raises(ob.OasisError):
        c.oasis_q8_sync()
    k, v, _ = Q.tokens(pages, [0], 16)
    for r, m in ((0, 16), (1, 16), (2, 3)):
        assert np.array_equal(small[r, :, 0, 0, :m].double().cpu().numpy(), k[:, :m])
        assert np.array_equal(small[r, :, 0, 1, :m].double().cpu().numpy(), v[:, :m])
    assert (small[2, :, 0, :, 3:] == 9).all()


# ------------------------------------------------------------- attention
def attend(c, q, table, lens, causal, pages=None, prefix=None, plen=0, ws=None, stream=None):
    out = torch.full(q.shape, 5.0, dtype=FP if c.cfg.out_fp32 else q.dtype, device=q.device)
    lens = torch.as_tensor(lens, dtype=torch.int32).cuda()
    if prefix is None:
        c.oasis_q8_attn(q, table.cuda(), lens, out, causal=causal, stream=stream)
    else:
        ws = c.prefix_workspace(q.shape[1], q.shape[0], plen) if ws is None else ws
        c.oasis_prefix_attn(q, prefix, plen, table.cuda(), lens, out, ws, causal=causal, stream=stream)
    return out


def close(out, o, bound):
    d = np.abs(out.double().cpu().numpy() - o)
    worst = float((d / np.maximum(bound, 1e-30)).max()) if d.size else 0.0
    assert np.isfinite(d).all() and (d <= bound).all(), f"{worst:.2f} times the bound"


LENS = [[1], [0], [16, 0, 1], [15, 17, 31, 33], [63, 64, 65, 0, 128], [200, 5], [1000], [3, 2, 1, 0]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("S,causal", [(1, False), (2, False), (4, True), (3, True)])
@pytest.mark.parametrize("Hq,Hkv,dtype,fp32", [(8, 2, BF, True), (3, 3, HF, False), (8, 1, BF, False),
                                               (5, 1, HF, True), (28, 4, BF, True)])
def test_attention(dev, lens, S, causal, Hq, Hkv, dtype, fp32):
    g = gen(sum(lens) * 31 + S)
    nb = max(1, max(-(-n // 16) for n in lens))
    c = cache_of(sum(-(-n // 16) for n in lens) + 3, nb + 2, Hq, Hkv, out_fp32=fp32)
    pages = fill(c, g, spread=1.0)
    table = Q.table_of(lens, c.cfg.num_pages, nb + 2, g)
    # what no query sees may be anything: NaN codes, odd exponents
    for r, n in enumerate(lens):
        if n % 16:
            u = pages[int(table[r, n // 16])]
            for j in range(n % 16, 16):
                u[:, Q.key_at(j, np.arange(128))] = 0x7F
                u[:, Q.value_at(j, np.arange(128))] = 0xFF
                u[:, [4096 + j, 4112 + j]] = 255 if j & 1 else 0
    c.pages.copy_(torch.from_numpy(pages))
    q = (2 * torch.randn(S, len(lens), Hq, 128, generator=g)).to(dtype)
    out = attend(c, q.cuda(), table, lens, causal)
    c.oasis_q8_sync()
    o, b = Q.attention(q, pages, table.numpy(), lens, causal, out=out.dtype)
    close(out, o, b)


@pytest.mark.parametrize("amp,spread,qamp", [(1.0, 6.0, 1.0), (1e-20, 3.0, 1e20), (1e18, 2.0, 1e-18), (1.0, 0.0, 30.0)])
def test_attention_scales(dev, amp, spread, qamp):
    """Token sizes many powers of two apart, tiny and huge keys, sharp softmax."""
    g = gen(11)
    lens = [300, 77]
    c = cache_of(40, 20, 8, 2, out_fp32=True)
    P = 40 * 16
    k = amp * torch.randn(P, 2, 128, generator=g) * torch.exp2(spread * torch.randn(P, 2, 1, generator=g)).clamp(max=4)
    v = amp * torch.randn(P, 2, 128, generator=g) * torch.exp2(spread * torch.randn(P, 2, 1, generator=g))
    v[::7] = 0
    c.oasis_q8_write(k.cuda(), v.cuda(), torch.arange(P).cuda())
    c.oasis_q8_sync()
    pages = c.pages.cpu().numpy()
    table = Q.table_of(lens, 40, 20, g)
    q = (qamp * torch.randn(2, 2, 8, 128, generator=g)).to(BF)
    out = attend(c, q.cuda(), table, lens, False)
    c.oasis_q8_sync()
    o, b = Q.attention(q, pages, table.numpy(), lens, False, out=out.dtype)
    # weights under 2^-28 of the largest weighted value may be rounded away
    b += 2.0 ** -27 * np.abs(o).max() * 8 + 2.0 ** -24 * amp * 0
    close(out, o, b)


def test_attention_scale_argument_and_zero_queries(dev):
    g = gen(12)
    c = cache_of(10, 4, 8, 2, out_fp32=True, softmax_scale=0.3)
    pages = fill(c, g, spread=0.5)
    table = Q.table_of([50, 33], 10, 4, g)
    q = torch.randn(1, 2, 8, 128, generator=g).to(BF)
    q[0, 1] = 0                                   # uniform weights
    out = attend(c, q.cuda(), table, [50, 33], False)
    c.oasis_q8_sync()
    o, b = Q.attention(q, pages, table.numpy(), [50, 33], False, scale=0.3, out=FP)
    close(out, o, b)
    none = torch.empty(1, 0, 8, 128, dtype=BF, device=dev)
    c.oasis_q8_attn(none, table[:0].cuda(), torch.empty(0, dtype=torch.int32, device=dev), torch.empty_like(none, dtype=FP))


def test_attention_nan_reaches_only_its_head(dev):
    g = gen(13)
    c = cache_of(10, 4, 4, 2, out_fp32=True)
    pages = fill(c, g).copy()
    table = Q.table_of([40], 10, 4, g)
    pages[int(table[0, 1]), 1, Q.value_at(3, 9)] = 0x7F   # a NaN value, head 1, token 19, dim 9
    c.pages.copy_(torch.from_numpy(pages))
    q = torch.randn(1, 1, 4, 128, generator=g).to(BF)
    out = attend(c, q.cuda(), table, [40], False).cpu()
    assert torch.isfinite(out[0, 0, :2]).all()
    bad = torch.isnan(out[0, 0, 2:])
    assert bad[:, 9].all() and bad.sum() == 2


@pytest.mark.parametrize("n", [7, 64, 67, 130])
def test_attention_nan_in_a_drafted_token_stays_with_its_readers(dev, n):
    """A NaN value of the last token is seen by the last query alone, one of the token before by
    two; NaN keys likewise."""
    g = gen(17 + n)
    c = cache_of(12, 10, 5, 1, out_fp32=True)
    pages = fill(c, g).copy()
    table = Q.table_of([n], 12, 10, g)
    clean = pages.copy()
    at = lambda t: (int(table[0, t // 16]), 0)  # noqa: E731
    pages[at(n - 1)][Q.value_at((n - 1) % 16, 100)] = 0xFF
    pages[at(n - 2)][Q.value_at((n - 2) % 16, 9)] = 0x7F
    c.pages.copy_(torch.from_numpy(pages))
    q = torch.randn(4, 1, 5, 128, generator=g).to(BF)
    out = attend(c, q.cuda(), table, [n], True).cpu()
    bad = torch.isnan(out[:, 0])
    want = torch.zeros_like(bad)
    want[3, :, 100] = True
    want[2:, :, 9] = True
    assert torch.equal(bad, want)
    o, b = Q.attention(q, clean, table.numpy(), [n], True, out=FP)
    close(torch.where(torch.isnan(out), torch.from_numpy(o).float(), out), o, b)
    pages = clean.copy()
    pages[at(n - 1)][Q.key_at((n - 1) % 16, 5)] = 0x7F
    c.pages.copy_(torch.from_numpy(pages))
    out = attend(c, q.cuda(), table, [n], True).cpu()
    assert torch.isnan(out[3]).all() and torch.isfinite(out[:3]).all()


def test_attention_nan_query_gives_nan(dev):
    g = gen(18)
    c = cache_of(12, 10, 4, 1, out_fp32=True)
    fill(c, g)
    table = Q.table_of([70], 12, 10, g)
    q = torch.randn(2, 1, 4, 128, generator=g).to(BF)
    q[1, 0, 2, 77] = float("nan")
    out = attend(c, q.cuda(), table, [70], False).cpu()
    assert torch.isnan(out[1, 0, 2]).all() and int(torch.isnan(out).sum()) == 128


def test_attention_bad_pages_are_left_out(dev):
    g = gen(14)
    c = cache_of(20, 8, 4, 2, out_fp32=True)
    pages = fill(c, g, spread=0.5)
    lens = [100, 40, 500]                              # 500 > 8 * 16
    table = Q.table_of([100, 40, 64], 20, 8, g)
    table[0, 2], table[0, 6], table[1, 0] = -1, 20, 1 << 30
    table[1, 1:3] = -7                                 # nothing of request 1 is there
    table[2, 4:] = table[2, :4]
    q = torch.randn(2, 3, 4, 128, generator=g).to(BF)
    out = attend(c, q.cuda(), table, lens, False)
    with pytest.raises(ob.OasisError) as e:
        c.oasis_q8_sync()
    assert "0x1" in str(e.value)
    o, b = Q.attention(q, pages, table.numpy(), [100, 40, 128], False, out=FP)
    close(out, o, b)
    assert (out[:, 1] == 0).all()


def test_attention_past_32_bit_offsets(dev):
    """Pages that lie past 4 GiB of the pool."""
    g = gen(15)
    P, H = 150000, 8
    assert P * H * Q.UNIT > (1 << 32) + (1 << 28)
    c = ob.Q8Cache(ob.make_q8_config(P, 8, 16, H, out_fp32=True),
                   pages=torch.empty(P, H, Q.UNIT, dtype=torch.uint8, device=dev))
    lens = [100, 128]
    table = Q.table_of(lens, P, 8, g, low=P - 16)
    table[0, 0] = 0
    slots = torch.cat([Q.slots_of(table, r, 0, n) for r, n in enumerate(lens)])
    k, v = torch.randn(2, len(slots), H, 128, generator=g).to(BF)
    c.oasis_q8_write(k.cuda(), v.cuda(), slots.cuda())
    ids = torch.unique(table[table >= 0]).long()
    small = np.zeros((len(ids), H, Q.UNIT), dtype=np.uint8)
    re = torch.full((P,), -1)
    re[ids] = torch.arange(len(ids))
    Q.write(small, k, v, re[slots // 16] * 16 + slots % 16)
    t2 = np.where(table.numpy() >= 0, re[table.clamp(min=0).long()].numpy(), -1)
    q = torch.randn(2, 2, 16, 128, generator=g).to(BF)
    out = attend(c, q.cuda(), table, lens, True)
    back = torch.zeros(2, H, 8, 2, 16, 128, dtype=FP, device=dev)
    c.oasis_q8_read(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), back)
    c.oasis_q8_sync()
    o, b = Q.attention(q, small, t2, lens, True, out=FP)
    close(out, o, b)
    kk, _, _ = Q.tokens(small, t2[1], 128)
    assert np.array_equal(back[1, :, :, 0].reshape(H, 128, 128).double().cpu().numpy(), kk)


def test_long_context_many_splits(dev):
    """One request, 20,000 tokens: the axis is split and joined; the order of the parts is fixed."""
    g = gen(16)
    n = 20011
    c = cache_of(n // 16 + 3, n // 16 + 2, 8, 2, out_fp32=True)
    P = c.cfg.num_pages
    k, v = torch.randn(2, P * 16, 2, 128, generator=g)
    c.oasis_q8_write(k.cuda(), v.cuda(), torch.arange(P * 16).cuda())
    table = Q.table_of([n], P, n // 16 + 2, g)
    q = (3 * torch.randn(2, 1, 8, 128, generator=g)).to(BF)
    out = attend(c, q.cuda(), table, [n], True)
    again = attend(c, q.cuda(), table, [n], True)
    c.oasis_q8_sync()
    assert torch.equal(out, again)
    o, b = Q.attention(q, c.pages.cpu().numpy(), table.numpy(), [n], True, out=FP)
    close(out, o, b)


# ------------------------------------- attention with requests cut into parts
def wide(lens, Hkv, G, dtype, fp32, g, least=7000):
    """A cache whose table is wide enough that attention over the batch cuts requests into parts."""
    R = len(lens)
    nb = max(4 * -(-least // (R * Hkv)), max(-(-n // 16) for n in lens), 4 * 32 * 16 if R == 1 else 4 * 256)
    c = cache_of(sum(-(-n // 16) for n in lens) + 3, nb, G * Hkv, Hkv, out_fp32=fp32)
    pages = fill(c, g, spread=1.0)
    return c, pages, Q.table_of(lens, c.cfg.num_pages, nb, g)


@pytest.mark.parametrize("lens", [[1], [0], [700], [0, 0], [64, 0, 65], [3000, 5], [16, 255, 256, 257, 1024, 1025, 0, 2],
                                  list(range(0, 128 * 9, 9)), list(range(33))], ids=lambda x: f"{len(x)}x{max(x)}")
@pytest.mark.parametrize("S,causal,Hkv,G,dtype,fp32", [(1, False, 2, 4, BF, True), (4, True, 2, 4, HF, True),
                                                       (2, False, 1, 5, BF, False), (4, True, 1, 8, HF, False),
                                                       (3, True, 3, 1, BF, True)])
def test_attention_in_parts(dev, lens, S, causal, Hkv, G, dtype, fp32):
    g = gen(sum(lens) + S)
    R = len(lens)
    c, pages, table = wide(lens, Hkv, G, dtype, fp32, g)
    n = c.oasis_q8_attn_workspace(R, S)
    if R * Hkv <= 128:
        assert n > 0
    q = (2 * torch.randn(S, R, G * Hkv, 128, generator=g)).to(dtype).cuda()
    o, b = Q.attention(q.cpu(), pages, table.numpy(), lens, causal, out=FP if fp32 else dtype)
    close(attend(c, q, table, lens, causal), o, b)
    # whatever the scratch holds, and nothing behind it is touched
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=dev)
    out = torch.full(q.shape, 5.0, dtype=FP if fp32 else dtype, device=dev)
    t, m = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    c.oasis_q8_attn(q, t, m, out, causal=causal, workspace=ws)
    close(out, o, b)
    assert (ws[n:] == 0xFF).all()
    # and without: in one piece
    c.oasis_q8_attn(q, t, m, out, causal=causal, workspace=ws[:0])
    close(out, o, b)
    assert c.oasis_q8_sync() == 0


@pytest.mark.parametrize("Hkv,lens", [(3, [(7 * i) % 431 for i in range(120)]), (2, [333, 1000, 31])],
                         ids=["rounds", "one round"])
def test_parts_behind_whose_ends_anything_stands(dev, Hkv, lens):
    """What no query sees may be NaN codes and odd exponents, in parts too; 120 x 3 pairs take
    rounds of CTAs."""
    g = gen(44)
    S, G = 4, 4
    c, pages, table = wide(lens, Hkv, G, BF, True, g)
    for r, n in enumerate(lens):
        if n % 16:
            u = pages[int(table[r, n // 16])]
            for j in range(n % 16, 16):
                u[:, Q.key_at(j, np.arange(128))] = 0x7F
                u[:, Q.value_at(j, np.arange(128))] = 0xFF
                u[:, [4096 + j, 4112 + j]] = 255 if j & 1 else 0
    c.pages.copy_(torch.from_numpy(pages))
    assert c.oasis_q8_attn_workspace(len(lens), S) > 0
    q = (2 * torch.randn(S, len(lens), G * Hkv, 128, generator=g)).to(BF)
    out = attend(c, q.cuda(), table, lens, True)
    assert c.oasis_q8_sync() == 0
    o, b = Q.attention(q, pages, table.numpy(), lens, True, out=FP)
    close(out, o, b)


def test_parts_lengths_and_pages_that_are_wrong(dev):
    """A length past the table is cut to it, a negative one is empty, tokens of bad pages are left
    out; each raises its bit but the negative one."""
    g = gen(41)
    lens = [40, 2000, 90]
    c, pages, table = wide(lens, 2, 4, BF, True, g)
    q = torch.randn(2, 3, 8, 128, generator=g).to(BF)
    out = attend(c, q.cuda(), table, [40, -5, -2 ** 31], False)
    assert c.oasis_q8_sync() == 0
    o, b = Q.attention(q, pages, table.numpy(), [40, 0, 0], False, out=FP)
    close(out, o, b)
    bad = table.clone()
    bad[1, 125 // 2:] = c.cfg.num_pages                 # the second request's last half and all behind
    out = attend(c, q.cuda(), bad, [40, 2000, 90], False)
    with pytest.raises(ob.OasisError) as e:
        c.oasis_q8_sync()
    assert "0x1" in str(e.value)
    o, b = Q.attention(q, pages, table.numpy(), [40, 125 // 2 * 16, 90], False, out=FP)
    close(out, o, b)
    wide_table = torch.full((3, c.cfg.max_blocks), -1, dtype=torch.int32)
    wide_table[:, :8] = table[1, :8]
    out = attend(c, q.cuda(), wide_table, [2 ** 31 - 1, 128, 16 * c.cfg.max_blocks + 1], False)
    with pytest.raises(ob.OasisError):
        c.oasis_q8_sync()
    o, b = Q.attention(q, pages, wide_table.numpy(), [128, 128, 128], False, out=FP)
    close(out, o, b)


def test_parts_workspace_refusals(dev):
    g = gen(42)
    lens = [40, 2000, 90]
    c, pages, table = wide(lens, 2, 4, BF, False, g)
    q = torch.randn(1, 3, 8, 128, generator=g).to(BF).cuda()
    n = c.oasis_q8_attn_workspace(3, 1)
    t, m = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=dev)
    for bad, err in [(ws[:n - 1], ob.OasisError), (ws[16:16 + n], ob.OasisError), (ws.view(torch.int32), ValueError),
                     (ws.cpu(), ValueError), (ws[::2], ValueError)]:
        with pytest.raises(err):
            c.oasis_q8_attn(q, t, m, torch.empty_like(q), workspace=bad)
    for args in [(-1, 1), (65536, 1), (1, 0), (1, 5)]:
        with pytest.raises(ob.OasisError):
            c.oasis_q8_attn_workspace(*args)
    assert c.oasis_q8_attn_workspace(129, 1) == 0 and c.oasis_q8_attn_workspace(0, 1) == 0


def test_parts_on_streams_and_in_graphs(dev):
    """Calls that take their own scratch: eager on two streams at once, and two captured graphs
    replayed side by side, all the same bytes as one by one."""
    g = gen(43)
    lens = [1500, 3, 0, 700]
    c, pages, table = wide(lens, 2, 4, BF, True, g)
    assert c.oasis_q8_attn_workspace(4, 3) > 0
    t, m = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    qs = [torch.randn(3, 4, 8, 128, generator=g).to(BF).cuda() for _ in range(2)]
    want = []
    for q in qs:
        o = torch.empty(q.shape, dtype=FP, device=dev)
        c.oasis_q8_attn(q, t, m, o, causal=True)
        torch.cuda.synchronize()
        want.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(3, 4, 8, 128, dtype=FP, device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(40):
        c.oasis_q8_attn(qs[0], t, m, outs[0], causal=True, stream=streams[0])
        c.oasis_q8_attn(qs[1], t, m, outs[1], causal=True, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    graphs = []
    for q, o in zip(qs, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _ in range(3):
                c.oasis_q8_attn(q, t, m, o, causal=True)
        graphs.append(gr)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    # the lengths are the device's, read at each replay
    m.copy_(torch.tensor([20, 900, 1, 0], dtype=torch.int32))
    table2 = Q.table_of([20, 900, 1, 0], c.cfg.num_pages, c.cfg.max_blocks, g)
    t.copy_(table2)
    graphs[0].replay()
    torch.cuda.synchronize()
    o, b = Q.attention(qs[0].cpu(), pages, table2.numpy(), [20, 900, 1, 0], True, out=FP)
    close(outs[0], o, b)
    assert c.oasis_q8_sync() == 0


# ---------------------------------------------------------------- prefix
def prefix_of(g, Hkv, blocks, plen, garbage=True):
    x = torch.randn(Hkv, blocks, 2, 16, 128, generator=g).to(BF)
    flat = x.permute(0, 2, 1, 3, 4).reshape(Hkv, 2, blocks * 16, 128)
    kv = flat[:, :, :plen].double().numpy()
    if garbage:
        pos = torch.arange(blocks * 16).view(blocks, 1, 16, 1)
        x = torch.where(pos >= plen, torch.tensor(float("nan"), dtype=BF), x)
        inf = (pos >= plen) & (pos % 2 == 0)
        x = torch.where(inf, torch.tensor(float("inf"), dtype=BF), x)
    return x.cuda(), (kv[:, 0], kv[:, 1])


@pytest.mark.parametrize("plen,extra", [(1, 0), (16, 0), (100, 1), (127, 0), (128, 0), (129, 2), (300, 0), (1025, 3)])
@pytest.mark.parametrize("lens,S,causal", [([5], 1, False), ([0, 20, 1], 2, False), ([40, 2, 0, 17], 4, True)])
@pytest.mark.parametrize("Hq,Hkv,fp32", [(8, 2, True), (8, 1, False), (3, 3, True)])
def test_prefix(dev, plen, extra, lens, S, causal, Hq, Hkv, fp32):
    g = gen(plen * 3 + S)
    nb = max(1, max(-(-n // 16) for n in lens))
    c = cache_of(sum(-(-n // 16) for n in lens) + 1, nb, Hq, Hkv, out_fp32=fp32)
    pages = fill(c, g, spread=0.5)
    table = Q.table_of(lens, c.cfg.num_pages, nb, g)
    kv, ref = prefix_of(g, Hkv, -(-plen // 16) + extra, plen)
    q = (1.5 * torch.randn(S, len(lens), Hq, 128, generator=g)).to(BF)
    out = attend(c, q.cuda(), table, lens, causal, prefix=kv, plen=plen)
    c.oasis_q8_sync()
    o, b = Q.attention(q, pages, table.numpy(), lens, causal, prefix=ref, p_half=2.0 ** -8, out=out.dtype)
    close(out, o, b)


@pytest.mark.parametrize("R,S,Hq,Hkv,plen", [(33, 1, 8, 2, 500), (64, 4, 8, 1, 260), (70, 2, 8, 1, 1500), (130, 1, 32, 8, 200), (2, 1, 16, 16, 5000)])
def test_prefix_batches(dev, R, S, Hq, Hkv, plen):
    """Row counts around the tile size, several tiles, long prefixes with few rows."""
    g = gen(R + plen)
    lens = [int(x) for x in torch.randint(0, 40, (R,), generator=g)]
    c = cache_of(R * 3 + 1, 3, Hq, Hkv, out_fp32=True)
    pages = fill(c, g, spread=0.5)
    table = Q.table_of(lens, c.cfg.num_pages, 3, g)
    kv, ref = prefix_of(g, Hkv, -(-plen // 16), plen)
    q = (1.5 * torch.randn(S, R, Hq, 128, generator=g)).to(BF)
    out = attend(c, q.cuda(), table, lens, True, prefix=kv, plen=plen)
    c.oasis_q8_sync()
    o, b = Q.attention(q, pages, table.numpy(), lens, True, prefix=ref, p_half=2.0 ** -8, out=FP)
    close(out, o, b)


def test_prefix_of_nothing_is_attention(dev):
    g = gen(21)
    c = cache_of(10, 4, 8, 2)
    fill(c, g)
    table = Q.table_of([50, 0], 10, 4, g)
    q = torch.randn(2, 2, 8, 128, generator=g).to(BF).cuda()
    kv = torch.zeros(2, 1, 2, 16, 128, dtype=BF, device=dev)
    a = attend(c, q, table, [50, 0], False)
    b = attend(c, q, table, [50, 0], False, prefix=kv, plen=0)
    c.oasis_q8_sync()
    assert torch.equal(a, b)


def test_prefix_large_logits(dev):
    """Scores far from zero on both sides: the prefix or the suffix carries all the weight."""
    g = gen(22)
    c = cache_of(10, 4, 4, 1, out_fp32=True)
    k, v = torch.randn(2, 160, 1, 128, generator=g)
    k[:, :, 0] = 20.0
    c.oasis_q8_write(k.cuda(), v.cuda(), torch.arange(160).cuda())
    table = Q.table_of([50, 30], 10, 4, g)
    kv, ref = prefix_of(g, 1, 10, 150)
    q = torch.randn(1, 2, 4, 128, generator=g)
    q[0, 0, :, 0], q[0, 1, :, 0] = 60.0, -60.0
    q = q.to(BF)
    out = attend(c, q.cuda(), table, [50, 30], False, prefix=kv, plen=150)
    c.oasis_q8_sync()
    o, b = Q.attention(q, c.pages.cpu().numpy(), table.numpy(), [50, 30], False, prefix=ref, p_half=2.0 ** -8, out=FP)
    close(out, o, b)


# ---------------------------------------------------------------- refusals
def test_python_refusals(dev):
    c = cache_of(4, 2, 8, 2)
    k = torch.zeros(3, 2, 128, dtype=BF, device=dev)
    s = torch.arange(3, device=dev)
    t, n = torch.zeros(1, 2, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
    q = torch.zeros(1, 1, 8, 128, dtype=BF, device=dev)
    kv = torch.zeros(2, 1, 2, 16, 128, dtype=BF, device=dev)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    for call in [
        lambda: c.oasis_q8_write(k.cpu(), k, s), lambda: c.oasis_q8_write(k, k.float(), s),
        lambda: c.oasis_q8_write(k, k, s.int()), lambda: c.oasis_q8_write(k[:2], k, s),
        lambda: c.oasis_q8_write(k.double(), k.double(), s),
        lambda: c.oasis_q8_write(torch.zeros(3, 128, 2, dtype=BF, device=dev).transpose(1, 2), k, s),
        lambda: c.oasis_q8_attn(q, t[:, :1], n, q.clone()), lambda: c.oasis_q8_attn(q, t.long(), n, q.clone()),
        lambda: c.oasis_q8_attn(q.float(), t, n, q.clone()), lambda: c.oasis_q8_attn(q, t, n, q.float()),
        lambda: c.oasis_q8_attn(q[:, :, :4], t, n, q.clone()), lambda: c.oasis_q8_attn(q[0], t, n, q[0].clone()),
        lambda: c.oasis_q8_read(t, n, torch.zeros(1, 2, 2, 2, 16, 64, dtype=BF, device=dev)),
        lambda: c.oasis_q8_read(t, n, torch.zeros(1, 2, 2, 2, 16, 128, dtype=torch.int8, device=dev)),
        lambda: c.oasis_prefix_attn(q, kv.half(), 3, t, n, q.clone(), ws),
        lambda: c.oasis_prefix_attn(q, kv, 3, t, n, q.clone(), ws.cpu()),
        lambda: ob.Q8Cache(c.cfg, pages=c.pages[:3]),
    ]:
        with pytest.raises(ValueError):
            call()
    for call in [
        lambda: c.oasis_q8_attn(torch.zeros(5, 1, 8, 128, dtype=BF, device=dev), t, n, torch.zeros(5, 1, 8, 128, dtype=BF, device=dev)),
        lambda: c.oasis_prefix_attn(q, kv, 17, t, n, q.clone(), ws),
        lambda: c.oasis_prefix_attn(q, kv, -1, t, n, q.clone(), ws),
        lambda: c.oasis_prefix_attn(q.half(), kv, 3, t, n, q.half(), ws),
        lambda: c.oasis_q8_write(torch.zeros(2 * 260, dtype=BF, device=dev).as_strided((2, 2, 128), (260, 128, 1)),
                                 k[:2], s[:2]),
        lambda: c.oasis_q8_write(torch.zeros(3 * 256 + 1, dtype=BF, device=dev)[1:].view(3, 2, 128), k, s),
    ]:
        with pytest.raises(ob.OasisError) as e:
            call()
        assert e.value.status == ob.OASIS_EINVAL and len(str(e.value)) > 12
    assert c.oasis_q8_sync() == 0


def test_workspace_is_checked(dev):
    c = cache_of(4, 2, 8, 2)
    t, n = torch.zeros(1, 2, dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
    q = torch.zeros(1, 1, 8, 128, dtype=BF, device=dev)
    kv = torch.zeros(2, 10, 2, 16, 128, dtype=BF, device=dev)
    ws = c.prefix_workspace(1, 1, 160)
    assert ws.numel() >= 2 * 4 * (128 * 4 + 8)
    for bad in (ws[:-1], torch.empty(0, dtype=torch.uint8, device=dev),
                torch.empty(ws.numel() + 1, dtype=torch.uint8, device=dev)[1:]):
        with pytest.raises(ob.OasisError) as e:
            c.oasis_prefix_attn(q, kv, 160, t, n, q.clone(), bad)
        assert "workspace" in str(e.value)
    c.oasis_prefix_attn(q, kv, 160, t, n, q.clone(), ws)
    assert c.oasis_q8_sync() == 0
    for args in ((1, 5, 3), (1, 0, 3), (-1, 1, 3), (1, 1, -1)):
        with pytest.raises(ob.OasisError):
            c.oasis_prefix_workspace(*args)
    assert c.oasis_prefix_workspace(0, 1, 100) == 0 and c.oasis_prefix_workspace(3, 1, 0) == 0


def test_negative_lengths_and_any_entries_behind_a_context(dev):
    g = gen(25)
    c = cache_of(10, 6, 8, 2, out_fp32=True)
    pages = fill(c, g, spread=0.5)
    lens = [-5, 20, -(1 << 31), 0]
    table = torch.randint(-(1 << 31), (1 << 31) - 1, (4, 6), generator=g).to(torch.int32)
    table[1, :2] = torch.tensor([3, 7])
    q = torch.randn(2, 4, 8, 128, generator=g).to(BF)
    kv, ref = prefix_of(g, 2, 3, 40)
    for causal in (False, True):
        out = attend(c, q.cuda(), table, lens, causal)
        o, b = Q.attention(q, pages, table.numpy(), lens, causal, out=FP)
        close(out, o, b)
        out = attend(c, q.cuda(), table, lens, causal, prefix=kv, plen=40)
        o, b = Q.attention(q, pages, table.numpy(), lens, causal, prefix=ref, p_half=2.0 ** -8, out=FP)
        close(out, o, b)
    back = torch.full((4, 2, 6, 2, 16, 128), 3.0, dtype=FP, device=dev)
    c.oasis_q8_read(table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), back)
    assert c.oasis_q8_sync() == 0
    assert (back[0] == 3).all() and (back[2:] == 3).all() and (back[1, :, 2:] == 3).all()


def test_waits_that_run_out_are_reported(dev):
    """A limit of one cycle, on a pool larger than the L2 cache so that copies are still under way
    when they are waited for: the calls return, the error bit is raised, and with the default
    limit the same handle answers as before."""
    R, n, Hkv, plen = 48, 2048, 8, 8000
    pages = torch.randint(0, 64, (R * n // 16, Hkv, Q.UNIT), dtype=torch.uint8, device=dev)
    pages[..., 4096:] = 124
    assert pages.numel() > 160 << 20
    c = ob.Q8Cache(ob.make_q8_config(R * n // 16, n // 16, 32, Hkv), pages=pages)
    g = gen(26)
    lens = [n] * R
    table = torch.randperm(R * n // 16, generator=g).to(torch.int32).view(R, n // 16)
    q = torch.randn(2, R, 32, 128, generator=g).to(BF).cuda()
    kv = torch.randn(Hkv, plen // 16, 2, 16, 128, device=dev).to(BF)

    def both():
        return [attend(c, q, table, lens, True), attend(c, q, table, lens, True, prefix=kv, plen=plen)]
    before = both()
    assert c.oasis_q8_sync() == 0
    for prefix in (None, kv):
        c.oasis_q8_set_wait_limit(1)
        attend(c, q, table, lens, True, prefix=prefix, plen=plen)
        with pytest.raises(ob.OasisError) as e:
            c.oasis_q8_sync()
        assert e.value.status == ob.OASIS_EDEVICE and "0x2" in str(e.value)
        c.oasis_q8_set_wait_limit(0)
        after = both()
        assert c.oasis_q8_sync() == 0
        assert all(torch.equal(x, y) for x, y in zip(before, after))


# ------------------------------------------------------- streams and graphs
def test_streams_and_graph_replay(dev):
    """Write and both attentions captured once, replayed on new contents; the same calls on a side
    stream give the same bytes."""
    g = gen(31)
    c = cache_of(30, 10, 8, 2)
    fill(c, g)
    lens = [100, 37]
    table = Q.table_of(lens, 30, 10, g).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    slots = torch.stack([Q.slots_of(table.cpu(), r, m - 1, m)[0] for r, m in enumerate(lens)]).cuda()
    kv, _ = prefix_of(g, 2, 9, 140)
    q, k, v = (torch.zeros(*s, dtype=BF, device=dev) for s in [(2, 2, 8, 128), (2, 2, 128), (2, 2, 128)])
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    ws = c.prefix_workspace(2, 2, 140)

    def step():
        c.oasis_q8_write(k, v, slots)
        c.oasis_q8_attn(q, table, n, o1)
        c.oasis_prefix_attn(q, kv, 140, table, n, o2, ws, causal=True)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for i in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        a, b, p = o1.clone(), o2.clone(), c.pages.clone()
        o1.zero_(), o2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        assert torch.equal(a, o1) and torch.equal(b, o2) and torch.equal(p, c.pages)
        assert float(a.float().abs().sum()) > 0 and not torch.equal(a, b)
    assert c.oasis_q8_sync() == 0


def test_calls_in_a_row_see_what_the_ones_before_wrote(dev):
    """Launches may begin before the one ahead has ended: every call of a long run without waiting
    gives what it gives when each is waited for."""
    g = gen(33)
    N, R = 60, 40
    c = cache_of(R * 4, 4, 8, 2)
    table = torch.randperm(R * 4, generator=g).to(torch.int32).view(R, 4).cuda()
    lens = torch.randint(30, 61, (R,), generator=g)
    slots = torch.stack([Q.slots_of(table.cpu(), r, m - 1, m)[0] for r, m in enumerate(lens.tolist())]).cuda()
    ks, vs = torch.randn(2, N, R, 2, 128, generator=g).to(BF).cuda()
    qs = torch.randn(N, 2, R, 8, 128, generator=g).to(BF).cuda()
    kv, _ = prefix_of(g, 2, 20, 310)
    ws = c.prefix_workspace(R, 2, 310)
    q, k, v = torch.zeros_like(qs[0]), torch.zeros_like(ks[0]), torch.zeros_like(vs[0])
    n = torch.zeros(R, dtype=torch.int32, device=dev)
    n_all = lens.to(torch.int32).cuda()

    def go(wait):
        c.pages.zero_()
        fill_k = torch.arange(R * 64, device=dev)
        c.oasis_q8_write(base, base, fill_k)
        out = torch.zeros(N, 3, *q.shape, dtype=BF, device=dev)
        back = torch.zeros(N, R, 2, 4, 2, 16, 128, dtype=BF, device=dev)
        w = torch.cuda.synchronize if wait else lambda: None
        for i in range(N):
            for a, b in ((q, qs[i]), (k, ks[i]), (v, vs[i]), (n, n_all - i % 3)):
                a.copy_(b)
                w()
            c.oasis_q8_write(k, v, slots)
            w()
            c.oasis_q8_attn(q, table, n, out[i, 0], causal=True)
            w()
            c.oasis_prefix_attn(q, kv, 310, table, n, out[i, 1], ws)
            w()
            c.oasis_q8_attn(out[i, 1], table, n, out[i, 2])        # reads what the call before wrote
            w()
            c.oasis_q8_read(table, n, back[i])
            w()
            q.zero_(), n.zero_()
        torch.cuda.synchronize()
        return out, back

    base = torch.randn(R * 64, 2, 128, generator=g).to(BF).cuda()
    want = go(True)
    for _ in range(3):
        got = go(False)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert float(want[0].abs().sum()) > 0


def test_calls_captured_on_two_streams_that_fork_and_join(dev):
    """One graph whose work forks to a second stream and joins again, replayed: the same bytes as
    the calls one by one."""
    g = gen(34)
    c = cache_of(30, 10, 8, 2)
    fill(c, g)
    lens = [100, 37, 0, 64]
    table = Q.table_of(lens, 30, 10, g).cuda()
    n = torch.tensor(lens, dtype=torch.int32).cuda()
    slots = torch.stack([Q.slots_of(table.cpu(), r, m - 1, m)[0] for r, m in enumerate(lens) if m]).cuda()
    kv, _ = prefix_of(g, 2, 9, 140)
    q, k, v = (torch.zeros(*s, dtype=BF, device=dev) for s in [(2, 4, 8, 128), (3, 2, 128), (3, 2, 128)])
    o = [torch.zeros_like(q) for _ in range(4)]
    back = torch.zeros(4, 2, 10, 2, 16, 128, dtype=BF, device=dev)
    ws = [c.prefix_workspace(4, 2, 140) for _ in range(2)]
    p = torch.softmax(torch.randn(4, 3, 700, generator=g), -1).cuda()
    d = torch.softmax(torch.randn(4, 2, 700, generator=g), -1).cuda()
    x = torch.randint(0, 700, (4, 2), generator=g).int().cuda()
    ua, us = torch.rand(4, 2, generator=g).cuda(), torch.rand(4, generator=g).cuda()
    tok, acc = torch.zeros(4, 3, dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()

    def work(fork):
        main = torch.cuda.current_stream()
        c.oasis_q8_write(k, v, slots)
        if fork:
            side.wait_stream(main)
        with torch.cuda.stream(side if fork else main):
            c.oasis_q8_attn(q, table, n, o[0], causal=True)
            c.oasis_prefix_attn(q, kv, 140, table, n, o[1], ws[0])
            ob.oasis_verify_drafts(p, d, x, ua, us, tok, acc)
        c.oasis_prefix_attn(q, kv, 140, table, n, o[2], ws[1], causal=True)
        c.oasis_q8_read(table, n, back)
        if fork:
            main.wait_stream(side)
        c.oasis_q8_attn(o[1], table, n, o[3])

    outs = [*o, back, tok, acc]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(True)
    for i in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        us.copy_(torch.rand(4, generator=g))
        for t in outs:
            t.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        work(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
        assert all(float(t.float().abs().sum()) > 0 for t in outs)
    assert c.oasis_q8_sync() == 0


def test_two_prefix_calls_at_once_with_scratch_of_their_own(dev):
    g = gen(32)
    c = cache_of(30, 10, 8, 2)
    fill(c, g)
    table = Q.table_of([100, 37], 30, 10, g).cuda()
    n = torch.tensor([100, 37], dtype=torch.int32).cuda()
    kv, _ = prefix_of(g, 2, 80, 1270)
    qs = [torch.randn(1, 2, 8, 128, generator=g).to(BF).cuda() for _ in range(2)]
    want = [attend(c, q, table, [100, 37], False, prefix=kv, plen=1270) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    ws = [c.prefix_workspace(2, 1, 1270) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            c.oasis_prefix_attn(qs[i], kv, 1270, table, n, outs[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


# --------------------------------------------------- a decode loop of them all
def test_speculative_decode_loop(dev):
    """A prompt is written and its whole blocks read back as the shared prefix; then steps of:
    append the last token's and the drafts' keys and values, attend causally behind the prefix,
    verify, and move each request on by what was accepted."""
    g = gen(41)
    R, Hq, Hkv, n, V, prompt = 3, 8, 2, 3, 517, 150
    S = n + 1
    pre = cache_of(10, 10, Hq, Hkv, out_fp32=True)
    pk, pv = torch.randn(2, prompt, Hkv, 128, generator=g).to(BF)
    ptab = torch.randperm(10, generator=g).to(torch.int32).view(1, 10)
    pre.oasis_q8_write(pk.cuda(), pv.cuda(), Q.slots_of(ptab, 0, 0, prompt).cuda())
    prefix = torch.empty(1, Hkv, 10, 2, 16, 128, dtype=BF, device=dev)
    pre.oasis_q8_read(ptab.cuda(), torch.tensor([prompt], dtype=torch.int32).cuda(), prefix)
    ppages = np.zeros((10, Hkv, Q.UNIT), dtype=np.uint8)
    Q.write(ppages, pk, pv, Q.slots_of(ptab, 0, 0, prompt))
    ref_prefix = Q.tokens(ppages, ptab[0].tolist(), prompt)[:2]

    c = cache_of(R * 4, 4, Hq, Hkv, out_fp32=True)
    pages = np.zeros((R * 4, Hkv, Q.UNIT), dtype=np.uint8)
    table = torch.randperm(R * 4, generator=g).to(torch.int32).view(R, 4)
    lens = [0, 14, 3]
    ws = c.prefix_workspace(R, S, prompt)
    moved = 0
    for step in range(8):
        new = [m + S for m in lens]
        slots = torch.cat([Q.slots_of(table, r, lens[r], new[r]) for r in range(R)])
        k, v = torch.randn(2, R * S, Hkv, 128, generator=g).to(BF)
        c.oasis_q8_write(k.cuda(), v.cuda(), slots.cuda())
        Q.write(pages, k, v, slots)
        q = torch.randn(S, R, Hq, 128, generator=g).to(BF)
        out = attend(c, q.cuda(), table, new, True, prefix=prefix[0], plen=prompt, ws=ws)
        o, b = Q.attention(q, pages, table.numpy(), new, True, prefix=ref_prefix, p_half=2.0 ** -8, out=FP)
        close(out, o, b)
        z = 2 * torch.randn(R, n + 1, V, generator=g)
        p, d = torch.softmax(z, -1), torch.softmax(z[:, :n] + 0.5 * torch.randn(R, n, V, generator=g), -1)
        x = torch.multinomial(d.view(-1, V), 1, generator=g).view(R, n).int()
        ua, us = torch.rand(R, n, generator=g), torch.rand(R, generator=g)
        tok = torch.empty(R, n + 1, dtype=torch.int32, device=dev)
        acc = torch.empty(R, dtype=torch.int32, device=dev)
        ob.oasis_verify_drafts(p.cuda(), d.cuda(), x.cuda(), ua.cuda(), us.cuda(), tok, acc)
        wt, wa = Q.verify(p, d, x, ua, us)
        assert np.array_equal(tok.cpu().numpy(), wt) and np.array_equal(acc.cpu().numpy(), wa)
        lens = [m + 1 + int(a) for m, a in zip(lens, wa)]    # the refused drafts' slots are written again
        moved += int(wa.sum())
        if max(lens) + S > 64:
            break
    assert moved > 0
    assert np.array_equal(c.pages.cpu().numpy(), pages)
    assert c.oasis_q8_sync() == 0

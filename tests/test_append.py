"""Appending with the rotation on the GPU against the 64-bit definitions:
queries within fp32's rounding, keys within one code's, values exactly as
oasis_q8_write's; everything else in the pages as it was."""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T
from tests.test_q8 import BF, FP, HF, cache_of, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def rope_of(rot, axes, interleaved, base=10000.0, scale=1.0):
    half = rot // 2
    return ob.make_rope(rot, base=base, axis=[i * axes // half for i in range(half)], interleaved=interleaved,
                        scale=scale)


def check(c, old, rope, x_q, x_k, x_v, q_out, positions, slots):
    """Pages and rotated queries of tokens whose inputs are x_*, given the pages before."""
    pages = c.pages.cpu().numpy()
    want = old.copy()
    free = Q.write(want, x_k, x_v, slots)                # values: exactly these
    dim, P = np.arange(128), old.shape[0]
    y, bound = T.rotate(x_k, positions, rope)
    keys = np.zeros(old.shape, dtype=bool)
    for t, slot in enumerate(slots.tolist()):
        if not 0 <= slot < P * 16:
            continue
        p, j = divmod(slot, 16)
        keys[p][:, Q.key_at(j, dim)] = True
        keys[p][:, 4096 + j] = True
        e = pages[p][:, 4096 + j].astype(int) - 127
        value = Q.TABLE[pages[p][:, Q.key_at(j, dim)]] * 2.0 ** e[:, None]
        top = np.abs(y[t]).max(-1)
        most = np.array([bound[t, h][np.abs(y[t, h]).argmax()] for h in range(len(top))])
        for s in (-1, 1):                                # the least e with max <= 448 * 2^e, of either end
            near = top + s * most
            least = np.clip(np.ceil(np.log2(np.maximum(near, 2.0 ** -140) / 448)), -100, 120)
            assert (e >= least).all() if s < 0 else (e <= least).all(), (t, e, least)
        off = np.abs(value - y[t])
        most = 2.0 ** -4 * np.abs(y[t]) + 2.0 ** (e[:, None] - 10.0) + 1.1 * bound[t]
        assert (off <= most).all(), (t, (off - most).max())
    assert np.array_equal(pages[~keys & ~free], want[~keys & ~free])
    if x_q is not None:
        y, bound = T.rotate(x_q, positions, rope)
        got = q_out.double().cpu().numpy()
        most = 1.01 * bound + Q.HALF[q_out.dtype] * np.abs(y) * 1.01 + 2.0 ** -25 * (q_out.dtype is HF) + 1e-40
        assert (np.abs(got - y) <= most).all(), (np.abs(got - y) - most).max()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("T_,Hq,Hkv,rot,axes,interleaved,mode", [
    (1, 1, 1, 128, 1, False, "random"), (2, 4, 2, 16, 1, True, "random"), (17, 7, 1, 64, 3, False, "block"),
    (33, 24, 8, 96, 2, True, "offset"), (161, 8, 2, 128, 4, True, "block"), (200, 5, 5, 32, 1, False, "random"),
    (64, 40, 8, 112, 3, False, "holes"), (700, 8, 8, 128, 1, False, "mixed")])
def test_append(dev, dtype, T_, Hq, Hkv, rot, axes, interleaved, mode):  # noqa: F811
    g = gen(T_ * 5 + rot)
    P = T_ // 16 + 5
    c = cache_of(P, 1, Hq, Hkv)
    old = torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8)
    c.pages.copy_(old)
    x = torch.randn(T_, Hq + 2 * Hkv, 128, generator=g) * torch.exp2(3 * torch.randn(T_, Hq + 2 * Hkv, 1, generator=g))
    x = x.to(dtype)
    slots = {"random": torch.randperm(P * 16, generator=g)[:T_], "block": torch.arange(T_) + 16,
             "offset": torch.arange(T_) + 5, "holes": torch.arange(T_) + 16,
             "mixed": torch.cat([torch.arange(300) + 3, torch.arange(500) + 320])[:T_]}[mode]
    if mode == "holes":
        slots[torch.rand(T_, generator=g) < 0.3] = -1
    pos = torch.randint(-3, 200000, (axes, T_), generator=g)
    rope = rope_of(rot, axes, interleaved)
    d = x.cuda()
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]     # slices of one projection
    out = torch.empty(T_, Hq, 128, dtype=dtype, device=dev)
    c.oasis_q8_append(rope, q, k, v, pos.cuda(), slots.cuda(), out)
    assert c.oasis_q8_sync() == 0
    check(c, old.numpy(), rope, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], out, pos, slots)
    c.pages.copy_(old)
    c.oasis_q8_append(rope, q, k, v, pos.cuda(), slots.cuda(), q)       # in place
    assert torch.equal(q, out)


def test_far_positions_and_scale(dev):  # noqa: F811
    """Positions to both ends of 64 bits; a scale; frequencies over a turn and below zero."""
    g = gen(3)
    f = [1.0, 7.5, -0.3, 1e-7, 2.0 ** 20, 0.0, 6.283185307179586, 1e-300]
    rope = ob.make_rope(16, frequency=f, scale=0.7071)
    pos = torch.tensor([0, 1, -1, 2 ** 31, 10 ** 9, 10 ** 6 + 1, 2 ** 40, -(2 ** 33)])
    c = cache_of(2, 1, 2, 1)
    x = torch.randn(8, 4, 128, generator=g)
    out = torch.empty(8, 2, 128, device=dev)
    slots = torch.arange(8) + 3
    c.oasis_q8_append(rope, x.cuda()[:, :2], x.cuda()[:, 2:3], x.cuda()[:, 3:], pos.cuda(), slots.cuda(), out)
    y, bound = T.rotate(x[:, :2], pos, rope)
    # a frequency is held to 2^-64 of a turn: past 2^32 positions that shows
    bound += (2 ** -64 * 2 * np.pi * pos.abs().double().numpy())[:, None, None] * 4
    assert (np.abs(out.double().cpu().numpy() - y) <= 1.01 * bound + 2.0 ** -23 * np.abs(y)).all()
    assert c.oasis_q8_sync() == 0


def test_position_zero_is_a_write(dev):  # noqa: F811
    """At position 0 nothing turns: pages are oasis_q8_write's, queries as they were (1,000 tokens
    and one, in every type)."""
    for dtype in (BF, HF, FP):
        for T_ in (1, 1000):
            g = gen(T_)
            a, b = cache_of(80, 1, 8, 2), cache_of(80, 1, 8, 2)
            x = torch.randn(T_, 12, 128, generator=g).to(dtype).cuda()
            x[0, 8, 3], x[0, 10, 4] = float("inf"), float("nan")
            slots = (torch.arange(T_) + 7).cuda()
            out = torch.empty(T_, 8, 128, dtype=dtype, device=dev)
            a.oasis_q8_append(ob.make_rope(64), x[:, :8], x[:, 8:10], x[:, 10:], torch.zeros(T_, dtype=torch.int64).cuda(),
                              slots, out)
            b.oasis_q8_write(x[:, 8:10], x[:, 10:], slots)
            at = (a.pages != b.pages)
            # (an infinite entry times sin 0 makes its pair's other entry NaN)
            assert int(at[0, 0].sum()) <= 1 and not at[1:].any() and torch.equal(out, x[:, :8])


def test_keys_alone_and_bad_slots(dev):  # noqa: F811
    g = gen(9)
    c = cache_of(3, 1, 4, 2)
    old = torch.randint(0, 256, c.pages.shape, generator=g, dtype=torch.uint8)
    x = torch.randn(20, 8, 128, generator=g).to(BF)
    d = x.cuda()
    pos, slots = torch.arange(20) * 1000, torch.arange(20) + 30          # the last two past the pool
    rope = rope_of(128, 1, False)
    c.pages.copy_(old)
    c.oasis_q8_append(rope, None, d[:, 4:6], d[:, 6:], pos.cuda(), slots.cuda(), None)
    with pytest.raises(ob.OasisError, match="0x4"):
        c.oasis_q8_sync()
    check(c, old.numpy(), rope, None, x[:, 4:6], x[:, 6:], None, pos, slots)
    c.oasis_q8_append(rope, None, d[:0, 4:6], d[:0, 6:], pos[:0].cuda(), slots[:0].cuda(), None)
    out = torch.empty(20, 4, 128, dtype=BF, device=dev)
    c.oasis_q8_append(rope, d[:, :4], d[:, 4:6], d[:, 6:], pos.cuda(), torch.full((20,), -5).cuda(), out)
    assert c.oasis_q8_sync() == 0
    check(c, c.pages.cpu().numpy(), rope, x[:, :4], x[:, 4:6], x[:, 6:], out, pos, torch.full((20,), -5))


def test_refusals(dev):  # noqa: F811
    c = cache_of(4, 1, 4, 2)
    rope = ob.make_rope(64, axis=[0] * 16 + [1] * 16)
    good = dict(rope=rope, q=torch.zeros(3, 4, 128, dtype=BF, device=dev), k=torch.zeros(3, 2, 128, dtype=BF, device=dev),
                v=torch.zeros(3, 2, 128, dtype=BF, device=dev), positions=torch.zeros(2, 3, dtype=torch.int64, device=dev),
                slots=torch.arange(3, device=dev), q_out=torch.zeros(3, 4, 128, dtype=BF, device=dev))
    c.oasis_q8_append(**good)
    z = torch.zeros
    for change in (dict(q=None), dict(q_out=None), dict(k=z(3, 2, 128, dtype=torch.float64, device=dev)),
                   dict(v=z(3, 2, 128, device=dev)), dict(q=z(3, 2, 128, dtype=BF, device=dev)),
                   dict(q_out=z(3, 4, 128, device=dev)), dict(positions=z(3, dtype=torch.int64, device=dev)),
                   dict(positions=z(2, 3, dtype=torch.int32, device=dev)), dict(positions=z(2, 3, dtype=torch.int64)),
                   dict(slots=z(3, dtype=torch.int32, device=dev)), dict(k=z(3, 2, 128, dtype=BF)),
                   dict(k=z(3, 4, 128, dtype=BF, device=dev)[:, ::2]), dict(k=z(2, 2, 128, dtype=BF, device=dev))):
        with pytest.raises(ValueError):
            c.oasis_q8_append(**{**good, **change})
    for change in (dict(k=z(3 * 256 + 1, dtype=BF, device=dev)[1:].view(3, 2, 128)),
                   dict(q_out=z(600, dtype=BF, device=dev).as_strided((3, 4, 128), (8, 128, 1))),
                   dict(v=z(3 * 260, dtype=BF, device=dev).as_strided((3, 2, 128), (257, 128, 1)))):
        with pytest.raises(ob.OasisError, match="EINVAL"):
            c.oasis_q8_append(**{**good, **change})
    bad = ob.make_rope(64)
    bad.num_axes = 0
    with pytest.raises((ob.OasisError, ValueError)):
        c.oasis_q8_append(**{**good, "rope": bad})
    assert c.oasis_q8_sync() == 0

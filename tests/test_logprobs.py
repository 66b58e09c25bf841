"""Log probabilities, entropy and alternatives on the GPU against 64 bits.

Bound, for x with maximum m: S is a sum of up to 2^20 terms 2^y, each off by
2^-22 (two units of fp32's exponential) + 2^-23 |y| (y rounded, and log2 e as a
float, 2^-26 |y|), summed in chains of at most 4096 and in trees: a relative
error of 2^-11 + 2^-22 at the very worst, but roundings of both signs: held to
2^-19 as documented.  log S: that, and log2's own 2^-22; times ln 2.  The
token's (x - m): 2^-22 of itself.  Entropy: both terms have the sums' error.
"""
import numpy as np
import pytest
import torch

from sparse_kv_block_gb300 import oasis as ob
from tests import _tree as T
from tests.test_q8 import BF, FP, HF, dev, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def go(x, tokens, k, old=5.0):
    rows = x.shape[0]
    d = "cuda"
    o = dict(logprobs=torch.full((rows,), old, device=d), entropy=torch.full((rows,), old, device=d),
             top_ids=torch.full((rows, k), int(old), dtype=torch.int32, device=d),
             top_logprobs=torch.full((rows, k), old, device=d))
    if tokens is None:
        o.pop("logprobs")
    if k == 0:
        o.pop("top_ids"), o.pop("top_logprobs")
    ob.oasis_token_logprobs(x, None if tokens is None else torch.as_tensor(tokens, dtype=torch.int32).cuda(), **o)
    return {n: t.cpu().numpy() for n, t in o.items()}


def check(x, tokens, k, got, old=5.0):
    lp, H, ids, top = T.logprobs(x, tokens, k)
    m = x.double().cpu().numpy().max(-1)
    want = np.ones(len(lp), dtype=bool) if tokens is None else np.asarray(tokens) >= 0

    def near(a, b, depth):
        same = (a == b) | (np.isnan(a) & np.isnan(b))
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(a - b) <= 2.0 ** -19 + 2.0 ** -21 * np.abs(b) + 2.0 ** -22 * depth)).all(), np.nanmax(np.abs(a - b))
    if tokens is not None:
        near(got["logprobs"][want], lp[want], np.where(np.isfinite(lp), -lp, 0)[want])
        assert (got["logprobs"][~want] == old).all()
    near(got["entropy"][want], H[want], 0)
    assert (got["entropy"][~want] == old).all()
    if k:
        fin = np.isfinite(m) & want
        assert np.array_equal(got["top_ids"][fin], ids[fin])
        near(got["top_logprobs"][want], top[want], np.where(np.isfinite(top), -top, 0)[want])
        assert (got["top_ids"][~want] == int(old)).all() and (got["top_logprobs"][~want] == old).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (1, 1, 0), (3, 2, 5), (2, 31, 32), (5, 100, 7), (4, 1000, 20), (1, 32000, 5),
                                      (7, 8191, 32), (33, 4097, 1), (2, 151936, 20), (700, 300, 3), (3, 50257, 32),
                                      (1, 1 << 20, 32)])
def test_logprobs(dev, dtype, rows, V, k):  # noqa: F811
    g = gen(rows + V)
    x = (3 * torch.randn(rows, V, generator=g)).to(dtype).cuda()
    tokens = torch.randint(0, V, (rows,), generator=g).tolist()
    if rows > 2:
        tokens[1] = -1
    check(x, tokens, k, go(x, tokens, k))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("V,pad,first", [(1001, 7, 0), (1001, 0, 3), (4096, 8, 1), (333, 1, 2), (5, 0, 1)])
def test_rows_at_any_alignment(dev, dtype, V, pad, first):  # noqa: F811
    """Rows of a padded or shifted buffer, whose neighbours would win if they were read."""
    g = gen(V + pad)
    rows = 9
    buf = torch.full((first + rows * (V + pad) + 64,), 1000.0, dtype=dtype)
    x = buf[first:].as_strided((rows, V), (V + pad, 1))
    x.copy_(2 * torch.randn(rows, V, generator=g))
    d = buf.cuda()[first:].as_strided((rows, V), (V + pad, 1))
    tokens = torch.randint(0, V, (rows,), generator=g).tolist()
    check(x, tokens, 5, go(d, tokens, 5))


@pytest.mark.parametrize("kind", ["equal", "two", "rising", "falling", "steps", "masked", "one", "clusters", "zeros"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_ties_and_orders(dev, kind, dtype):  # noqa: F811
    """Equal entries go by the lower token; orders that defeat a threshold; mostly -infinity."""
    V, rows = 20000, 3
    g = gen(5)
    i = torch.arange(V).float()
    x = {"equal": torch.zeros(V), "two": (i % 2), "rising": i / 3000, "falling": -i / 3000, "steps": torch.floor(i / 500) / 10,
         "masked": torch.where(i % 2999 == 7, i / 1000, -float("inf")), "one": torch.where(i == 12345, 0.0, -float("inf")),
         "clusters": torch.where((i // 8) % 256 == 3, 5.0 + i / 20000, i / 20000),
         "zeros": torch.where(i % 3 == 0, -0.0, 0.0)}[kind]
    x = x.repeat(rows, 1)
    x[1] = x[1].flip(0)
    x[2] = x[2][torch.randperm(V, generator=g)]
    x = x.to(dtype).cuda()
    for k in (1, 20, 32):
        check(x, [5, 12345, 0], k, go(x, [5, 12345, 0], k))


@pytest.mark.parametrize("amp", [0.0, 1e-3, 30.0, 1e4])
def test_flat_and_sharp(dev, amp):  # noqa: F811
    g = gen(8)
    x = (amp * torch.randn(6, 3000, generator=g)).cuda()
    tokens = x.argmax(1).tolist()
    check(x, tokens, 4, go(x, tokens, 4))
    x = x + 5e4
    check(x, tokens, 4, go(x, tokens, 4))


def test_rows_without_a_sum(dev):  # noqa: F811
    """NaN, +infinity, only -infinity: NaN; the rows beside them as ever; tokens past V."""
    g = gen(9)
    for dtype in (BF, HF, FP):
        x = torch.randn(6, 700, generator=g).to(dtype)
        x[0, 300], x[1, 699], x[2] = float("nan"), float("inf"), -float("inf")
        x[4, ::2] = -float("inf")
        got = go(x.cuda(), [0, 0, 0, 700, 1, 0], 3)
        for n in ("logprobs", "entropy", "top_logprobs"):
            assert np.isnan(got[n][:3]).all(), n
        assert got["logprobs"][3] == -np.inf
        check(x[3:], [700, 1, 0], 3, {n: v[3:] for n, v in got.items()})
        got = go(x.cuda(), [0, 0, 0, 0, 0, 0], 1)
        assert got["logprobs"][4] == -np.inf
    x = torch.zeros(2, 9000)
    x[0, 8999], x[1, 8999] = float("nan"), float("inf")
    got = go(x.cuda(), [0, 0], 2)
    assert np.isnan(got["logprobs"]).all() and np.isnan(got["entropy"]).all()


def test_parts_of_the_outputs(dev):  # noqa: F811
    x = torch.randn(2, 3, 500, device=dev)
    full = go(x.view(6, 500), [1] * 6, 4)
    H = torch.empty(2, 3, device=dev)
    ob.oasis_token_logprobs(x, entropy=H)
    assert np.array_equal(H.cpu().numpy().ravel(), full["entropy"])
    ids, top = torch.empty(2, 3, 4, dtype=torch.int32, device=dev), torch.empty(2, 3, 4, device=dev)
    ob.oasis_token_logprobs(x, top_ids=ids, top_logprobs=top)
    assert np.array_equal(ids.cpu().numpy().reshape(6, 4), full["top_ids"])
    lp = torch.empty(2, 3, device=dev)
    ob.oasis_token_logprobs(x, torch.ones(2, 3, dtype=torch.int32, device=dev), lp)
    assert np.array_equal(lp.cpu().numpy().ravel(), full["logprobs"])
    view = x.transpose(0, 1)                                 # rows 500 and 1500 apart
    with pytest.raises(ValueError):
        ob.oasis_token_logprobs(view, entropy=torch.empty(3, 2, device=dev))
    ob.oasis_token_logprobs(x[:, 1], entropy=H[:, 1].contiguous())


def test_captured_on_a_stream(dev):  # noqa: F811
    x = torch.randn(40, 30000, device=dev)
    tokens = torch.arange(40, dtype=torch.int32, device=dev)
    lp, H = torch.empty(40, device=dev), torch.empty(40, device=dev)
    ids, top = torch.empty(40, 8, dtype=torch.int32, device=dev), torch.empty(40, 8, device=dev)
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        ob.oasis_token_logprobs(x, tokens, lp, H, ids, top, stream=st)
    for _ in range(2):
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        check(x, tokens.tolist(), 8, dict(logprobs=lp.cpu().numpy(), entropy=H.cpu().numpy(), top_ids=ids.cpu().numpy(),
                                          top_logprobs=top.cpu().numpy()))


def test_refusals(dev):  # noqa: F811
    x = torch.zeros(4, 100, device=dev)
    f = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    for args, kw in (((x.double(),), {}), ((x.cpu(),), {}), ((x[0],), {}), ((x.t(),), {}), ((x, None, f(4)), {}),
                     ((x, i(4).long()), {}), ((x, i(3)), {}), ((x, i(4), f(4, 1)), {}), ((x, i(4), f(4).double()), {}),
                     ((x,), dict(top_ids=i(4, 3))), ((x,), dict(top_ids=i(4, 3), top_logprobs=f(4, 2))),
                     ((x,), dict(entropy=f(8)[::2]))):
        with pytest.raises(ValueError):
            ob.oasis_token_logprobs(*args, **kw)
    with pytest.raises(ob.OasisError, match="top"):
        ob.oasis_token_logprobs(x, top_ids=i(4, 33), top_logprobs=f(4, 33))
    with pytest.raises(ob.OasisError, match="stride"):
        ob.oasis_token_logprobs(x[:1].expand(4, 100), entropy=f(4))
    ob.oasis_token_logprobs(x[:0], i(0), f(0), f(0))

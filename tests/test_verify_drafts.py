"""oasis_verify_drafts on the GPU against its 64-bit definition: tokens and
counts are whole numbers and have to be equal."""
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


def go(p, q, x, ua, us, nd=None, stream=None):
    R, n1, _ = p.shape
    tok = torch.full((R, n1), 99, dtype=torch.int32, device="cuda")
    acc = torch.full((R,), 99, dtype=torch.int32, device="cuda")
    up = lambda t: None if t is None else t if t.is_cuda else t.cuda()  # noqa: E731
    ob.oasis_verify_drafts(up(p), up(q), up(x), up(ua), up(us), tok, acc, n_drafts=up(nd), stream=stream)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), acc.cpu().numpy()


def draw(R, n, V, g, dtype=FP, temp=2.0, noise=0.7):
    z = temp * torch.randn(R, n + 1, V, generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :n] + noise * torch.randn(R, n, V, generator=g), -1)
    x = torch.multinomial(q.reshape(-1, V), 1, generator=g).view(R, n).int() if n else torch.zeros(R, 0, dtype=torch.int32)
    return p.to(dtype), q.to(dtype), x, torch.rand(R, n, generator=g), torch.rand(R, generator=g)


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("R,n,V", [(1, 1, 1), (2, 0, 7), (3, 2, 31), (1, 3, 1023), (40, 3, 1024), (5, 6, 1025),
                                   (2, 4, 32000), (64, 3, 5003), (170, 2, 2500), (3, 3, 151936), (1, 64, 300), (270, 1, 9001)])
def test_against_definition(dev, dtype, R, n, V):
    p, q, x, ua, us = draw(R, n, V, gen(R * 1000 + V + n), dtype)
    for d in (q, None):
        wt, wa = Q.verify(p, d, x, ua, us)
        tok, acc = go(p, d, x, ua, us)
        assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


def test_every_count_occurs(dev):
    p, q, x, ua, us = draw(300, 3, 200, gen(5))
    _, wa = Q.verify(p, q, x, ua, us)
    assert set(wa.tolist()) == {0, 1, 2, 3}
    tok, acc = go(p, q, x, ua, us)
    wt, _ = Q.verify(p, q, x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


def test_ragged_drafts(dev):
    p, q, x, ua, us = draw(8, 3, 1500, gen(6))
    nd = torch.tensor([0, 1, 2, 3, 5, -1, 3, 0], dtype=torch.int32)   # held to 0..3
    x[0, 0], x[1, 2] = -5, 1 << 30          # behind the last draft: not read
    wt, wa = Q.verify(p, q, x, ua, us, nd)
    tok, acc = go(p, q, x, ua, us, nd)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


def test_bad_token_spoils_only_its_request(dev):
    p, q, x, ua, us = draw(4, 3, 1500, gen(7))
    x[1, 2], x[2, 0] = 1500, -1
    wt, wa = Q.verify(p, q, x, ua, us)
    assert wa[1] == -1 and wa[2] == -1
    tok, acc = go(p, q, x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


def test_equal_distributions_and_empty_rows(dev):
    """p = q: everything is accepted for u < 1; u = 1 refuses, nothing is left, p itself is drawn
    from.  A row of zeros gives -1; NaN entries count as 0."""
    p, q, x, ua, us = draw(4, 2, 3000, gen(8))
    q = p[:, :2].clone()
    wt, wa = Q.verify(p, q, x, ua, us)
    assert (wa == 2).all()
    tok, acc = go(p, q, x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)
    ua[:, 0] = 1.0
    wt, wa = Q.verify(p, q, x, ua, us)
    assert (wa == 0).all() and (wt[:, 0] >= 0).all()
    tok, acc = go(p, q, x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)
    p[1] = 0
    p[2, 0, 100:2000] = float("nan")
    ua[2, 0] = 1.0
    wt, wa = Q.verify(p, q, x, ua, us)
    tok, acc = go(p, q, x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt) and tok[1, 0] == -1


def test_nan_negative_and_infinite_entries(dev):
    """NaN and negative entries count as 0, for acceptance too; an infinite entry of a row that is
    drawn from, p's or the one subtracted, leaves no token."""
    p, q, x, ua, us = draw(9, 2, 1500, gen(9))
    ua[:, 0], ua[:, 1] = 0.0, 0.5
    nan, inf = float("nan"), float("inf")
    at = lambda r, i: (r, i, int(x[r, i]))  # noqa: E731
    q[at(0, 0)] = nan                                  # 0 < p: accepted
    p[at(1, 0)] = nan                                  # refused
    q[at(2, 0)], p[at(2, 0)], ua[2, 0] = -0.5, 0.0, 0.5    # 0 < 0: refused
    p[at(3, 0)] = -1.0                                 # refused, and no part of the difference
    p[at(4, 0)], q[4, 0, 7] = 0.0, inf                 # refused, no difference
    p[at(5, 0)], p[5, 0, 7] = 0.0, inf
    q[at(6, 0)] = q[at(6, 1)] = 0.0                    # both accepted, p drawn from
    p[6, 2, 1200] = inf
    q[7, 0, :] = -q[7, 0, :]                           # accepted; the second as it comes
    p[8], q[8, 0, 3] = -p[8], inf
    for dtype in (FP, BF, HF):
        pt, qt = p.to(dtype), q.to(dtype)
        for d in (qt, None):
            wt, wa = Q.verify(pt, d, x, ua, us)
            tok, acc = go(pt, d, x, ua, us)
            assert np.array_equal(acc, wa) and np.array_equal(tok, wt)
            if d is not None:
                assert acc[0] >= 1 and acc[7] >= 1 and (acc[1:6] == 0).all() and acc[6] == 2 and acc[8] == 0
                assert (tok[[4, 5, 8], 0] == -1).all() and tok[6, 2] == -1 and (tok[[1, 2, 3], 0] >= 0).all()


@pytest.mark.parametrize("V", [1, 33, 2049, 40000])
def test_borders(dev, V):
    """u on the exact borders of dyadic probabilities: the first sum above u * total wins; u = 0
    takes the first positive entry, u = 1 the last."""
    w = torch.zeros(V)
    idx = torch.unique(torch.linspace(0, V - 1, 16).long())
    w[idx] = 2.0 ** -6
    us = torch.arange(0, len(idx) + 1).float() / len(idx) if len(idx) in (1, 2, 4, 8, 16) else torch.tensor([0.0, 1.0])
    R = len(us)
    p = w.view(1, 1, V).expand(R, 1, V).contiguous()
    e = torch.zeros(R, 0)
    tok, acc = go(p, None, e.int(), e, us)
    want, _ = Q.verify(p, None, e.int(), e, us)
    assert np.array_equal(tok, want)
    assert tok[0, 0] == idx[0] and tok[-1, 0] == idx[-1]


def test_tiny_entries_count(dev):
    """150,000 entries of 1e-9 behind one of 1: a 32-bit running sum would lose them."""
    V = 150001
    p = torch.full((64, 1, V), 1e-9)
    p[:, 0, 0] = 1.0
    us = torch.linspace(0.99986, 0.99999, 64)
    e = torch.zeros(64, 0)
    tok, _ = go(p, None, e.int(), e, us)
    want, _ = Q.verify(p, None, e.int(), e, us)
    assert np.array_equal(tok, want) and (want[1:, 0] > 0).all()


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("pad,off", [(0, 1), (5, 0), (8, 0), (3, 3)])
def test_padded_and_unaligned_rows(dev, dtype, pad, off):
    R, n, V = 5, 3, 2000
    p, q, x, ua, us = draw(R, n, V, gen(9), dtype)

    def place(t):
        m = t.shape[1]
        buf = torch.full((R * m * (V + pad) + off,), float("nan"), dtype=dtype, device="cuda")
        v = buf[off:].as_strided((R, m, V), (m * (V + pad), V + pad, 1), off)
        v.copy_(t)
        return v
    wt, wa = Q.verify(p, q, x, ua, us)
    tok, acc = go(place(p), place(q), x, ua, us)
    assert np.array_equal(acc, wa) and np.array_equal(tok, wt)


def test_python_refusals(dev):
    p, q, x, ua, us = (t.cuda() for t in draw(2, 3, 50, gen(10)))
    tok = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    acc = torch.zeros(2, dtype=torch.int32, device=dev)
    for args in [(p.double(), q, x, ua, us, tok, acc), (p, q[:, :2], x, ua, us, tok, acc),
                 (p, q.half(), x, ua, us, tok, acc), (p, q, x.long(), ua, us, tok, acc),
                 (p, q, x, ua.double(), us, tok, acc), (p, q, x, ua, us, tok[:, :3], acc),
                 (p.cpu(), q, x, ua, us, tok, acc), (p[0], q, x, ua, us, tok, acc),
                 (p.transpose(1, 2).contiguous().transpose(1, 2), q, x, ua, us, tok, acc),
                 (p[:, :, ::2], q[:, :, ::2], x, ua, us, tok, acc)]:
        with pytest.raises(ValueError):
            ob.oasis_verify_drafts(*args)
    big = torch.zeros(1, 66, 2, device=dev)
    with pytest.raises(ob.OasisError):
        ob.oasis_verify_drafts(big, None, torch.zeros(1, 65, dtype=torch.int32, device=dev),
                               torch.zeros(1, 65, device=dev), us[:1], torch.zeros(1, 66, dtype=torch.int32, device=dev), acc[:1])


def test_graph_and_side_stream(dev):
    R, n, V = 6, 3, 9000
    bufs = [t.cuda() for t in draw(R, n, V, gen(11))]
    tok = torch.zeros(R, n + 1, dtype=torch.int32, device=dev)
    acc = torch.zeros(R, dtype=torch.int32, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ob.oasis_verify_drafts(*bufs, tok, acc)
    for i in range(3):
        new = draw(R, n, V, gen(12 + i))
        for b, t in zip(bufs, new):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        wt, wa = Q.verify(*new)
        assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)
        t2, a2 = go(*bufs, stream=torch.cuda.Stream())
        assert np.array_equal(a2, wa) and np.array_equal(t2, wt)

"""The tree step's calls without a GPU: refused arguments (all checked before
any device work), host helpers, and the 64-bit definitions against hand-made
cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q
from tests import _tree as T


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def rope(**kw):
    r = ob.oasis_rope(32, 2, 0, 0.0)
    for i in range(16):
        r.frequency[i], r.axis[i] = 0.5 ** i, i & 1
    for k, v in kw.items():
        if k in ("frequency", "axis"):
            getattr(r, k)[3] = v
        else:
            setattr(r, k, v)
    return r


@pytest.mark.parametrize("change,msg", [
    (dict(rot_dim=0), "rot_dim"), (dict(rot_dim=24), "rot_dim"), (dict(rot_dim=144), "rot_dim"),
    (dict(rot_dim=-16), "rot_dim"), (dict(num_axes=0), "num_axes"), (dict(num_axes=5), "num_axes"),
    (dict(num_axes=1), "axis"), (dict(interleaved=2), "interleaved"), (dict(scale=-1.0), "scale"),
    (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"),
    (dict(frequency=math.nan), "frequencies"), (dict(frequency=math.inf), "frequencies"),
    (dict(frequency=-2.0 ** 21), "frequencies"), (dict(axis=2), "axis"), (dict(axis=-1), "axis"),
])
def test_rope_refusals(change, msg):
    assert ob.lib().oasis_rope_error(ctypes.byref(rope())) is None
    assert msg in ob.lib().oasis_rope_error(ctypes.byref(rope(**change))).decode()


def test_null_handles():
    L = ob.lib()
    assert L.oasis_rope_error(None) == b"null rotation"
    r = rope()
    assert L.oasis_q8_append(None, ctypes.byref(r), 16, 16, 16, 16, 0, 256, 256, 256, 256, 16, 16, 1, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_tree_attn(None, 1, 1, 16, 0, 16, None, 16, 16, 16, None, 0, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_tree_workspace(None, 1, 1, 0, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_keep(None, 1, 1, None, 16, 16, 16, 16, 1, None) == ob.OASIS_EINVAL
    assert L.oasis_token_logprobs(None, None) == ob.OASIS_EINVAL


def logprobs_args(**kw):
    a = ob.oasis_logprobs_args(4, 100, ob.OASIS_FP32, 3, 0, 4096, 100, 4096, 4096, 4096, 4096, 4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,msg", [
    (dict(num_rows=-1), "num_rows"), (dict(num_rows=(1 << 24) + 1), "num_rows"),
    (dict(vocab=0), "vocab"), (dict(vocab=(1 << 20) + 1), "vocab"), (dict(type=3), "type"),
    (dict(type=-1), "type"), (dict(top=-1), "top"), (dict(top=33), "top"), (dict(device=-1), "device"),
    (dict(logits=None), "null"), (dict(top_ids=None), "null"), (dict(top_logprobs=None), "null"),
    (dict(tokens=None), "without tokens"), (dict(stride=99), "stride"), (dict(logits=4098), "aligned"),
    (dict(logits=4097, type=ob.OASIS_BF16), "aligned"), (dict(tokens=4098), "aligned"),
    (dict(entropy=4097), "aligned"), (dict(top_ids=4098), "aligned"),
])
def test_logprobs_refusals(change, msg):
    a = logprobs_args(**change)
    assert msg in ob.lib().oasis_logprobs_error(ctypes.byref(a)).decode()
    assert ob.lib().oasis_token_logprobs(ctypes.byref(a), None) == ob.OASIS_EINVAL


def test_logprobs_accepts():
    L = ob.lib()
    for a in (logprobs_args(), logprobs_args(top=0, top_ids=None, top_logprobs=None),
              logprobs_args(tokens=None, logprobs=None), logprobs_args(entropy=None),
              logprobs_args(num_rows=0, logits=None)):
        assert L.oasis_logprobs_error(ctypes.byref(a)) is None
    assert L.oasis_token_logprobs(ctypes.byref(logprobs_args(num_rows=0, logits=None)), None) == ob.OASIS_OK


def test_make_rope():
    r = ob.make_rope(64, base=10000.0, sections=(8, 12, 12), interleaved=True, scale=1.25)
    assert (r.rot_dim, r.num_axes, r.interleaved, r.scale) == (64, 3, 1, 1.25)
    assert list(r.axis[:32]) == [0] * 8 + [1] * 12 + [2] * 12
    assert r.frequency[0] == 1.0 and r.frequency[16] == 10000.0 ** -0.5
    assert ob.make_rope().num_axes == 1
    with pytest.raises(ValueError):
        ob.make_rope(64, sections=(8, 12))
    with pytest.raises(ValueError):
        ob.make_rope(64, frequency=[1.0] * 31)
    with pytest.raises(ValueError):
        ob.make_rope(64, sections=(32,), axis=[0] * 32)
    with pytest.raises(ValueError):
        ob.make_rope(256)
    with pytest.raises(ob.OasisError):
        ob.make_rope(40)
    with pytest.raises(ob.OasisError):
        ob.make_rope(64, axis=[4] * 32)


def test_tree_words():
    parents = [-1, -1, 0, 2, 1, 3]
    want = [1, 2, 5, 13, 18, 45]
    assert ob.tree_words(parents).tolist() == want and T.words_of(parents) == want
    both = ob.tree_words(torch.tensor([parents, [-1, 0, 1, 2, 3, 4]]))
    assert both.tolist() == [want, [1, 3, 7, 15, 31, 63]] and both.dtype == torch.int64
    chain = ob.tree_words(list(range(-1, 63)))
    assert chain[63].item() == -1 and chain[62].item() == (1 << 63) - 1
    for bad in ([0], [-1, 1], [-1] * 65):
        with pytest.raises(ValueError):
            ob.tree_words(bad)


def test_angles_by_hand():
    assert abs(T.TWO_PI / 2 ** 200 - 2 * math.pi) < 1e-15
    assert abs(T.angle(1, math.pi / 2) - math.pi / 2) < 1e-15
    assert T.angle(0, 1.0) == 0
    assert abs(T.angle(-3, 1.0) + 3) < 1e-15
    assert abs(math.sin(T.angle(10 ** 6, 1.0)) - math.sin(1e6)) < 1e-15


def test_rotation_by_hand():
    x = torch.zeros(2, 1, 128)
    x[:, 0, 0], x[:, 0, 16], x[:, 0, 1], x[:, 0, 40] = 1.0, 2.0, 3.0, 4.0
    r = ob.make_rope(32, frequency=[math.pi / 2] + [0.0] * 15)
    y, _ = T.rotate(x, torch.tensor([0, 1]), r)
    assert y[0, 0, [0, 16, 1, 40]].tolist() == [1, 2, 3, 4]
    assert np.abs(y[1, 0, [0, 16, 1, 40]] - [-2, 1, 3, 4]).max() < 1e-15
    r = ob.make_rope(32, frequency=[math.pi / 2] + [0.0] * 15, interleaved=True, scale=0.5)
    y, _ = T.rotate(x, torch.tensor([1, 0]), r)
    assert np.abs(y[0, 0, [0, 1, 16, 40]] - [-1.5, 0.5, 1, 4]).max() < 1e-15


def test_keep_by_hand():
    pages = np.arange(3 * Q.UNIT, dtype=np.int64).reshape(3, 1, Q.UNIT).astype(np.uint8)
    table, nodes = np.array([[2, 0]]), np.array([[1, 3, 3]])
    new = T.keep(pages, table, [18], None, 5, nodes, [3])       # nodes are tokens 13 .. 17
    i = np.arange(128)
    assert np.array_equal(new[2, 0, Q.key_at(13, i)], pages[2, 0, Q.key_at(14, i)])
    assert np.array_equal(new[2, 0, Q.value_at(14, i)], pages[0, 0, Q.value_at(0, i)])
    assert np.array_equal(new[2, 0, Q.value_at(15, i)], pages[0, 0, Q.value_at(0, i)])
    assert new[2, 0, 4096 + 13] == pages[2, 0, 4096 + 14] and np.array_equal(new[[0, 1]], pages[[0, 1]])
    assert (new != pages).sum() <= 3 * 258


def test_attention_by_hand():
    """One query head over a context token and two nodes that do not see each other."""
    k = torch.zeros(3, 1, 128)
    v = torch.zeros(3, 1, 128)
    v[0], v[1], v[2] = 1.0, 2.0, 4.0
    pages = np.zeros((1, 1, Q.UNIT), dtype=np.uint8)
    Q.write(pages, k, v, torch.arange(3))
    q = torch.zeros(1, 2, 1, 128)
    o, b, node = T.attention(q, [[1, 2]], None, pages, [[0]], [3])
    assert np.allclose(o[0, :, 0, 0], [1.5, 2.5]) and node.all() and (b < 0.01).all()
    o, _, node = T.attention(q, [[3, 2]], [1], pages, [[0]], [3])   # the last token is the one node
    assert np.allclose(o[0, 0, 0], 7 / 3) and node.tolist() == [[True, False]]
    o, _, _ = T.attention(q, [[0, 0]], None, pages, [[0]], [2])
    assert (o == 0).all()


def test_logprobs_by_hand():
    x = torch.tensor([[0.0, math.log(2.0), -math.inf, math.log(2.0)]])
    lp, H, ids, top = T.logprobs(x, [3], 5)
    assert abs(lp[0] - math.log(0.4)) < 1e-7 and ids[0].tolist() == [1, 3, 0, 2, -1]
    assert abs(H[0] + 0.2 * math.log(0.2) + 0.8 * math.log(0.4)) < 1e-7
    assert abs(top[0, 2] - math.log(0.2)) < 1e-7 and top[0, 3] == -math.inf and top[0, 4] == -math.inf
    assert np.isnan(T.logprobs(torch.full((1, 3), -math.inf), [0], 1)[0]).all()

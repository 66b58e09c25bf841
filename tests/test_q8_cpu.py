"""The 8-bit cache's calls without a GPU: sizes, configuration errors, refused
arguments (all checked before any device work), and the 64-bit definitions
against hand-made cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__
from sparse_kv_block_gb300 import oasis as ob
from tests import _q8 as Q


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()


def cfg(**kw):
    return ob.make_q8_config(**{**dict(num_pages=10, max_blocks=4, Hq=8, Hkv=2), **kw})


def test_sizes():
    s = ob.oasis_q8_query_sizes(cfg())
    assert s.pages_bytes == 10 * 2 * 4128 and s.workspace_bytes % 256 == 0
    big = ob.oasis_q8_query_sizes(cfg(num_pages=1 << 27, Hkv=8, Hq=32))
    assert big.pages_bytes == (1 << 27) * 8 * 4128


@pytest.mark.parametrize("field,value,msg", [
    ("num_pages", 0, "num_pages"), ("num_pages", (1 << 27) + 1, "num_pages"),
    ("max_blocks", 0, "max_blocks"), ("max_blocks", 131073, "max_blocks"),
    ("num_q_heads", 0, "head counts"), ("num_q_heads", 9, "multiple"),
    ("num_q_heads", 18, "per KV head"), ("head_dim", 64, "head_dim"),
    ("block_size", 32, "block_size"), ("softmax_scale", -1.0, "softmax_scale"),
    ("softmax_scale", math.inf, "softmax_scale"), ("softmax_scale", math.nan, "softmax_scale"),
    ("out_fp32", 2, "out_fp32"), ("device", -1, "device"),
])
def test_config_errors(field, value, msg):
    c = cfg()
    assert ob.oasis_q8_config_error(c) is None
    setattr(c, field, value)
    assert msg in ob.oasis_q8_config_error(c)
    with pytest.raises(ob.OasisError):
        ob.oasis_q8_query_sizes(c)
    h = ctypes.c_void_p(1)
    assert ob.lib().oasis_q8_init(ctypes.byref(c), 4096, 4096, ctypes.byref(h)) == ob.OASIS_EINVAL
    assert h.value is None


def test_null_and_misaligned_arguments():
    L, h, c = ob.lib(), ctypes.c_void_p(), cfg()
    for pages, ws in [(None, 4096), (4096, None), (4104, 4096), (4096, 4112)]:
        assert L.oasis_q8_init(ctypes.byref(c), pages, ws, ctypes.byref(h)) == ob.OASIS_EINVAL
        assert h.value is None
    assert L.oasis_q8_write(None, 16, 16, 0, 256, 256, 16, 1, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_read(None, 1, 16, 16, 16, 0, 1, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_attn(None, 1, 1, 0, 16, 0, 16, 16, 16, None, 0, None) == ob.OASIS_EINVAL
    assert L.oasis_prefix_attn(None, 1, 1, 0, 16, 0, 16, 1, 1, 16, 16, 16, None, 0, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_attn_workspace(None, 1, 1, None) == ob.OASIS_EINVAL
    assert L.oasis_prefix_workspace(None, 1, 1, 1, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_sync(None, None) == ob.OASIS_EINVAL
    assert L.oasis_q8_set_wait_limit(None, 5) == ob.OASIS_EINVAL
    assert L.oasis_q8_last_error(None) == b"null handle"
    assert L.oasis_q8_destroy(None) == ob.OASIS_OK
    assert L.oasis_verify_drafts(None, None) == ob.OASIS_EINVAL


def verify_args(**kw):
    a = ob.oasis_verify_args(2, 3, 100, ob.OASIS_FP32, 0, 4096, 4096, 100, 100, 4096, None, 4096,
                             4096, 4096, 4096)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,msg", [
    (dict(num_requests=-1), "num_requests"), (dict(num_requests=(1 << 20) + 1), "num_requests"),
    (dict(num_drafts=-1), "num_drafts"), (dict(num_drafts=65), "num_drafts"),
    (dict(vocab=0), "vocab"), (dict(vocab=(1 << 20) + 1), "vocab"), (dict(type=3), "type"),
    (dict(type=-1), "type"), (dict(device=-1), "device"), (dict(target=None), "null"),
    (dict(tokens=None), "null"), (dict(u_accept=None), "null"), (dict(u_sample=None), "null"),
    (dict(out_tokens=None), "null"), (dict(n_accept=None), "null"),
    (dict(target_stride=99), "target_stride"), (dict(draft_stride=99), "draft_stride"),
    (dict(target=4098), "aligned"), (dict(draft=4097, type=ob.OASIS_BF16), "aligned"),
    (dict(tokens=4098), "aligned"),
])
def test_verify_refusals(change, msg):
    a = verify_args(**change)
    assert msg in ob.lib().oasis_verify_error(ctypes.byref(a)).decode()
    assert ob.lib().oasis_verify_drafts(ctypes.byref(a), None) == ob.OASIS_EINVAL


def test_verify_accepts():
    L = ob.lib()
    for a in (verify_args(), verify_args(draft=None, draft_stride=0),
              verify_args(num_drafts=0, tokens=None, u_accept=None, draft_stride=0),
              verify_args(num_requests=0, target=None)):
        assert L.oasis_verify_error(ctypes.byref(a)) is None
    assert L.oasis_verify_drafts(ctypes.byref(verify_args(num_requests=0, target=None)), None) == ob.OASIS_OK


def test_table_is_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, Q.TABLE, equal_nan=True)


def test_rounding_by_hand():
    x = torch.zeros(6, 128)
    x[0, 0], x[0, 1] = 448.0, 1.0625            # e = 0; 1.0625 ties between 1 and 1.125
    x[1, 0], x[1, 1] = 448.1, -1.0              # just past 448: e = 1
    x[2, 0], x[2, 1] = math.inf, 3.5            # finite maximum 3.5 = 448 * 2^-7
    x[3, 0], x[3, 1] = math.nan, 1e-44          # e held at -100
    c, e, nan = Q.quantise(x)
    assert e.tolist() == [0, 1, -7, -100, -100, -100]
    assert Q.TABLE[c[0, 0]] == 448 and Q.TABLE[c[0, 1]] == 1.0
    assert Q.TABLE[c[1, 0]] == 224 and Q.TABLE[c[1, 1]] == -0.5
    assert Q.TABLE[c[2, 0]] == 448 and Q.TABLE[c[2, 1]] == 448
    assert nan[3, 0] and Q.TABLE[c[3, 1]] == 0
    assert c[4].tolist() == [0] * 128


def test_every_byte_of_a_unit_has_one_meaning():
    seen = np.zeros(Q.UNIT, dtype=int)
    i = np.arange(128)
    for j in range(16):
        seen[Q.key_at(j, i)] += 1
        seen[Q.value_at(j, i)] += 1
        seen[[4096 + j, 4112 + j]] += 1
    assert (seen == 1).all()


def test_verify_definition_by_hand():
    p = torch.tensor([[[0.5, 0.3, 0.2], [0.1, 0.6, 0.3]]])
    q = torch.tensor([[[0.25, 0.75, 0.0]]])
    def go(x, ua, us):
        o, a = Q.verify(p, q, torch.tensor([[x]]), torch.tensor([[ua]]), torch.tensor([us]))
        return o[0].tolist(), int(a[0])
    assert go(0, 0.99, 0.65) == ([0, 1], 1)      # 0.99 * 0.25 < 0.5; then 0.1, 0.7: token 1
    assert go(1, 0.41, 0.55) == ([0, -1], 0)     # 0.3075 > 0.3: refused; left 0.25, 0, 0.2
    assert go(1, 0.41, 0.56) == ([2, -1], 0)
    assert go(1, 0.39, 0.0) == ([1, 0], 1)
    assert go(3, 0.1, 0.1) == ([-1, -1], -1)

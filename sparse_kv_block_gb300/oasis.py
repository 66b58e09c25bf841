"""ctypes binding of the C ABI in ``include/oasis.h`` (``liboasis.so``).

Every function here marshals arguments and calls the library; all device
work runs in the library's CUDA kernels.  PyTorch is used only to allocate
device / pinned memory and to name streams.  If the library is missing the
import fails loudly: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
from ctypes import POINTER, c_char_p, c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_uint32, c_void_p
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liboasis.so")

OASIS_OK, OASIS_EINVAL, OASIS_ENOMEM, OASIS_ECUDA = 0, -1, -2, -3
OASIS_ETIMEOUT, OASIS_ESTATE, OASIS_EDEVICE = -4, -5, -6
STATUS_NAMES = {0: "OK", -1: "EINVAL", -2: "ENOMEM", -3: "ECUDA", -4: "ETIMEOUT",
                -5: "ESTATE", -6: "EDEVICE"}


class oasis_config(ctypes.Structure):
    _fields_ = [("num_layers", c_int32), ("num_requests", c_int32), ("max_blocks", c_int32),
                ("num_q_heads", c_int32), ("num_kv_heads", c_int32), ("head_dim", c_int32),
                ("block_size", c_int32), ("topk", c_int32), ("fetch_ratio", c_float),
                ("softmax_scale", c_float), ("out_fp32", c_int32), ("device", c_int32),
                ("side_groups", c_int32), ("schedule", c_int32), ("num_drafts", c_int32)]


SCHEDULE_SCAN_FIRST, SCHEDULE_CONCURRENT, SCHEDULE_THREE_STREAMS, SCHEDULE_AUTO = 0, 1, 2, 3
SCHEDULE_EARLY_SCAN = 4


class oasis_sizes(ctypes.Structure):
    _fields_ = [("kv_pool_bytes", c_size_t), ("summaries_bytes", c_size_t),
                ("host_kv_bytes", c_size_t), ("res_ids_bytes", c_size_t),
                ("stamps_bytes", c_size_t), ("phys_bytes", c_size_t),
                ("ctx_len_bytes", c_size_t), ("workspace_bytes", c_size_t),
                ("fetch_cap", c_int32), ("units_per_head", c_int32)]


class oasis_buffers(ctypes.Structure):
    _fields_ = [("kv_pool", POINTER(c_void_p)), ("summaries", POINTER(c_void_p)),
                ("host_kv", POINTER(c_void_p)), ("res_ids", POINTER(c_void_p)),
                ("stamps", POINTER(c_void_p)), ("phys", POINTER(c_void_p)),
                ("ctx_len", c_void_p), ("workspace", c_void_p)]


class oasis_remote_config(ctypes.Structure):
    _fields_ = [("capacity", c_int32), ("gbps", c_float), ("threads", c_int32)]


class oasis_remote_sizes(ctypes.Structure):
    _fields_ = [("local_tier_bytes", c_size_t), ("local_map_bytes", c_size_t),
                ("miss_lists_bytes", c_size_t)]


class oasis_q8_config(ctypes.Structure):
    _fields_ = [("num_pages", c_int32), ("max_blocks", c_int32), ("num_q_heads", c_int32),
                ("num_kv_heads", c_int32), ("head_dim", c_int32), ("block_size", c_int32),
                ("softmax_scale", c_float), ("out_fp32", c_int32), ("device", c_int32)]


class oasis_q8_sizes(ctypes.Structure):
    _fields_ = [("pages_bytes", c_size_t), ("workspace_bytes", c_size_t)]


class oasis_verify_args(ctypes.Structure):
    _fields_ = [("num_requests", c_int32), ("num_drafts", c_int32), ("vocab", c_int32),
                ("type", c_int32), ("device", c_int32), ("target", c_void_p),
                ("draft", c_void_p), ("target_stride", c_int64), ("draft_stride", c_int64),
                ("tokens", c_void_p), ("n_drafts", c_void_p), ("u_accept", c_void_p),
                ("u_sample", c_void_p), ("out_tokens", c_void_p), ("n_accept", c_void_p)]


class oasis_rope(ctypes.Structure):
    _fields_ = [("rot_dim", c_int32), ("num_axes", c_int32), ("interleaved", c_int32),
                ("scale", c_float), ("frequency", c_double * 64), ("axis", c_int32 * 64)]


class oasis_logprobs_args(ctypes.Structure):
    _fields_ = [("num_rows", c_int32), ("vocab", c_int32), ("type", c_int32), ("top", c_int32),
                ("device", c_int32), ("logits", c_void_p), ("stride", c_int64),
                ("tokens", c_void_p), ("logprobs", c_void_p), ("entropy", c_void_p),
                ("top_ids", c_void_p), ("top_logprobs", c_void_p)]


_LOGPROBS_ARGS = struct.Struct("@5iPqPPPPP")
assert _LOGPROBS_ARGS.size == ctypes.sizeof(oasis_logprobs_args)
_VERIFY_ARGS = struct.Struct("@5iPPqqPPPPPP")
assert _VERIFY_ARGS.size == ctypes.sizeof(oasis_verify_args)

OASIS_BF16, OASIS_FP16, OASIS_FP32 = 0, 1, 2
_TYPES = {torch.bfloat16: OASIS_BF16, torch.float16: OASIS_FP16, torch.float32: OASIS_FP32}
Q8_UNIT_BYTES = 4128  # one KV head's block of 16 tokens in the 8-bit cache

DEVERR_NOT_LOCAL = 0x8


class OasisError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


# Declared exports: name -> (restype, argtypes).  Tests check this list against
# include/oasis.h.
_P = c_void_p
EXPORTS = {
    "oasis_config_error": (c_char_p, [POINTER(oasis_config)]),
    "oasis_query_sizes": (c_int, [POINTER(oasis_config), POINTER(oasis_sizes)]),
    "oasis_init": (c_int, [POINTER(oasis_config), POINTER(oasis_buffers), POINTER(c_void_p)]),
    "oasis_destroy": (c_int, [_P]),
    "oasis_last_error": (c_char_p, [_P]),
    "oasis_sync": (c_int, [_P, POINTER(c_uint32)]),
    "oasis_build_summaries": (c_int, [_P, c_int, c_int, _P]),
    "oasis_load_resident": (c_int, [_P, c_int, c_int, _P]),
    "oasis_resume_resident": (c_int, [_P, c_int, c_int, _P]),
    "oasis_lookahead_attn": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P]),
    "oasis_dense_attn": (c_int, [_P, _P, c_int, _P, _P, _P, _P, _P]),
    "oasis_score_topk": (c_int, [_P, c_int, c_int, _P, _P, _P, _P]),
    "oasis_admit_evict": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P, _P]),
    "oasis_score_admit_noalloc": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P, _P]),
    "oasis_prefetch": (c_int, [_P, c_int, c_int, _P, _P, _P, _P]),
    "oasis_step": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P]),
    "oasis_wait": (c_int, [_P, c_int, c_double]),
    "oasis_join": (c_int, [_P, c_int, _P]),
    "oasis_step_host": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P]),
    "oasis_step_host_async": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P]),
    "oasis_wait_outputs": (c_int, [_P, c_int, c_int, c_double]),
    "oasis_step_lists": (c_int, [_P, c_int, c_int, POINTER(c_void_p), POINTER(c_void_p),
                                 POINTER(c_void_p), POINTER(c_void_p), POINTER(c_void_p),
                                 POINTER(c_void_p)]),
    "oasis_append_token": (c_int, [_P, c_int, c_int, _P, _P, _P]),
    "oasis_refresh_blocks": (c_int, [_P, c_int, c_int, _P, _P, c_int, _P]),
    "oasis_advance_context": (c_int, [_P, c_int, c_int, _P]),
    "oasis_remote_query_sizes": (c_int, [POINTER(oasis_config), POINTER(oasis_remote_config),
                                         POINTER(oasis_remote_sizes)]),
    "oasis_remote_attach": (c_int, [_P, c_int, POINTER(oasis_remote_config), _P, _P, _P]),
    "oasis_remote_stats": (c_int, [_P, c_int, POINTER(c_int64), POINTER(c_int64),
                                   POINTER(c_double), POINTER(c_int64)]),
    "oasis_demand_topk": (c_int, [_P, c_int, c_int, _P, _P, _P, _P]),
    "oasis_admit_demand": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P, _P]),
    "oasis_fetch_demand": (c_int, [_P, c_int, c_int, _P, _P, _P, _P]),
    "oasis_step_stall": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P]),
    "oasis_stall_lists": (c_int, [_P, c_int, c_int, POINTER(c_void_p), POINTER(c_void_p),
                                  POINTER(c_void_p), POINTER(c_void_p), POINTER(c_void_p),
                                  POINTER(c_void_p)]),
    "oasis_set_wait_limit": (c_int, [_P, ctypes.c_longlong]),
    "oasis_profile_enable": (c_int, [_P, c_int]),
    "oasis_profile_read_n": (c_int, [_P, c_int, POINTER(c_double), POINTER(c_int64),
                                     POINTER(c_double)]),
    "oasis_profile_read": (c_int, [_P, POINTER(c_double), POINTER(c_int64), POINTER(c_double)]),
    "oasis_q8_config_error": (c_char_p, [POINTER(oasis_q8_config)]),
    "oasis_q8_query_sizes": (c_int, [POINTER(oasis_q8_config), POINTER(oasis_q8_sizes)]),
    "oasis_q8_init": (c_int, [POINTER(oasis_q8_config), _P, _P, POINTER(c_void_p)]),
    "oasis_q8_destroy": (c_int, [_P]),
    "oasis_q8_last_error": (c_char_p, [_P]),
    "oasis_q8_sync": (c_int, [_P, POINTER(c_uint32)]),
    "oasis_q8_set_wait_limit": (c_int, [_P, ctypes.c_longlong]),
    "oasis_q8_write": (c_int, [_P, _P, _P, c_int, c_int64, c_int64, _P, c_int, _P]),
    "oasis_q8_read": (c_int, [_P, c_int, _P, _P, _P, c_int, c_int, _P]),
    "oasis_q8_attn": (c_int, [_P, c_int, c_int, c_int, _P, c_int, _P, _P, _P, _P, c_size_t, _P]),
    "oasis_q8_attn_workspace": (c_int, [_P, c_int, c_int, POINTER(c_size_t)]),
    "oasis_prefix_workspace": (c_int, [_P, c_int, c_int, c_int, POINTER(c_size_t)]),
    "oasis_prefix_attn": (c_int, [_P, c_int, c_int, c_int, _P, c_int, _P, c_int, c_int, _P, _P,
                                  _P, _P, c_size_t, _P]),
    "oasis_verify_error": (c_char_p, [_P]),
    "oasis_verify_drafts": (c_int, [_P, _P]),
    "oasis_rope_error": (c_char_p, [POINTER(oasis_rope)]),
    "oasis_q8_append": (c_int, [_P, POINTER(oasis_rope), _P, _P, _P, _P, c_int, c_int64, c_int64,
                                c_int64, c_int64, _P, _P, c_int, _P]),
    "oasis_q8_tree_attn": (c_int, [_P, c_int, c_int, _P, c_int, _P, _P, _P, _P, _P, _P, c_size_t, _P]),
    "oasis_q8_tree_workspace": (c_int, [_P, c_int, c_int, c_int, POINTER(c_size_t)]),
    "oasis_q8_keep": (c_int, [_P, c_int, c_int, _P, _P, _P, _P, _P, c_int, _P]),
    "oasis_logprobs_error": (c_char_p, [_P]),
    "oasis_token_logprobs": (c_int, [_P, _P]),
}

PROFILE_KINDS = ["attention", "score_topk", "admit_evict", "prefetch", "demand_score",
                 "demand_gather", "topk_select"]

_lib = None


def lib():
    """Load liboasis.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        import torch.cuda  # noqa: F401  (loads the CUDA runtime the library links)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _stream(s) -> Optional[int]:
    if s is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def make_config(R, NBmax, Hq, Hkv, K, fetch_ratio, layers=1, softmax_scale=0.0,
                out_fp32=False, device=0, d=128, B=16, side_groups=0,
                schedule=SCHEDULE_AUTO, num_drafts=1) -> oasis_config:
    """``num_drafts`` D: draft queries per step; q_draft / out_draft then hold
    D planes ``[D][R][Hq][d]`` (a ``[R][Hq][d]`` tensor is the one-draft case).
    ``schedule``: one of SCHEDULE_*; with SCHEDULE_EARLY_SCAN the device-buffer
    oasis_step reads q_draft when it is called, so it must be complete then."""
    return oasis_config(layers, R, NBmax, Hq, Hkv, d, B, K, fetch_ratio, softmax_scale,
                        1 if out_fp32 else 0, device, side_groups, schedule, num_drafts)


def oasis_config_error(cfg: oasis_config) -> Optional[str]:
    m = lib().oasis_config_error(ctypes.byref(cfg))
    return None if m is None else m.decode()


def oasis_query_sizes(cfg: oasis_config) -> oasis_sizes:
    out = oasis_sizes()
    rc = lib().oasis_query_sizes(ctypes.byref(cfg), ctypes.byref(out))
    if rc != OASIS_OK:
        raise OasisError(rc, oasis_config_error(cfg) or "query_sizes failed")
    return out


def oasis_remote_query_sizes(cfg: oasis_config, rcfg: oasis_remote_config) -> oasis_remote_sizes:
    out = oasis_remote_sizes()
    rc = lib().oasis_remote_query_sizes(ctypes.byref(cfg), ctypes.byref(rcfg), ctypes.byref(out))
    if rc != OASIS_OK:
        raise OasisError(rc, "remote_query_sizes: bad config or remote config")
    return out


class Oasis:
    """A library context plus the caller-owned buffers it was given.

    Buffers are allocated with torch (device memory and pinned host memory
    for the KV store unless ``host_kv`` tensors are passed in) and kept alive
    here.  Methods map one-to-one onto the C ABI calls.
    """

    def __init__(self, cfg: oasis_config, host_kv: Optional[Sequence[torch.Tensor]] = None):
        self.cfg = cfg
        self.sizes = oasis_query_sizes(cfg)
        L, R, Hkv = cfg.num_layers, cfg.num_requests, cfg.num_kv_heads
        K, U, NB = cfg.topk, self.sizes.units_per_head, cfg.max_blocks
        self.C, self.U = self.sizes.fetch_cap, U
        dev = torch.device("cuda", cfg.device)
        self.device = dev
        if host_kv is None:
            host_kv = [torch.zeros((R, Hkv, NB, 2, 16, 128), dtype=torch.bfloat16,
                                   pin_memory=True) for _ in range(L)]
        if len(host_kv) != L:
            raise ValueError("need one host store per layer")
        for t in host_kv:
            if t.numel() * t.element_size() != self.sizes.host_kv_bytes or not t.is_pinned():
                raise ValueError("host_kv must be pinned and of host_kv_bytes")
        self.host_kv = list(host_kv)
        self.kv_pool = [torch.zeros((R, Hkv, U, 2, 16, 128), dtype=torch.bfloat16, device=dev)
                        for _ in range(L)]
        self.summaries = [torch.zeros((R, Hkv, NB, 2, 128), dtype=torch.bfloat16, device=dev)
                          for _ in range(L)]
        self.res_ids = [torch.full((2, R, Hkv, K), -1, dtype=torch.int32, device=dev)
                        for _ in range(L)]
        self.stamps = [torch.full((R, Hkv, K), -1, dtype=torch.int32, device=dev)
                       for _ in range(L)]
        self.phys = [torch.zeros((2, R, Hkv, U), dtype=torch.int32, device=dev) for _ in range(L)]
        self.ctx_len = torch.zeros((2, R), dtype=torch.int32, device=dev)
        self.workspace = torch.zeros(self.sizes.workspace_bytes, dtype=torch.uint8, device=dev)

        def arr(ts):
            a = (c_void_p * L)(*[t.data_ptr() for t in ts])
            return a
        self._arrs = [arr(self.kv_pool), arr(self.summaries), arr(self.host_kv),
                      arr(self.res_ids), arr(self.stamps), arr(self.phys)]
        bufs = oasis_buffers(*[ctypes.cast(a, POINTER(c_void_p)) for a in self._arrs],
                             self.ctx_len.data_ptr(), self.workspace.data_ptr())
        handle = c_void_p()
        torch.cuda.synchronize(dev)
        rc = lib().oasis_init(ctypes.byref(cfg), ctypes.byref(bufs), ctypes.byref(handle))
        if rc != OASIS_OK:
            raise OasisError(rc, oasis_config_error(cfg) or "oasis_init failed "
                             "(buffers not pinned/mapped, or CUDA error)")
        self.ctx = handle.value

    # ------------------------------------------------------------------ util
    def _check(self, rc: int) -> None:
        if rc != OASIS_OK:
            raise OasisError(rc, lib().oasis_last_error(self.ctx).decode())

    def close(self) -> None:
        if getattr(self, "ctx", None):
            lib().oasis_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------ C ABI calls
    def oasis_sync(self) -> int:
        bits = c_uint32(0)
        rc = lib().oasis_sync(self.ctx, ctypes.byref(bits))
        if rc not in (OASIS_OK, OASIS_EDEVICE):
            self._check(rc)
        if rc == OASIS_EDEVICE:
            raise OasisError(rc, f"device error bits 0x{bits.value:x}")
        return bits.value

    def oasis_build_summaries(self, layer: int, table: int = 0, stream=None) -> None:
        self._check(lib().oasis_build_summaries(self.ctx, layer, table, _stream(stream)))

    def oasis_load_resident(self, layer: int, first_step: int = 0, stream=None) -> None:
        self._check(lib().oasis_load_resident(self.ctx, layer, first_step, _stream(stream)))

    def oasis_resume_resident(self, layer: int, first_step: int, stream=None) -> None:
        self._check(lib().oasis_resume_resident(self.ctx, layer, first_step, _stream(stream)))

    def _sized(self, q=None, qd=None, out=None, outd=None) -> None:
        """Refuse torch tensors smaller than the call reads or writes (the
        library takes plain pointers and cannot check their extent)."""
        c = self.cfg
        D = c.num_drafts if c.num_drafts > 0 else 1
        qb = c.num_requests * c.num_q_heads * c.head_dim * 2
        ob = qb * (2 if c.out_fp32 else 1)
        for name, x, need in (("q", q, qb), ("q_draft", qd, D * qb), ("out", out, ob),
                              ("out_draft", outd, D * ob)):
            if isinstance(x, torch.Tensor) and x.numel() * x.element_size() < need:
                raise ValueError(f"{name} holds {x.numel() * x.element_size()} bytes, "
                                 f"the call needs {need}")

    def oasis_lookahead_attn(self, layer, step, q, qd, out, outd, stream=None) -> None:
        self._sized(q, qd, out, outd)
        self._check(lib().oasis_lookahead_attn(self.ctx, layer, step, _ptr(q), _ptr(qd),
                                               _ptr(out), _ptr(outd), _stream(stream)))

    def oasis_dense_attn(self, kv_dense, table, q, qd, out, outd, stream=None) -> None:
        self._sized(q, qd, out, outd)
        self._check(lib().oasis_dense_attn(self.ctx, _ptr(kv_dense), table, _ptr(q), _ptr(qd),
                                           _ptr(out), _ptr(outd), _stream(stream)))

    def oasis_score_topk(self, layer, step, qd, topk_ids, topk_scores=None, stream=None) -> None:
        self._sized(qd=qd)
        self._check(lib().oasis_score_topk(self.ctx, layer, step, _ptr(qd), _ptr(topk_ids),
                                           _ptr(topk_scores), _stream(stream)))

    def oasis_admit_evict(self, layer, step, topk_ids, admit_ids, admit_slots, evict_ids,
                          n_admit, stream=None) -> None:
        self._check(lib().oasis_admit_evict(self.ctx, layer, step, _ptr(topk_ids),
                                            _ptr(admit_ids), _ptr(admit_slots),
                                            _ptr(evict_ids), _ptr(n_admit), _stream(stream)))

    def oasis_score_admit_noalloc(self, layer, step, qd, admit_ids, admit_slots, evict_ids,
                                  n_admit, stream=None) -> None:
        self._sized(qd=qd)
        self._check(lib().oasis_score_admit_noalloc(self.ctx, layer, step, _ptr(qd),
                                                    _ptr(admit_ids), _ptr(admit_slots),
                                                    _ptr(evict_ids), _ptr(n_admit),
                                                    _stream(stream)))

    def oasis_prefetch(self, layer, step, admit_ids, admit_slots, n_admit, stream=None) -> None:
        self._check(lib().oasis_prefetch(self.ctx, layer, step, _ptr(admit_ids),
                                         _ptr(admit_slots), _ptr(n_admit), _stream(stream)))

    def oasis_step(self, layer, step, q, qd, out, outd, stream=None) -> None:
        self._sized(q, qd, out, outd)
        self._check(lib().oasis_step(self.ctx, layer, step, _ptr(q), _ptr(qd), _ptr(out),
                                     _ptr(outd), _stream(stream)))

    def oasis_demand_topk(self, layer, step, q, topk_ids, topk_scores=None, stream=None) -> None:
        self._sized(q=q)
        self._check(lib().oasis_demand_topk(self.ctx, layer, step, _ptr(q), _ptr(topk_ids),
                                            _ptr(topk_scores), _stream(stream)))

    def oasis_admit_demand(self, layer, step, topk_ids, admit_ids, admit_slots, evict_ids,
                           n_admit, stream=None) -> None:
        """Lists [R][Hkv][K] int32 and n_admit [R][Hkv] int32 (device)."""
        self._check(lib().oasis_admit_demand(self.ctx, layer, step, _ptr(topk_ids),
                                             _ptr(admit_ids), _ptr(admit_slots),
                                             _ptr(evict_ids), _ptr(n_admit), _stream(stream)))

    def oasis_fetch_demand(self, layer, step, admit_ids, admit_slots, n_admit,
                           stream=None) -> None:
        self._check(lib().oasis_fetch_demand(self.ctx, layer, step, _ptr(admit_ids),
                                             _ptr(admit_slots), _ptr(n_admit), _stream(stream)))

    def oasis_step_stall(self, layer, step, q, qd, out, outd, stream=None) -> None:
        self._sized(q, qd, out, outd)
        self._check(lib().oasis_step_stall(self.ctx, layer, step, _ptr(q), _ptr(qd), _ptr(out),
                                           _ptr(outd), _stream(stream)))

    def oasis_stall_lists(self, layer: int, step: int) -> dict:
        ps = [c_void_p() for _ in range(6)]
        self._check(lib().oasis_stall_lists(self.ctx, layer, step,
                                            *[ctypes.byref(p) for p in ps]))
        return dict(zip(["topk_ids", "topk_scores", "admit_ids", "admit_slots", "evict_ids",
                         "n_admit"], [p.value for p in ps]))

    def oasis_wait(self, layer: int, timeout_ms: float) -> bool:
        """True when the layer's side work is done, False on timeout."""
        rc = lib().oasis_wait(self.ctx, layer, float(timeout_ms))
        if rc == OASIS_ETIMEOUT:
            return False
        self._check(rc)
        return True

    def oasis_join(self, layer, stream=None) -> None:
        self._check(lib().oasis_join(self.ctx, layer, _stream(stream)))

    def oasis_step_host(self, layer, step, q_host, qd_host, out_host, outd_host,
                        stream=None) -> None:
        self._sized(q_host, qd_host, out_host, outd_host)
        self._check(lib().oasis_step_host(self.ctx, layer, step, _ptr(q_host), _ptr(qd_host),
                                          _ptr(out_host), _ptr(outd_host), _stream(stream)))

    def oasis_step_host_async(self, layer, step, q_host, qd_host, out_host, outd_host,
                              stream=None) -> None:
        self._sized(q_host, qd_host, out_host, outd_host)
        self._check(lib().oasis_step_host_async(self.ctx, layer, step, _ptr(q_host),
                                                _ptr(qd_host), _ptr(out_host), _ptr(outd_host),
                                                _stream(stream)))

    def oasis_wait_outputs(self, layer: int, step: int, timeout_ms: float) -> bool:
        """True when the outputs of host-buffer step `step` are in host
        memory, False on timeout."""
        rc = lib().oasis_wait_outputs(self.ctx, layer, step, float(timeout_ms))
        if rc == OASIS_ETIMEOUT:
            return False
        self._check(rc)
        return True

    def oasis_step_lists(self, layer: int, step: int) -> dict:
        ps = [c_void_p() for _ in range(6)]
        self._check(lib().oasis_step_lists(self.ctx, layer, step,
                                           *[ctypes.byref(p) for p in ps]))
        return dict(zip(["topk_ids", "topk_scores", "admit_ids", "admit_slots", "evict_ids",
                         "n_admit"], [p.value for p in ps]))

    def oasis_append_token(self, layer, step, k_new, v_new, stream=None) -> None:
        self._check(lib().oasis_append_token(self.ctx, layer, step, _ptr(k_new), _ptr(v_new),
                                             _stream(stream)))

    def oasis_refresh_blocks(self, layer, step, ids, n_ids, stream=None) -> None:
        """ids: int32 [R][Hkv][max_ids] (device), n_ids: int32 [R][Hkv] (device)."""
        self._check(lib().oasis_refresh_blocks(self.ctx, layer, step, _ptr(ids), _ptr(n_ids),
                                               int(ids.shape[-1]), _stream(stream)))

    def oasis_advance_context(self, step, grow=1, stream=None) -> None:
        self._check(lib().oasis_advance_context(self.ctx, step, grow, _stream(stream)))

    def oasis_remote_attach(self, layer: int, capacity: int, gbps: float = 0.0,
                            threads: int = 0) -> dict:
        """Allocate the remote tier's buffers (pinned local tier and miss
        lists, device local map), attach them to `layer` and return them as
        tensors: local_tier [R][Hkv][capacity][2][16][128] bf16, local_map
        [R][Hkv][NBmax] int32, local_count [R][Hkv] int32 (a view into the
        same buffer), miss_lists (flat int32)."""
        rcfg = oasis_remote_config(capacity, gbps, threads)
        sz = oasis_remote_query_sizes(self.cfg, rcfg)
        R, Hkv, NB = self.cfg.num_requests, self.cfg.num_kv_heads, self.cfg.max_blocks
        local = torch.zeros((R, Hkv, capacity, 2, 16, 128), dtype=torch.bfloat16,
                            pin_memory=True)
        assert local.numel() * 2 == sz.local_tier_bytes
        mp = torch.empty(sz.local_map_bytes // 4, dtype=torch.int32, device=self.device)
        lists = torch.zeros(sz.miss_lists_bytes // 4, dtype=torch.int32, pin_memory=True)
        self._check(lib().oasis_remote_attach(self.ctx, layer, ctypes.byref(rcfg),
                                              local.data_ptr(), mp.data_ptr(),
                                              lists.data_ptr()))
        pairs = R * Hkv
        M = max(self.cfg.topk, self.C)
        t = dict(local_tier=local, local_map=mp[:pairs * NB].view(R, Hkv, NB),
                 local_count=mp[pairs * NB:pairs * NB + pairs].view(R, Hkv),
                 local_base=mp[pairs * NB + pairs:].view(R, Hkv), miss_lists=lists,
                 n_miss=lists[:pairs].view(R, Hkv),
                 miss_ids=lists[pairs:pairs + pairs * M].view(R, Hkv, M),
                 miss_slots=lists[pairs + pairs * M:pairs + 2 * pairs * M].view(R, Hkv, M))
        if not hasattr(self, "remote"):
            self.remote = {}
        self.remote[layer] = t
        return t

    def oasis_remote_stats(self, layer: int) -> dict:
        u, n, b = c_int64(0), c_int64(0), c_int64(0)
        sec = c_double(0.0)
        self._check(lib().oasis_remote_stats(self.ctx, layer, ctypes.byref(u), ctypes.byref(n),
                                             ctypes.byref(sec), ctypes.byref(b)))
        return dict(units=u.value, transfers=n.value, seconds=sec.value, bad_entries=b.value)

    def oasis_set_wait_limit(self, cycles: int) -> None:
        """Barrier-wait limit of the following launches in clock cycles
        (<= 0: the default, about a second)."""
        self._check(lib().oasis_set_wait_limit(self.ctx, int(cycles)))

    def oasis_profile_enable(self, enable: bool = True) -> None:
        self._check(lib().oasis_profile_enable(self.ctx, 1 if enable else 0))

    def oasis_profile_read(self, nkinds: int = 4) -> tuple:
        """(summed ms, launch counts, summed start offsets in ms) per kernel
        kind, for the first `nkinds` of PROFILE_KINDS."""
        ms = (c_double * nkinds)()
        cnt = (c_int64 * nkinds)()
        off = (c_double * nkinds)()
        self._check(lib().oasis_profile_read_n(self.ctx, nkinds, ms, cnt, off))
        return list(ms), list(cnt), list(off)

    # ------------------------------------------------------- tensor views
    def step_lists(self, layer: int, step: int) -> dict:
        """The workspace lists of oasis_step(layer, step) as torch tensors
        (views, no copy; valid until step + 2 is issued)."""
        return self._list_views(self.oasis_step_lists(layer, step), max(self.C, 1))

    def stall_lists(self, layer: int, step: int) -> dict:
        """The demand lists of oasis_step_stall(layer, step) as torch tensors
        (views, no copy; admission lists [R][Hkv][K])."""
        return self._list_views(self.oasis_stall_lists(layer, step), self.cfg.topk)

    def _list_views(self, p: dict, width: int) -> dict:
        R, Hkv, K = self.cfg.num_requests, self.cfg.num_kv_heads, self.cfg.topk
        out = {}
        for name, shape, dt in [("topk_ids", (R, Hkv, K), torch.int32),
                                ("topk_scores", (R, Hkv, K), torch.float32),
                                ("admit_ids", (R, Hkv, width), torch.int32),
                                ("admit_slots", (R, Hkv, width), torch.int32),
                                ("evict_ids", (R, Hkv, width), torch.int32),
                                ("n_admit", (R, Hkv), torch.int32)]:
            n = 1
            for s in shape:
                n *= s
            off = p[name] - self.workspace.data_ptr()
            es = torch.tensor([], dtype=dt).element_size()
            out[name] = self.workspace[off:off + n * es].view(dt).view(shape)
        return out

    def set_context(self, lens) -> None:
        """Set both ctx_len tables (plain host-to-device copy)."""
        t = torch.as_tensor(lens, dtype=torch.int32)
        self.ctx_len.copy_(t.view(1, -1).expand(2, -1))

    def set_resident(self, layer: int, res, first_step: int = 0) -> None:
        """Write the caller's resident table for `first_step` (host-to-device copy)."""
        self.res_ids[layer][first_step & 1].copy_(torch.as_tensor(res, dtype=torch.int32))


# ------------------------------------------------- decoding over an 8-bit cache
def _want(name: str, t: torch.Tensor, dtype, shape: tuple, device: int) -> int:
    """The address of a contiguous tensor of that type, shape and CUDA device; ValueError
    otherwise.  (On the path of every call: a few hundred nanoseconds.)"""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name} must be {dtype} {list(shape)} on cuda:{device}, got {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream_on(s, device: int) -> int:
    """The handle of stream `s`, or of the device's current stream."""
    if s is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return s if isinstance(s, int) else s.cuda_stream


def make_q8_config(num_pages, max_blocks, Hq, Hkv, softmax_scale=0.0, out_fp32=False, device=0,
                   d=128, B=16) -> oasis_q8_config:
    return oasis_q8_config(num_pages, max_blocks, Hq, Hkv, d, B, softmax_scale,
                           1 if out_fp32 else 0, device)


def oasis_q8_config_error(cfg: oasis_q8_config) -> Optional[str]:
    m = lib().oasis_q8_config_error(ctypes.byref(cfg))
    return None if m is None else m.decode()


def oasis_q8_query_sizes(cfg: oasis_q8_config) -> oasis_q8_sizes:
    out = oasis_q8_sizes()
    rc = lib().oasis_q8_query_sizes(ctypes.byref(cfg), ctypes.byref(out))
    if rc != OASIS_OK:
        raise OasisError(rc, oasis_q8_config_error(cfg) or "q8_query_sizes failed")
    return out


def make_rope(rot_dim=128, base=10000.0, sections=None, frequency=None, axis=None, interleaved=False,
              scale=1.0) -> oasis_rope:
    """A rotation by position.  ``frequency``: radians a position of each of the rot_dim / 2 pairs
    (default base^(-2 i / rot_dim)).  Several position axes (time, height, width): ``sections``,
    the pairs of each axis in order, or ``axis``, each pair's axis."""
    half = rot_dim // 2
    if frequency is None:
        frequency = [float(base) ** (-2.0 * i / rot_dim) for i in range(half)]
    if sections is not None:
        if axis is not None:
            raise ValueError("sections or axis, not both")
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    axis = [0] * half if axis is None else [int(a) for a in axis]
    if len(frequency) != half or len(axis) != half or half > 64:
        raise ValueError(f"a rotation of {rot_dim} dims has {half} pairs (at most 64): got {len(frequency)} "
                         f"frequencies and {len(axis)} axes")
    r = oasis_rope(rot_dim, max(axis, default=0) + 1, 1 if interleaved else 0, scale)
    r.frequency[:half] = [float(f) for f in frequency]
    r.axis[:half] = axis
    m = lib().oasis_rope_error(ctypes.byref(r))
    if m is not None:
        raise OasisError(OASIS_EINVAL, m.decode())
    return r


def tree_words(parents) -> torch.Tensor:
    """The words of oasis_q8_tree_attn, int64 like parents, of trees given by their nodes' parents
    [..., N] (before the node; negative: the context): a node sees its ancestors and itself."""
    p = torch.as_tensor(parents).cpu().long()
    N = p.shape[-1]
    if N > 64 or (p >= torch.arange(N)).any():
        raise ValueError("a tree has up to 64 nodes, and a node's parent stands before it")
    w = torch.zeros(*p.shape[:-1], N + 1, dtype=torch.int64)  # the last: the context's
    for i in range(N):
        up = torch.where(p[..., i] < 0, N, p[..., i]).unsqueeze(-1)
        w[..., i] = w.gather(-1, up).squeeze(-1) | (-(1 << 63) if i == 63 else 1 << i)
    return w[..., :N].contiguous()


class Q8Cache:
    """A handle on an 8-bit paged KV cache: ``pages`` [num_pages][Hkv][4128]
    uint8 (allocated zeroed unless passed in, 16-byte aligned; several handles
    may have the same) and the handle's workspace.
    Methods map one-to-one onto the C ABI calls; tensors of another type,
    shape, device or layout than documented there are refused (ValueError).
    Calls run on ``stream`` (default: the device's current one); tensors
    allocated on another stream have to live until it is done with them.
    """

    def __init__(self, cfg: oasis_q8_config, pages: Optional[torch.Tensor] = None):
        self.q8 = None
        self.cfg = cfg
        self.sizes = oasis_q8_query_sizes(cfg)
        self.device = torch.device("cuda", cfg.device)
        shape = (cfg.num_pages, cfg.num_kv_heads, Q8_UNIT_BYTES)
        if pages is None:
            pages = torch.zeros(shape, dtype=torch.uint8, device=self.device)
        _want("pages", pages, torch.uint8, shape, cfg.device)
        self.pages = pages
        self.workspace = torch.empty(self.sizes.workspace_bytes, dtype=torch.uint8,
                                     device=self.device)
        handle = c_void_p()
        rc = lib().oasis_q8_init(ctypes.byref(cfg), pages.data_ptr(), self.workspace.data_ptr(),
                                 ctypes.byref(handle))
        if rc != OASIS_OK:
            raise OasisError(rc, "oasis_q8_init failed (misaligned pages, or CUDA error)")
        self.q8 = handle.value
        # what every call asks of its tensors, in plain Python values
        self._lib, self._dev = lib(), int(cfg.device)
        self._Hq, self._Hkv, self._max_blocks = int(cfg.num_q_heads), int(cfg.num_kv_heads), int(cfg.max_blocks)
        self._out_fp32 = bool(cfg.out_fp32)
        self._scratch = {}  # bytes that attention over (R, S) can use

    def _check(self, rc: int) -> None:
        if rc != OASIS_OK:
            raise OasisError(rc, lib().oasis_q8_last_error(self.q8).decode())

    def close(self) -> None:
        if getattr(self, "q8", None):
            lib().oasis_q8_destroy(self.q8)
            self.q8 = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def oasis_q8_sync(self) -> int:
        bits = c_uint32(0)
        rc = lib().oasis_q8_sync(self.q8, ctypes.byref(bits))
        if rc == OASIS_EDEVICE:
            raise OasisError(rc, f"device error bits 0x{bits.value:x}")
        self._check(rc)
        return bits.value

    def oasis_q8_set_wait_limit(self, cycles: int) -> None:
        """Barrier-wait limit of the following attention launches in clock cycles (<= 0: the
        default, about a second)."""
        self._check(lib().oasis_q8_set_wait_limit(self.q8, int(cycles)))

    def _rows(self, name: str, x: torch.Tensor, T: int, dtype) -> int:
        """Elements between consecutive tokens of x [T][Hkv][d], whose heads are contiguous."""
        H = self._Hkv
        if x.dtype is not dtype or x.shape != (T, H, 128) or x.get_device() != self._dev:
            raise ValueError(f"{name} must be {dtype} {[T, H, 128]} on {self.device}, got {x.dtype} "
                             f"{list(x.shape)} on {x.device}")
        st = x.stride()
        if T and (st[2] != 1 or (H > 1 and st[1] != 128)):
            raise ValueError(f"{name}: a token's heads must be contiguous")
        return st[0] if T > 1 else 0

    def oasis_q8_write(self, k, v, slots, stream=None) -> None:
        """k, v [T][Hkv][128] bf16, fp16 or fp32 (tokens may be strided), slots [T] int64."""
        T = slots.numel()
        typ = _TYPES.get(k.dtype)
        if typ is None:
            raise ValueError(f"k must be bfloat16, float16 or float32, got {k.dtype}")
        ks, vs = self._rows("k", k, T, k.dtype), self._rows("v", v, T, k.dtype)
        self._check(self._lib.oasis_q8_write(
            self.q8, k.data_ptr(), v.data_ptr(), typ, ks, vs,
            _want("slots", slots, torch.int64, (T,), self._dev), T, _stream_on(stream, self._dev)))

    def _table(self, page_table, seq_len) -> tuple:
        R = seq_len.numel()
        return (R, _want("page_table", page_table, torch.int32, (R, self._max_blocks), self._dev),
                _want("seq_len", seq_len, torch.int32, (R,), self._dev))

    def oasis_q8_read(self, page_table, seq_len, out, stream=None) -> None:
        """out [R][Hkv][out_blocks][2][16][128] bf16, fp16 or fp32."""
        R, table, lens = self._table(page_table, seq_len)
        typ = _TYPES.get(out.dtype)
        if typ is None:
            raise ValueError(f"out must be bfloat16, float16 or float32, got {out.dtype}")
        blocks = out.shape[2] if out.dim() == 6 else -1
        o = _want("out", out, out.dtype, (R, self._Hkv, blocks, 2, 16, 128), self._dev)
        self._check(self._lib.oasis_q8_read(self.q8, R, table, lens, o, typ, blocks,
                                            _stream_on(stream, self._dev)))

    def _queries(self, q, out, R: int) -> tuple:
        dt = q.dtype
        if dt is not torch.bfloat16 and dt is not torch.float16:
            raise ValueError(f"q must be bfloat16 or float16, got {dt}")
        S = q.shape[0] if q.dim() == 4 else -1
        shape = (S, R, self._Hq, 128)
        return (S, _want("q", q, dt, shape, self._dev), _TYPES[dt],
                _want("out", out, torch.float32 if self._out_fp32 else dt, shape, self._dev))

    def oasis_q8_attn_workspace(self, R: int, S: int) -> int:
        n = c_size_t(0)
        rc = lib().oasis_q8_attn_workspace(self.q8, R, S, ctypes.byref(n))
        if rc != OASIS_OK:
            raise OasisError(rc, "q8_attn_workspace: bad size")
        return n.value

    def oasis_q8_attn(self, q, page_table, seq_len, out, causal=False, stream=None, workspace=None) -> None:
        """q, out [S][R][Hq][128].  workspace: scratch of oasis_q8_attn_workspace bytes (uint8),
        by default taken from the allocator for this call (on its stream, so that it is also right
        inside a graph's capture)."""
        R, table, lens = self._table(page_table, seq_len)
        S, qp, typ, o = self._queries(q, out, R)
        st = _stream_on(stream, self._dev)
        if workspace is None:
            n = self._scratch.get((R, S))
            if n is None:
                n = self._scratch[R, S] = self.oasis_q8_attn_workspace(R, S) if 1 <= S <= 4 else 0
            if n:
                workspace = self._scratch_on(n, stream)
        else:
            n = workspace.numel()
        ws = _want("workspace", workspace, torch.uint8, (n,), self._dev) if n else None
        self._check(self._lib.oasis_q8_attn(self.q8, R, S, 1 if causal else 0, qp, typ, table, lens, o, ws, n, st))

    def _scratch_on(self, n: int, stream) -> torch.Tensor:
        if stream is None:
            return torch.empty(n, dtype=torch.uint8, device=self.device)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(n, dtype=torch.uint8, device=self.device)

    def oasis_prefix_workspace(self, R: int, S: int, prefix_len: int) -> int:
        n = c_size_t(0)
        rc = lib().oasis_prefix_workspace(self.q8, R, S, prefix_len, ctypes.byref(n))
        if rc != OASIS_OK:
            raise OasisError(rc, "prefix_workspace: bad size")
        return n.value

    def prefix_workspace(self, R: int, S: int, prefix_len: int) -> torch.Tensor:
        """Scratch for oasis_prefix_attn calls of these sizes that follow one another."""
        return torch.empty(self.oasis_prefix_workspace(R, S, prefix_len), dtype=torch.uint8,
                           device=self.device)

    def oasis_prefix_attn(self, q, prefix_kv, prefix_len, page_table, seq_len, out, workspace,
                          causal=False, stream=None) -> None:
        """q, out [S][R][Hq][128]; prefix_kv [Hkv][blocks][2][16][128] bf16; workspace from
        prefix_workspace."""
        R, table, lens = self._table(page_table, seq_len)
        S, qp, typ, o = self._queries(q, out, R)
        blocks = prefix_kv.shape[1] if prefix_kv.dim() == 5 else -1
        kv = _want("prefix_kv", prefix_kv, torch.bfloat16, (self._Hkv, blocks, 2, 16, 128), self._dev)
        n = workspace.numel()
        ws = _want("workspace", workspace, torch.uint8, (n,), self._dev)
        self._check(self._lib.oasis_prefix_attn(self.q8, R, S, 1 if causal else 0, qp, typ, kv, blocks,
                                                prefix_len, table, lens, o, ws, n,
                                                _stream_on(stream, self._dev)))


    def _tokens(self, name: str, x: torch.Tensor, T: int, H: int, dtype) -> tuple:
        """The address of x [T][H][d], whose heads are contiguous, and its elements a token."""
        if x.dtype is not dtype or x.shape != (T, H, 128) or x.get_device() != self._dev:
            raise ValueError(f"{name} must be {dtype} {[T, H, 128]} on {self.device}, got {x.dtype} "
                             f"{list(x.shape)} on {x.device}")
        st = x.stride()
        if T and (st[2] != 1 or (H > 1 and st[1] != 128)):
            raise ValueError(f"{name}: a token's heads must be contiguous")
        return x.data_ptr(), st[0] if T > 1 else H * 128

    def oasis_q8_append(self, rope: oasis_rope, q, k, v, positions, slots, q_out, stream=None) -> None:
        """q, q_out [T][Hq][128] (or both None), k, v [T][Hkv][128] bf16, fp16 or fp32 (tokens may
        be strided; q_out may be q), positions [axes][T] (or [T]) and slots [T] int64; rope from
        make_rope."""
        T = slots.numel()
        typ = _TYPES.get(k.dtype)
        if typ is None:
            raise ValueError(f"k must be bfloat16, float16 or float32, got {k.dtype}")
        kp, ks = self._tokens("k", k, T, self._Hkv, k.dtype)
        vp, vs = self._tokens("v", v, T, self._Hkv, k.dtype)
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out come together")
        qp, qs = (None, 0) if q is None else self._tokens("q", q, T, self._Hq, k.dtype)
        op, os_ = (None, 0) if q is None else self._tokens("q_out", q_out, T, self._Hq, k.dtype)
        shape = (rope.num_axes, T) if rope.num_axes > 1 or positions.dim() != 1 else (T,)
        self._check(self._lib.oasis_q8_append(
            self.q8, ctypes.byref(rope), qp, op, kp, vp, typ, qs, os_, ks, vs,
            _want("positions", positions, torch.int64, shape, self._dev),
            _want("slots", slots, torch.int64, (T,), self._dev), T, _stream_on(stream, self._dev)))

    def oasis_q8_tree_workspace(self, R: int, N: int, dtype=torch.bfloat16) -> int:
        n = c_size_t(0)
        rc = lib().oasis_q8_tree_workspace(self.q8, R, N, _TYPES.get(dtype, -1), ctypes.byref(n))
        if rc != OASIS_OK:
            raise OasisError(rc, "q8_tree_workspace: bad size")
        return n.value

    def oasis_q8_tree_attn(self, q, tree, page_table, seq_len, out, tree_size=None, stream=None,
                           workspace=None) -> None:
        """q, out [R][N][Hq][128], tree [R][N] int64 (see tree_words), tree_size [R] int32.
        workspace: scratch of oasis_q8_tree_workspace bytes (uint8), by default taken from the
        allocator for this call, like oasis_q8_attn's."""
        R, table, lens = self._table(page_table, seq_len)
        dt = q.dtype
        if dt is not torch.bfloat16 and dt is not torch.float16:
            raise ValueError(f"q must be bfloat16 or float16, got {dt}")
        N = q.shape[1] if q.dim() == 4 else -1
        shape = (R, N, self._Hq, 128)
        qp = _want("q", q, dt, shape, self._dev)
        o = _want("out", out, torch.float32 if self._out_fp32 else dt, shape, self._dev)
        w = _want("tree", tree, torch.int64, (R, N), self._dev)
        sz = None if tree_size is None else _want("tree_size", tree_size, torch.int32, (R,), self._dev)
        st = _stream_on(stream, self._dev)
        if workspace is None:
            n = self._scratch.get((R, N, dt))
            if n is None:
                n = self._scratch[R, N, dt] = self.oasis_q8_tree_workspace(R, N, dt) if 1 <= N <= 64 else 0
            if n:
                workspace = self._scratch_on(n, stream)
        else:
            n = workspace.numel()
        ws = _want("workspace", workspace, torch.uint8, (n,), self._dev) if n else None
        self._check(self._lib.oasis_q8_tree_attn(self.q8, R, N, qp, _TYPES[dt], w, sz, table, lens, o, ws, n, st))

    def oasis_q8_keep(self, page_table, seq_len, nodes, keep, num_nodes, tree_size=None, stream=None) -> None:
        """nodes [R][M] and keep [R] int32: the nodes of each request's tree that stay, in order;
        seq_len counts the whole trees still."""
        R, table, lens = self._table(page_table, seq_len)
        M = nodes.shape[1] if nodes.dim() == 2 else -1
        sz = None if tree_size is None else _want("tree_size", tree_size, torch.int32, (R,), self._dev)
        self._check(self._lib.oasis_q8_keep(
            self.q8, R, num_nodes, sz, table, lens, _want("nodes", nodes, torch.int32, (R, M), self._dev),
            _want("keep", keep, torch.int32, (R,), self._dev), M, _stream_on(stream, self._dev)))


def oasis_token_logprobs(logits, tokens=None, logprobs=None, entropy=None, top_ids=None,
                         top_logprobs=None, stream=None) -> None:
    """logits [rows][V] (or [..., V] with evenly spaced rows) in bf16, fp16 or fp32, tokens [rows]
    int32 (negative: the row is not wanted, its outputs stay); logprobs, entropy [rows] fp32,
    top_ids [rows][k] int32 and top_logprobs [rows][k] fp32 are written where given."""
    typ = _TYPES.get(logits.dtype)
    if logits.dim() < 2 or typ is None or not logits.is_cuda:
        raise ValueError("logits must be a bfloat16, float16 or float32 CUDA tensor [rows][V]")
    V, dev = logits.shape[-1], logits.get_device()
    st, lead = logits.stride(), logits.shape[:-1]
    rows = lead.numel()
    stride, ok, want = V, V <= 1 or st[-1] == 1, None
    for d in range(len(lead) - 1, -1, -1):  # one distance between all rows
        if lead[d] == 1:
            continue
        if want is None:
            stride = st[d]
        elif st[d] != want:
            ok = False
        want = st[d] * lead[d]
    if rows and not ok:
        raise ValueError("logits: rows must be contiguous and evenly spaced")

    def get(name, t, dtype, shape):
        return 0 if t is None else _want(name, t, dtype, shape, dev)

    if logprobs is not None and tokens is None:
        raise ValueError("logprobs needs tokens")
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs come together")
    k = 0 if top_ids is None else top_ids.shape[-1]
    a = _LOGPROBS_ARGS.pack(rows, V, typ, k, dev, logits.data_ptr(), stride,
                            get("tokens", tokens, torch.int32, lead),
                            get("logprobs", logprobs, torch.float32, lead),
                            get("entropy", entropy, torch.float32, lead),
                            get("top_ids", top_ids, torch.int32, (*lead, k)),
                            get("top_logprobs", top_logprobs, torch.float32, (*lead, k)))
    rc = lib().oasis_token_logprobs(a, _stream_on(stream, dev))
    if rc != OASIS_OK:
        m = lib().oasis_logprobs_error(a)
        raise OasisError(rc, m.decode() if m else "oasis_token_logprobs: CUDA error")


def oasis_verify_drafts(target, draft, tokens, u_accept, u_sample, out_tokens, n_accept,
                        n_drafts=None, stream=None) -> None:
    """target [R][n + 1][V] and draft [R][n][V] (or None: certain drafts) probabilities in bf16,
    fp16 or fp32 (rows may be padded: a common stride between them), tokens [R][n] int32,
    u_accept [R][n] and u_sample [R] fp32; out_tokens [R][n + 1] and n_accept [R] int32 are
    written.  n_drafts [R] int32: drafts of each request, n where None."""
    typ = _TYPES.get(target.dtype)
    if target.dim() != 3 or typ is None or not target.is_cuda or target.shape[1] < 1:
        raise ValueError("target must be a bfloat16, float16 or float32 CUDA tensor [R][n + 1][V]")
    R, n, V = target.shape
    n -= 1
    dev = target.get_device()

    def rows(name, x, m):
        if x.dtype is not target.dtype or x.shape != (R, m, V) or x.get_device() != dev:
            raise ValueError(f"{name} must be {target.dtype} {[R, m, V]} on cuda:{dev}, got {x.dtype} "
                             f"{list(x.shape)} on {x.device}")
        st = x.stride()
        stride = st[1] if m > 1 else st[0] if R > 1 else V
        if V > 1 and R and st[2] != 1 or (R > 1 and m > 1 and st[0] != m * stride):
            raise ValueError(f"{name}: rows must be contiguous and evenly spaced")
        return x.data_ptr(), stride

    p, ps = rows("target", target, n + 1)
    q, qs = rows("draft", draft, n) if draft is not None and n > 0 else (None, 0)
    # an oasis_verify_args, packed
    a = _VERIFY_ARGS.pack(R, n, V, typ, dev, p, q or 0, ps, qs,
                          _want("tokens", tokens, torch.int32, (R, n), dev),
                          0 if n_drafts is None else _want("n_drafts", n_drafts, torch.int32, (R,), dev),
                          _want("u_accept", u_accept, torch.float32, (R, n), dev),
                          _want("u_sample", u_sample, torch.float32, (R,), dev),
                          _want("out_tokens", out_tokens, torch.int32, (R, n + 1), dev),
                          _want("n_accept", n_accept, torch.int32, (R,), dev))
    rc = lib().oasis_verify_drafts(a, _stream_on(stream, dev))
    if rc != OASIS_OK:
        m = lib().oasis_verify_error(a)
        raise OasisError(rc, m.decode() if m else "oasis_verify_drafts: CUDA error")

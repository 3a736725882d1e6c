"""Thin Python binding of libgdn's C ABI (include/gdn.h).

Argument marshalling only: torch tensors supply device memory and the
current CUDA stream; every step of the computation runs in libgdn's CUDA
kernels.  The functions carry the C names.  If libgdn.so has not been built
the first call raises -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16, GDN_F16 = 0, 1, 2
STATUS = {0: "GDN_OK", 1: "GDN_ERR_ARG", 2: "GDN_ERR_SLOT", 3: "GDN_ERR_DUP_SLOT",
          4: "GDN_ERR_DTYPE", 5: "GDN_ERR_SIZE", 6: "GDN_ERR_UNSUPPORTED", 7: "GDN_ERR_CUDA"}
DEVERR_SLOT, DEVERR_SEQ, DEVERR_COUNT, DEVERR_TIMEOUT = 1, 2, 4, 8
DEVERR_PAGE, DEVERR_VALUE, DEVERR_ADAPTER = 16, 32, 64
GDN_KV_I8, GDN_KV_E4M3 = 0, 1
GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
TEST_DECODE_WAIT_TIMEOUT = 1
TEST_ADAPT_WAIT_TIMEOUT, TEST_ADAPT_SIDE_TIMEOUT = 4, 8
TEST_KV_WAIT_TIMEOUT = 1

EXPORTED = ("gdn_pool_state_bytes", "gdn_pool_conv_bytes", "gdn_pool_create", "gdn_pool_reset",
            "gdn_pool_copy",
            "gdn_pool_destroy", "gdn_pool_get_error", "gdn_pool_set_test_flags", "gdn_conv_silu",
            "gdn_decode_step",
            "gdn_decode_step_conv", "gdn_decode_step_conv_launches", "gdn_gated_rmsnorm",
            "gdn_in_proj",
            "gdn_prefill_chunked", "gdn_prefill_recurrent", "gdn_spec_verify",
            "gdn_spec_verify_deferred", "gdn_prefill_chunked_noalloc", "gdn_prefill_chunked_ckpt",
            "gdn_kv_code_bytes", "gdn_kv_scale_bytes", "gdn_kv_create", "gdn_kv_destroy",
            "gdn_kv_get_error", "gdn_kv_set_test_flags", "gdn_kv_append", "gdn_kv_read",
            "gdn_kv_attend", "gdn_kv_pages_grow", "gdn_kv_pages_trim",
            "gdn_rope_create", "gdn_rope_destroy", "gdn_rope",
            "gdn_adapters_create", "gdn_adapters_destroy", "gdn_in_proj_adapted",
            "gdn_status_string",
            "gdn_last_error_message")


class GDNError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.name = STATUS.get(status, str(status))


class gdn_pool_desc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("h_v", ctypes.c_int32), ("h_k", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
                ("conv_ch", ctypes.c_int32), ("conv_k", ctypes.c_int32),
                ("conv_dtype", ctypes.c_int), ("host_checks", ctypes.c_int32),
                ("prefill_workspace_max", ctypes.c_uint64), ("state_dtype", ctypes.c_int)]


class gdn_qkv(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("ld_qk", ctypes.c_int64), ("ld_v", ctypes.c_int64), ("dtype", ctypes.c_int)]


class gdn_kv_desc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("h_q", ctypes.c_int32),
                ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32), ("code", ctypes.c_int),
                ("host_checks", ctypes.c_int32)]


class gdn_kv_pages(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("held", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("n_free", ctypes.c_void_p)]


class gdn_rope_desc(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("rot", ctypes.c_int32), ("layout", ctypes.c_int),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_int64), ("low_turns", ctypes.c_double),
                ("high_turns", ctypes.c_double), ("out_scale", ctypes.c_float),
                ("host_checks", ctypes.c_int32)]


class gdn_adapters_desc(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("n_out", ctypes.c_int32),
                ("host_checks", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (once).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libgdn.so not found at {path}; build it with "
                           "`python -m gated_deltanet_recurrent_gb300.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    P = ctypes.POINTER
    sig = {
        "gdn_pool_state_bytes": (ctypes.c_size_t, [P(gdn_pool_desc)]),
        "gdn_pool_conv_bytes": (ctypes.c_size_t, [P(gdn_pool_desc)]),
        "gdn_pool_create": (st, [P(gdn_pool_desc), vp, ctypes.c_size_t, vp, ctypes.c_size_t,
                                 P(vp)]),
        "gdn_pool_reset": (st, [vp, vp, i32, vp]),
        "gdn_pool_copy": (st, [vp, vp, vp, i32, vp]),
        "gdn_pool_destroy": (st, [vp]),
        "gdn_pool_get_error": (st, [vp, P(ctypes.c_uint32)]),
        "gdn_pool_set_test_flags": (st, [vp, ctypes.c_uint32]),
        "gdn_conv_silu": (st, [vp, i32, vp, vp, i32, i32, i32, vp, i64, st, vp, vp, vp, i64,
                               vp, vp]),
        "gdn_decode_step": (st, [vp, i32, vp, i32, P(gdn_qkv), vp, st, ctypes.c_float, vp]),
        "gdn_decode_step_conv": (st, [vp, i32, vp, i32, vp, i64, vp, vp, vp, i64, vp, vp, st,
                                      vp, st, ctypes.c_float, vp]),
        "gdn_decode_step_conv_launches": (st, [vp, i32, st, st, P(i32)]),
        "gdn_gated_rmsnorm": (st, [i64, i32, vp, st, vp, st, vp, ctypes.c_float, vp, st, vp]),
        "gdn_in_proj": (st, [vp, i64, i32, i32, vp, i64, vp, i64, vp, i64, st, vp]),
        "gdn_prefill_chunked": (st, [vp, i32, vp, vp, i32, i32, i32, P(gdn_qkv), vp, st,
                                     ctypes.c_float, vp]),
        "gdn_prefill_recurrent": (st, [vp, i32, vp, vp, i32, i32, i32, P(gdn_qkv), vp, st,
                                       ctypes.c_float, vp]),
        "gdn_spec_verify": (st, [vp, i32, vp, i32, i32, P(gdn_qkv), vp, st, vp,
                                 ctypes.c_float, vp]),
        "gdn_spec_verify_deferred": (st, [vp, i32, vp, i32, i32, P(gdn_qkv), vp, st, i32,
                                          P(gdn_qkv), vp, ctypes.c_float, vp]),
        "gdn_prefill_chunked_noalloc": (st, [vp, i32, vp, vp, i32, i32, i32, P(gdn_qkv), vp, st,
                                             ctypes.c_float, vp]),
        "gdn_prefill_chunked_ckpt": (st, [vp, i32, vp, vp, i32, i32, i32, P(gdn_qkv), vp, st,
                                          ctypes.c_float, vp, i32, i32, vp]),
        "gdn_kv_code_bytes": (ctypes.c_size_t, [P(gdn_kv_desc)]),
        "gdn_kv_scale_bytes": (ctypes.c_size_t, [P(gdn_kv_desc)]),
        "gdn_kv_create": (st, [P(gdn_kv_desc), vp, vp, ctypes.c_size_t, vp, vp, ctypes.c_size_t,
                               vp, P(vp)]),
        "gdn_kv_destroy": (st, [vp]),
        "gdn_kv_get_error": (st, [vp, P(ctypes.c_uint32)]),
        "gdn_kv_set_test_flags": (st, [vp, ctypes.c_uint32]),
        "gdn_kv_append": (st, [vp, i32, vp, vp, vp, i32, i32, i32, vp, i64, vp, i64, st, vp]),
        "gdn_kv_read": (st, [vp, i32, vp, vp, vp, i32, i32, i32, vp, i64, vp, i64, st, vp]),
        "gdn_kv_attend": (st, [vp, i32, vp, vp, vp, i32, i32, i32, i32, vp, i64, st, vp, i64, st,
                               ctypes.c_float, vp]),
        "gdn_kv_pages_grow": (st, [vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp]),
        "gdn_kv_pages_trim": (st, [vp, vp, vp, vp, i32, vp]),
        "gdn_rope_create": (st, [P(gdn_rope_desc), P(vp)]),
        "gdn_rope_destroy": (st, [vp]),
        "gdn_rope": (st, [vp, i32, vp, vp, i64, i32, vp, i64, i32, vp, i64, vp, i64, st, vp]),
        "gdn_adapters_create": (st, [P(gdn_adapters_desc), vp, i64, vp, i64, vp, P(vp)]),
        "gdn_adapters_destroy": (st, [vp]),
        "gdn_in_proj_adapted": (st, [vp, vp, i64, vp, i64, vp, i64, vp, vp, i64, st, vp]),
        "gdn_status_string": (ctypes.c_char_p, [st]),
        "gdn_last_error_message": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _released(owner):
    """The owner's handle, which it no longer has: a destroy call frees it even where it reports
    an error, so that it must not be made again."""
    handle, owner.handle = owner.handle, None
    return handle


def _check(status: int):
    if status != 0:
        msg = load_library().gdn_last_error_message().decode()
        raise GDNError(status, msg)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN_F32
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    raise GDNError(4, f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _idx(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise GDNError(1, f"{name} must be a contiguous int32 tensor")
    return _ptr(t)


def _row_stride(t: torch.Tensor, width: int, name: str) -> int:
    """Stride of t's rows of `width` elements: that width for one row or none, whose stride says
    nothing.  Rows that overlap are refused, as those expanded from one (stride 0, which the
    library takes for packed)."""
    if t.shape[0] <= 1:
        return width
    if t.stride(0) < width:
        raise GDNError(1, f"{name}: row stride {t.stride(0)} smaller than a row of {width}")
    return t.stride(0)


def _token_rows(t: torch.Tensor, heads: int, dim: int, name: str) -> int:
    """Token stride (elements) of a [tokens, heads, dim] view whose heads are packed."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise GDNError(5, f"{name} must be [tokens, {heads}, {dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1 or (t.stride(1) != dim and heads > 1):
        raise GDNError(1, f"{name}: heads must be packed (strides {t.stride()})")
    return _row_stride(t, heads * dim, name)


def _qkv(pool: "Pool", q, k, v, g, beta) -> gdn_qkv:
    d = pool.desc
    ld_q = _token_rows(q, d.h_k, d.dk, "q")
    ld_k = _token_rows(k, d.h_k, d.dk, "k")
    ld_v = _token_rows(v, d.h_v, d.dv, "v")
    if ld_q != ld_k:
        raise GDNError(1, "q and k must share one token stride")
    for name, t in (("g", g), ("beta", beta)):
        if t.shape != (q.shape[0], d.h_v) or not t.is_contiguous():
            raise GDNError(5, f"{name} must be contiguous [tokens, {d.h_v}]")
    dts = {_dt(t) for t in (q, k, v, g, beta)}
    if len(dts) != 1:
        raise GDNError(4, "q, k, v, g and beta must share one dtype")
    return gdn_qkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                   ld_q, ld_v, dts.pop())


_STATE_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float16: GDN_F16}


class Pool:
    """A pool handle plus the torch tensors holding its state and conv cache:
    state [n_layers, n_slots, h_v, dv, dk] in state_dtype (float32, or
    bfloat16 / float16 storage), conv [n_layers, n_slots, conv_ch, conv_k-1]
    in conv_dtype.  Both start at zero."""

    def __init__(self, n_layers, n_slots, h_v, h_k, dk, dv, conv_ch, conv_k,
                 conv_dtype=torch.bfloat16, host_checks=True, device="cuda",
                 prefill_workspace_max=0, state_dtype=torch.float32):
        if state_dtype not in _STATE_DTYPES:
            raise GDNError(4, f"unsupported state dtype {state_dtype}")
        self.desc = gdn_pool_desc(n_layers, n_slots, h_v, h_k, dk, dv, conv_ch, conv_k,
                                  GDN_F32 if conv_dtype == torch.float32 else GDN_BF16,
                                  1 if host_checks else 0, prefill_workspace_max,
                                  _STATE_DTYPES[state_dtype])
        self.state = torch.zeros((n_layers, n_slots, h_v, dv, dk), dtype=state_dtype,
                                 device=device)
        self.conv = torch.zeros((n_layers, n_slots, conv_ch, conv_k - 1), dtype=conv_dtype,
                                device=device)
        self.handle = gdn_pool_create(self.desc, self.state, self.conv)

    @classmethod
    def for_shape(cls, shape, n_layers, n_slots, conv_dtype=torch.bfloat16, host_checks=True,
                  device="cuda", prefill_workspace_max=0, state_dtype=torch.float32):
        return cls(n_layers, n_slots, shape.h_v, shape.h_k, shape.dk, shape.dv,
                   shape.conv_ch, shape.conv_k, conv_dtype, host_checks, device,
                   prefill_workspace_max, state_dtype)

    def set_host_checks(self, on: bool):
        """Recreate the handle with host checks switched on or off (same memory)."""
        self.close()
        self.desc.host_checks = 1 if on else 0
        self.handle = gdn_pool_create(self.desc, self.state, self.conv)

    def close(self):
        if getattr(self, "handle", None):
            gdn_pool_destroy(self)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------- entry points

def gdn_pool_state_bytes(desc: gdn_pool_desc) -> int:
    return load_library().gdn_pool_state_bytes(ctypes.byref(desc))


def gdn_pool_conv_bytes(desc: gdn_pool_desc) -> int:
    return load_library().gdn_pool_conv_bytes(ctypes.byref(desc))


def gdn_pool_create(desc: gdn_pool_desc, state: torch.Tensor, conv: torch.Tensor):
    lib = load_library()
    out = ctypes.c_void_p()
    _check(lib.gdn_pool_create(ctypes.byref(desc), _ptr(state),
                               state.numel() * state.element_size(), _ptr(conv),
                               conv.numel() * conv.element_size(), ctypes.byref(out)))
    return out


def gdn_pool_destroy(pool: Pool):
    _check(load_library().gdn_pool_destroy(_released(pool)))


def gdn_pool_reset(pool: Pool, slot_ids: torch.Tensor, stream=None):
    _check(load_library().gdn_pool_reset(pool.handle, _idx(slot_ids, "slot_ids"),
                                         slot_ids.numel(), _stream(stream)))


def gdn_pool_copy(pool: Pool, src_slots: torch.Tensor, dst_slots: torch.Tensor, stream=None):
    if src_slots.numel() != dst_slots.numel():
        raise GDNError(5, "src_slots and dst_slots differ in length")
    _check(load_library().gdn_pool_copy(pool.handle, _idx(src_slots, "src_slots"),
                                        _idx(dst_slots, "dst_slots"), src_slots.numel(),
                                        _stream(stream)))


def gdn_pool_get_error(pool: Pool) -> int:
    err = ctypes.c_uint32(0)
    _check(load_library().gdn_pool_get_error(pool.handle, ctypes.byref(err)))
    return err.value


def gdn_pool_set_test_flags(pool: Pool, flags: int):
    """Test hook of the C ABI (see gdn.h); 0 restores normal operation."""
    _check(load_library().gdn_pool_set_test_flags(pool.handle, flags))


def gdn_conv_silu(pool: Pool, layer: int, slot_ids: torch.Tensor, x: torch.Tensor,
                  w: torch.Tensor, y: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, bias=None, advance=None,
                  max_seqlen: int = 0, stream=None):
    """x, y [tokens, conv_ch] (row stride may exceed conv_ch); w [conv_ch, conv_k] float32."""
    n = slot_ids.numel()
    if w.dtype != torch.float32 or not w.is_contiguous():
        raise GDNError(1, "w must be contiguous float32 [conv_ch, conv_k]")
    if x.dim() != 2 or x.stride(1) != 1 or (y is not None and y.stride(1) != 1):
        raise GDNError(1, "x and y must be [tokens, channels] with unit channel stride")
    if max_seqlen <= 0:
        max_seqlen = x.shape[0]
    _check(load_library().gdn_conv_silu(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), _idx(cu_seqlens, "cu_seqlens"), n,
        x.shape[0], max_seqlen, _ptr(x), _row_stride(x, x.shape[1], "x"), _dt(x), _ptr(w),
        _ptr(bias), _ptr(y), 0 if y is None else _row_stride(y, y.shape[1], "y"),
        _idx(advance, "advance"), _stream(stream)))
    return y


def gdn_decode_step(pool: Pool, layer: int, slot_ids: torch.Tensor, q, k, v, g, beta,
                    o: torch.Tensor, scale: float = 1.0, stream=None):
    """q, k [n, h_k, dk]; v [n, h_v, dv]; g, beta [n, h_v]; o [n, h_v, dv]."""
    inp = _qkv(pool, q, k, v, g, beta)
    _check(load_library().gdn_decode_step(pool.handle, layer, _idx(slot_ids, "slot_ids"),
                                          slot_ids.numel(), ctypes.byref(inp), _ptr(o),
                                          _dt(o), scale, _stream(stream)))
    return o


def gdn_decode_step_conv(pool: Pool, layer: int, slot_ids: torch.Tensor, x: torch.Tensor,
                         w: torch.Tensor, y: torch.Tensor, g, beta, o: torch.Tensor, bias=None,
                         scale: float = 1.0, stream=None):
    """conv + SiLU then the decode step in one call.  x, y [n, conv_ch] (row
    stride may exceed conv_ch; y is split into q | k | v); w [conv_ch, conv_k]
    float32; g, beta [n, h_v] in x's dtype; o [n, h_v, dv]."""
    n = slot_ids.numel()
    if w.dtype != torch.float32 or not w.is_contiguous():
        raise GDNError(1, "w must be contiguous float32 [conv_ch, conv_k]")
    for name, t in (("x", x), ("y", y)):
        if t.dim() != 2 or t.stride(1) != 1 or t.shape[0] != n:
            raise GDNError(1, f"{name} must be [n, channels] with unit channel stride")
    for name, t in (("g", g), ("beta", beta)):
        if t.shape != (n, pool.desc.h_v) or not t.is_contiguous():
            raise GDNError(5, f"{name} must be contiguous [n, {pool.desc.h_v}]")
    dts = {_dt(t) for t in (x, y, g, beta)}
    if len(dts) != 1:
        raise GDNError(4, "x, y, g and beta must share one dtype")
    _check(load_library().gdn_decode_step_conv(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), n, _ptr(x),
        _row_stride(x, x.shape[1], "x"), _ptr(w), _ptr(bias), _ptr(y),
        _row_stride(y, y.shape[1], "y"), _ptr(g), _ptr(beta), dts.pop(), _ptr(o), _dt(o), scale,
        _stream(stream)))
    return o


def gdn_decode_step_conv_launches(pool: Pool, n: int, dtype: torch.dtype,
                                  o_dtype: torch.dtype = torch.float32) -> int:
    """Kernel launches gdn_decode_step_conv makes for n slots (1 or 2; 0 if n = 0)."""
    codes = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float16: GDN_F16}
    out = ctypes.c_int32(-1)
    _check(load_library().gdn_decode_step_conv_launches(pool.handle, n, codes[dtype],
                                                         codes[o_dtype], ctypes.byref(out)))
    return out.value


def gdn_in_proj(pool: Pool, x: torch.Tensor, w: torch.Tensor,
                y: Optional[torch.Tensor] = None, stream=None):
    """y = x w^T: x [tokens, hidden] bf16, w [n_out, hidden] bf16 (unit
    column strides), y [tokens, n_out] float32 or bf16 (default float32)."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise GDNError(4, "x and w must be bf16")
    if x.dim() != 2 or w.dim() != 2 or x.stride(1) != 1 or w.stride(1) != 1 or \
            x.shape[1] != w.shape[1]:
        raise GDNError(1, "x [tokens, hidden] and w [n_out, hidden] with unit column strides")
    if y is None:
        y = torch.empty(x.shape[0], w.shape[0], dtype=torch.float32, device=x.device)
    if y.dim() != 2 or y.stride(1) != 1 or tuple(y.shape) != (x.shape[0], w.shape[0]):
        raise GDNError(1, "y must be [tokens, n_out] with a unit column stride")
    _check(load_library().gdn_in_proj(pool.handle, x.shape[0], x.shape[1], w.shape[0], _ptr(x),
                                      _row_stride(x, x.shape[1], "x"), _ptr(w),
                                      _row_stride(w, w.shape[1], "w"), _ptr(y),
                                      _row_stride(y, y.shape[1], "y"), _dt(y), _stream(stream)))
    return y


def gdn_gated_rmsnorm(o: torch.Tensor, z: torch.Tensor, w: torch.Tensor,
                      y: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None):
    """Output gated RMSNorm over the last axis: o, z, y [..., d] contiguous
    (each float32 or bf16; y defaults to float32), w [d] float32."""
    d = o.shape[-1]
    if y is None:
        y = torch.empty(o.shape, dtype=torch.float32, device=o.device)
    for name, t in (("o", o), ("z", z), ("y", y)):
        if t.shape != o.shape or not t.is_contiguous():
            raise GDNError(1, f"{name} must be contiguous with o's shape {tuple(o.shape)}")
    if w.dtype != torch.float32 or not w.is_contiguous() or w.numel() != d:
        raise GDNError(1, f"w must be contiguous float32 [{d}]")
    _check(load_library().gdn_gated_rmsnorm(o.numel() // max(d, 1), d, _ptr(o), _dt(o), _ptr(z),
                                            _dt(z), _ptr(w), eps, _ptr(y), _dt(y),
                                            _stream(stream)))
    return y


def gdn_prefill_chunked(pool: Pool, layer: int, slot_ids: torch.Tensor,
                        cu_seqlens: torch.Tensor, q, k, v, g, beta, o: torch.Tensor,
                        scale: float = 1.0, max_seqlen: int = 0, stream=None):
    """Packed varlen tokens: q, k [T, h_k, dk]; v [T, h_v, dv]; o [T, h_v, dv]."""
    inp = _qkv(pool, q, k, v, g, beta)
    if max_seqlen <= 0:
        max_seqlen = q.shape[0]
    _check(load_library().gdn_prefill_chunked(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), _idx(cu_seqlens, "cu_seqlens"),
        slot_ids.numel(), q.shape[0], max_seqlen, ctypes.byref(inp), _ptr(o), _dt(o), scale,
        _stream(stream)))
    return o


def gdn_prefill_recurrent(pool: Pool, layer: int, slot_ids: torch.Tensor,
                          cu_seqlens: torch.Tensor, q, k, v, g, beta, o: torch.Tensor,
                          scale: float = 1.0, max_seqlen: int = 0, stream=None):
    """Token-by-token prefill; same arguments and results as gdn_prefill_chunked."""
    inp = _qkv(pool, q, k, v, g, beta)
    if max_seqlen <= 0:
        max_seqlen = q.shape[0]
    _check(load_library().gdn_prefill_recurrent(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), _idx(cu_seqlens, "cu_seqlens"),
        slot_ids.numel(), q.shape[0], max_seqlen, ctypes.byref(inp), _ptr(o), _dt(o), scale,
        _stream(stream)))
    return o


def gdn_spec_verify(pool: Pool, layer: int, slot_ids: torch.Tensor, T: int, q, k, v, g, beta,
                    o: Optional[torch.Tensor] = None,
                    accept_len: Optional[torch.Tensor] = None, scale: float = 1.0,
                    stream=None):
    """Draft t of slot i is token i*T + t; o [n, T, h_v, dv] (or None)."""
    inp = _qkv(pool, q, k, v, g, beta)
    o_dt = GDN_F32 if o is None else _dt(o)
    _check(load_library().gdn_spec_verify(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), slot_ids.numel(), T,
        ctypes.byref(inp), _ptr(o), o_dt, _idx(accept_len, "accept_len"), scale,
        _stream(stream)))
    return o


def gdn_spec_verify_deferred(pool: Pool, layer: int, slot_ids: torch.Tensor, T: int, q, k, v, g,
                             beta, o: torch.Tensor, prev=None,
                             prev_accept: Optional[torch.Tensor] = None, scale: float = 1.0,
                             stream=None):
    """Commit the first prev_accept[i] of last round's drafts, then output this
    round's T drafts without committing them.  prev = (q, k, v, g, beta) of
    last round ([n*T_prev, ...] each) or None; o [n, T, h_v, dv]."""
    inp = _qkv(pool, q, k, v, g, beta)
    n = slot_ids.numel()
    T_prev, pin = 0, None
    if prev is not None:
        pin = _qkv(pool, *prev)
        if n == 0 or prev[0].shape[0] % n:
            raise GDNError(5, "prev holds no whole number of drafts per slot")
        T_prev = prev[0].shape[0] // n
    _check(load_library().gdn_spec_verify_deferred(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), n, T, ctypes.byref(inp), _ptr(o),
        _dt(o), T_prev, None if pin is None else ctypes.byref(pin),
        _idx(prev_accept, "prev_accept"), scale, _stream(stream)))
    return o


def gdn_prefill_chunked_noalloc(pool: Pool, layer: int, slot_ids: torch.Tensor,
                                cu_seqlens: torch.Tensor, q, k, v, g, beta, o: torch.Tensor,
                                scale: float = 1.0, max_seqlen: int = 0, stream=None):
    """gdn_prefill_chunked without any device allocation: its workspace is a
    fixed 64 MiB array inside the library, shared by all calls."""
    inp = _qkv(pool, q, k, v, g, beta)
    if max_seqlen <= 0:
        max_seqlen = q.shape[0]
    _check(load_library().gdn_prefill_chunked_noalloc(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), _idx(cu_seqlens, "cu_seqlens"),
        slot_ids.numel(), q.shape[0], max_seqlen, ctypes.byref(inp), _ptr(o), _dt(o), scale,
        _stream(stream)))
    return o


def gdn_prefill_chunked_ckpt(pool: Pool, layer: int, slot_ids: torch.Tensor,
                             cu_seqlens: torch.Tensor, q, k, v, g, beta, o: torch.Tensor,
                             ckpt_slots: torch.Tensor, ckpt_every: int, scale: float = 1.0,
                             max_seqlen: int = 0, stream=None):
    """gdn_prefill_chunked that also writes the state after every ckpt_every
    tokens of sequence i into slot ckpt_slots[i, j] (int32 [n_seqs, m], -1: none)."""
    inp = _qkv(pool, q, k, v, g, beta)
    if max_seqlen <= 0:
        max_seqlen = q.shape[0]
    if ckpt_slots.dim() != 2 or ckpt_slots.shape[0] != slot_ids.numel():
        raise GDNError(5, "ckpt_slots must be [n_seqs, m]")
    _check(load_library().gdn_prefill_chunked_ckpt(
        pool.handle, layer, _idx(slot_ids, "slot_ids"), _idx(cu_seqlens, "cu_seqlens"),
        slot_ids.numel(), q.shape[0], max_seqlen, ctypes.byref(inp), _ptr(o), _dt(o), scale,
        _idx(ckpt_slots.contiguous(), "ckpt_slots"), ckpt_slots.shape[1], ckpt_every,
        _stream(stream)))
    return o


# ------------------------------------------------------- 8-bit paged KV cache

_KV_CODES = {torch.int8: GDN_KV_I8, torch.float8_e4m3fn: GDN_KV_E4M3}


class KVCache:
    """A handle on an 8-bit paged KV cache plus the torch tensors that hold it:
    k, v [n_layers, n_pages, h_kv, page_tokens, d] codes (int8 or
    float8_e4m3fn: the latter where a few channels of the keys are much larger
    than the others), k_scale, v_scale [n_layers, n_pages, h_kv] float32 powers
    of two (value = code * scale) and page_table [n_slots, max_pages] int32,
    which the caller fills with page ids.  See gdn.h for the layout's rules."""

    def __init__(self, k, v, k_scale, v_scale, page_table, h_q, host_checks=True):
        if k.dtype not in _KV_CODES:
            raise GDNError(4, f"unsupported code type {k.dtype}")
        if k.dim() != 5 or v.shape != k.shape or v.dtype != k.dtype:
            raise GDNError(5, "k and v must share one shape [n_layers, n_pages, h_kv, "
                              "page_tokens, d] and type")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or t.shape != k.shape[:3]:
                raise GDNError(5, f"{name} must be float32 {tuple(k.shape[:3])}")
        if page_table.dtype != torch.int32 or page_table.dim() != 2:
            raise GDNError(1, "page_table must be int32 [n_slots, max_pages]")
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale),
                        ("page_table", page_table)):
            if not t.is_contiguous() or t.device != k.device:
                raise GDNError(1, f"{name} must be contiguous and on k's device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table = page_table
        self.h_q, self.h_kv, self.d = h_q, k.shape[2], k.shape[4]
        self.desc = gdn_kv_desc(k.shape[0], page_table.shape[0], k.shape[1], page_table.shape[1],
                                k.shape[3], h_q, k.shape[2], k.shape[4], _KV_CODES[k.dtype],
                                1 if host_checks else 0)
        self.handle = gdn_kv_create(self.desc, k, v, k_scale, v_scale, page_table)

    @classmethod
    def empty(cls, n_layers, n_slots, n_pages, max_pages, page_tokens, h_q, h_kv, d,
              code=torch.int8, host_checks=True, device="cuda"):
        """A cache in new memory.  The page table starts at -1 (no page)."""
        shape = (n_layers, n_pages, h_kv, page_tokens, d)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(code) for _ in range(2))
        ks, vs = (torch.zeros(shape[:3], device=device) for _ in range(2))
        table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=device)
        return cls(k, v, ks, vs, table, h_q, host_checks)

    def close(self):
        if getattr(self, "handle", None):
            gdn_kv_destroy(self)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gdn_kv_code_bytes(desc: gdn_kv_desc) -> int:
    return load_library().gdn_kv_code_bytes(ctypes.byref(desc))


def gdn_kv_scale_bytes(desc: gdn_kv_desc) -> int:
    return load_library().gdn_kv_scale_bytes(ctypes.byref(desc))


def gdn_kv_create(desc: gdn_kv_desc, k, v, k_scale, v_scale, page_table):
    out = ctypes.c_void_p()
    _check(load_library().gdn_kv_create(
        ctypes.byref(desc), _ptr(k), _ptr(v), k.numel() * k.element_size(), _ptr(k_scale),
        _ptr(v_scale), k_scale.numel() * 4, _ptr(page_table), ctypes.byref(out)))
    return out


def gdn_kv_destroy(kv: KVCache):
    _check(load_library().gdn_kv_destroy(_released(kv)))


def gdn_kv_get_error(kv: KVCache) -> int:
    err = ctypes.c_uint32(0)
    _check(load_library().gdn_kv_get_error(kv.handle, ctypes.byref(err)))
    return err.value


def gdn_kv_set_test_flags(kv: KVCache, flags: int):
    """Test hook of the C ABI (see gdn.h); 0 restores normal operation."""
    _check(load_library().gdn_kv_set_test_flags(kv.handle, flags))


# A decode step's calls are a few microseconds long: the checks below read each
# attribute once, and the stream comes as a raw handle.

def _kv_stream(stream, t: torch.Tensor) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(t.device.index)


_KV_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _kv_dtype(t: torch.Tensor) -> int:
    code = _KV_DTYPES.get(t.dtype)
    if code is None:
        raise GDNError(4, f"unsupported dtype {t.dtype}")
    return code


def _kv_index(slot_ids, starts, cu_seqlens, tokens, name):
    """Pointers of the index arrays, and the number of sequences."""
    i32 = torch.int32
    n = slot_ids.numel()
    if slot_ids.dtype != i32 or starts.dtype != i32 or not slot_ids.is_contiguous() or \
            not starts.is_contiguous():
        raise GDNError(1, f"slot_ids and {name} must be contiguous int32 tensors")
    if starts.numel() != n:
        raise GDNError(5, f"{name} must have an entry per slot id")
    if cu_seqlens is None:
        if tokens != n:
            raise GDNError(5, "without cu_seqlens there is one token per slot")
        return slot_ids.data_ptr(), starts.data_ptr(), None, n
    if cu_seqlens.dtype != i32 or not cu_seqlens.is_contiguous():
        raise GDNError(1, "cu_seqlens must be a contiguous int32 tensor")
    if cu_seqlens.numel() != n + 1:
        raise GDNError(5, "cu_seqlens must have one entry more than slot_ids")
    return slot_ids.data_ptr(), starts.data_ptr(), cu_seqlens.data_ptr(), n


def _kv_token_rows(shape, stride, heads, dim, name):
    """Token stride of [tokens, heads, dim] rows whose heads are packed (0: one row, whose
    stride says nothing)."""
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise GDNError(5, f"{name} must be [tokens, {heads}, {dim}], got {tuple(shape)}")
    if stride[2] != 1 or (stride[1] != dim and heads > 1):
        raise GDNError(1, f"{name}: heads must be packed (strides {stride})")
    if shape[0] <= 1:
        return 0
    if stride[0] < heads * dim:  # an expanded row (stride 0) is not the library's "packed" (0)
        raise GDNError(1, f"{name}: token stride {stride[0]} smaller than a token")
    return stride[0]


def _kv_rows(kv, slot_ids, pos, k, v, cu_seqlens, max_seqlen):
    k_ptr = v_ptr = None
    ld_k = ld_v = 0
    tokens = dtype = None
    if k is not None:
        shape = k.shape
        tokens, dtype = shape[0], k.dtype
        ld_k = _kv_token_rows(shape, k.stride(), kv.h_kv, kv.d, "k")
        k_ptr = k.data_ptr()
    if v is not None:
        shape = v.shape
        if tokens is None:
            tokens, dtype = shape[0], v.dtype
        elif shape[0] != tokens or v.dtype != dtype:
            raise GDNError(4, "k and v must share one dtype and token count")
        ld_v = _kv_token_rows(shape, v.stride(), kv.h_kv, kv.d, "v")
        v_ptr = v.data_ptr()
    code = _KV_DTYPES.get(dtype)
    if code is None:
        raise GDNError(1 if dtype is None else 4, f"k or v of float32 or bf16 needed, got {dtype}")
    slots, starts, cu, n = _kv_index(slot_ids, pos, cu_seqlens, tokens, "pos")
    if max_seqlen <= 0:
        max_seqlen = 1 if cu is None else tokens
    return slots, starts, cu, n, tokens, max_seqlen, k_ptr, ld_k, v_ptr, ld_v, code


def gdn_kv_append(kv: KVCache, layer: int, slot_ids: torch.Tensor, pos: torch.Tensor,
                  k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  max_seqlen: int = 0, stream=None):
    """Quantise k, v [tokens, h_kv, d] (float32 or bf16; the token stride may
    exceed h_kv * d) into positions pos[i], pos[i] + 1, ... of slot slot_ids[i]."""
    if k is None or v is None:
        raise GDNError(1, "k and v are both needed")
    status = _lib.gdn_kv_append(
        kv.handle, layer, *_kv_rows(kv, slot_ids, pos, k, v, cu_seqlens, max_seqlen),
        _kv_stream(stream, slot_ids))
    if status:
        _check(status)


def gdn_kv_read(kv: KVCache, layer: int, slot_ids: torch.Tensor, pos: torch.Tensor,
                k: Optional[torch.Tensor], v: Optional[torch.Tensor],
                cu_seqlens: Optional[torch.Tensor] = None, max_seqlen: int = 0, stream=None):
    """Read cached tokens back as values into k, v [tokens, h_kv, d] (either may be None)."""
    status = _lib.gdn_kv_read(
        kv.handle, layer, *_kv_rows(kv, slot_ids, pos, k, v, cu_seqlens, max_seqlen),
        _kv_stream(stream, slot_ids))
    if status:
        _check(status)
    return k, v


def gdn_kv_attend(kv: KVCache, layer: int, slot_ids: torch.Tensor, kv_lens: torch.Tensor,
                  q: torch.Tensor, o: Optional[torch.Tensor] = None,
                  cu_seqlens: Optional[torch.Tensor] = None, max_seqlen: int = 0,
                  max_kv_len: int = 0, scale: Optional[float] = None, stream=None):
    """Causal attention of q [tokens, h_q, d] over the slots' cached tokens;
    kv_lens counts the query tokens themselves (append them first).  o
    [tokens, h_q, d] (default: q's type); scale defaults to d ** -0.5.  With
    bf16 q the softmax weights are rounded to 2^-11, whichever type o has; with
    float32 q they and q are held to 2^-22."""
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    shape = q.shape
    if o.shape != shape:
        raise GDNError(5, f"o must have q's shape {tuple(shape)}")
    ld_q = _kv_token_rows(shape, q.stride(), kv.h_q, kv.d, "q")
    ld_o = _kv_token_rows(shape, o.stride(), kv.h_q, kv.d, "o")
    tokens = shape[0]
    slots, starts, cu, n = _kv_index(slot_ids, kv_lens, cu_seqlens, tokens, "kv_lens")
    if max_seqlen <= 0:
        max_seqlen = 1 if cu is None else tokens
    if max_kv_len <= 0:
        max_kv_len = kv.desc.max_pages * kv.desc.page_tokens
    status = _lib.gdn_kv_attend(
        kv.handle, layer, slots, starts, cu, n, tokens, max_seqlen, max_kv_len, q.data_ptr(), ld_q,
        _kv_dtype(q), o.data_ptr(), ld_o, _kv_dtype(o), kv.d ** -0.5 if scale is None else scale,
        _kv_stream(stream, slot_ids))
    if status:
        _check(status)
    return o


_INT32 = 2 ** 31 - 1  # (larger sizes would be cut to 32 bits on their way to the library)


def _elsewhere(t, device):
    """Whether t is not on the GPU of that index (-1: the host's memory)."""
    d = t.get_device()
    return d != device or (d < 0 and t.is_meta)


# ----------------------------------------- pages of the KV cache, on the GPU

class KVPages:
    """What the page calls keep beside the cache's page table: held [n_slots], free_pages
    [n_pages] and n_free [1], int32 on the cache's device.  By default no slot holds a page
    (the page table's entries are -1) and page 0 is the first to be given out."""

    def __init__(self, kv: KVCache, held=None, free_pages=None, n_free=None):
        d, device = kv.desc, kv.page_table.device
        if (held is None) != (free_pages is None) or (held is None) != (n_free is None):
            raise GDNError(1, "held, free_pages and n_free are given together")
        if held is None:
            held = torch.zeros(d.n_slots, dtype=torch.int32, device=device)
            free_pages = torch.arange(d.n_pages - 1, -1, -1, dtype=torch.int32, device=device)
            n_free = torch.full((1,), d.n_pages, dtype=torch.int32, device=device)
        for name, t, size in (("held", held, d.n_slots), ("free_pages", free_pages, d.n_pages),
                              ("n_free", n_free, 1)):
            if t.dtype != torch.int32 or not t.is_contiguous() or t.device != device:
                raise GDNError(1, f"{name} must be contiguous int32 on the cache's device")
            if t.numel() != size:
                raise GDNError(5, f"{name} must have {size} entries")
        self.page_table, self.held, self.free_pages, self.n_free = \
            kv.page_table, held, free_pages, n_free
        self.device = held.get_device()
        self.kv, self.sizes = kv, (d.n_slots, d.n_pages)
        self.desc = gdn_kv_pages(kv.page_table.data_ptr(), held.data_ptr(),
                                 free_pages.data_ptr(), n_free.data_ptr())
        self.desc_ptr = ctypes.addressof(self.desc)


def _book_of(kv, pages):
    """The arrays' sizes are those of the cache that they were made for: another on the same page
    table may have more slots or pages."""
    d = kv.desc
    if pages.sizes != (d.n_slots, d.n_pages):
        raise GDNError(5, f"held and free_pages have {pages.sizes} entries, the cache has "
                          f"{d.n_slots} slots and {d.n_pages} pages")


def _like(t, name, dtype, size, device):
    """Pointer of an optional output array; device: an index."""
    if t is None:
        return None
    if t.dtype != dtype or _elsewhere(t, device) or not t.is_contiguous():
        raise GDNError(1, f"{name} must be a contiguous {dtype} tensor on slot_ids' device")
    if t.numel() != size:
        raise GDNError(5, f"{name} must have {size} entries")
    return t.data_ptr()


def gdn_kv_pages_grow(kv: KVCache, pages: KVPages, slot_ids: torch.Tensor, pos: torch.Tensor,
                      cu_seqlens: Optional[torch.Tensor] = None, total_tokens: int = -1,
                      positions: Optional[torch.Tensor] = None,
                      rows: Optional[torch.Tensor] = None,
                      granted: Optional[torch.Tensor] = None, stream=None):
    """Pages for the new tokens at pos[i], pos[i] + 1, ... of slot slot_ids[i] (one each, or
    packed by cu_seqlens).  positions (int32), rows (int64): [total_tokens], where each token
    goes; granted (int32): [n_seqs], 0 where the free pages did not suffice; each is written if
    given.  total_tokens is needed where neither positions nor rows says it."""
    tokens = rows.numel() if rows is not None else \
        positions.numel() if positions is not None else total_tokens
    if total_tokens not in (-1, tokens):
        raise GDNError(5, f"total_tokens is {total_tokens}, the outputs hold {tokens}")
    if tokens < 0:
        if cu_seqlens is not None:
            raise GDNError(1, "total_tokens is needed with cu_seqlens")
        tokens = slot_ids.numel()
    if tokens > _INT32:
        raise GDNError(5, f"{tokens} tokens: more than 2^31 - 1")
    device = pages.device
    if kv is not pages.kv:
        _book_of(kv, pages)
    if _elsewhere(slot_ids, device) or _elsewhere(pos, device) or \
            (cu_seqlens is not None and _elsewhere(cu_seqlens, device)):
        raise GDNError(1, "slot_ids, pos and cu_seqlens must be on the cache's device")
    slots, starts, cu, n = _kv_index(slot_ids, pos, cu_seqlens, tokens, "pos")
    status = _lib.gdn_kv_pages_grow(
        kv.handle, pages.desc_ptr, slots, starts, cu, n, tokens,
        _like(positions, "positions", torch.int32, tokens, device),
        _like(rows, "rows", torch.int64, tokens, device),
        _like(granted, "granted", torch.int32, n, device),
        stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device))
    if status:
        _check(status)


def gdn_kv_pages_trim(kv: KVCache, pages: KVPages, slot_ids: torch.Tensor, lens: torch.Tensor,
                      stream=None):
    """Give back the pages that the first lens[i] tokens of slot slot_ids[i] do not use."""
    device = pages.device
    if kv is not pages.kv:
        _book_of(kv, pages)
    if _elsewhere(slot_ids, device) or _elsewhere(lens, device):
        raise GDNError(1, "slot_ids and lens must be on the cache's device")
    slots, starts, _, n = _kv_index(slot_ids, lens, None, slot_ids.numel(), "lens")
    status = _lib.gdn_kv_pages_trim(
        kv.handle, pages.desc_ptr, slots, starts, n,
        stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device))
    if status:
        _check(status)


# ------------------------------------------------------------ rotary positions

_only = None  # the GPU's index where there is one only, as soon as that is known


def _rope_positions(positions, tokens, device):
    """Refuses positions that cannot be.  The plan belongs to no device: the launch goes to the
    current one, on which they have to be."""
    global _only
    if positions.dtype != torch.int32 or device < 0 or not positions.is_contiguous():
        raise GDNError(1, "positions must be a contiguous int32 tensor on the GPU")
    if tokens > _INT32:
        raise GDNError(5, f"{tokens} tokens: more than 2^31 - 1")
    if device != torch._C._cuda_getDevice():
        raise GDNError(1, f"the tensors are on GPU {device}, which is not the current one")
    if torch.cuda.device_count() == 1:
        _only = device


_ROPE_LAYOUTS = {"half": GDN_ROPE_HALF, "interleaved": GDN_ROPE_INTERLEAVED}


class Rope:
    """A plan of rotary positions: heads of d elements whose first `rot` (default: all) are
    turned, in pairs (j, j + rot/2) ("half") or (2j, 2j + 1) ("interleaved"), by position *
    base ** (-2j / rot).  factor, original_len, low_turns and high_turns scale the frequencies
    for long contexts and out_scale what is rotated: see gdn.h."""

    def __init__(self, d, rot=None, layout="half", base=10000.0, factor=1.0, original_len=0,
                 low_turns=1.0, high_turns=32.0, out_scale=1.0, host_checks=False):
        if layout not in _ROPE_LAYOUTS:
            raise GDNError(1, f"layout must be one of {sorted(_ROPE_LAYOUTS)}, got {layout!r}")
        self.d, self.rot = d, d if rot is None else rot
        self.desc = gdn_rope_desc(d, self.rot, _ROPE_LAYOUTS[layout], base, factor, original_len,
                                  low_turns, high_turns, out_scale, 1 if host_checks else 0)
        self.handle = gdn_rope_create(self.desc)

    def close(self):
        if getattr(self, "handle", None):
            gdn_rope_destroy(self)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gdn_rope_create(desc: gdn_rope_desc):
    out = ctypes.c_void_p()
    _check(load_library().gdn_rope_create(ctypes.byref(desc), ctypes.byref(out)))
    return out


def gdn_rope_destroy(rope: Rope):
    _check(load_library().gdn_rope_destroy(_released(rope)))


def _rope_rows(x, out, d, tokens, dtype, device, name):
    """Pointer, token stride and heads of x [tokens, heads, d], and pointer and stride of out
    (None: x itself); device: an index."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != tokens:
        raise GDNError(5, f"{name} must be [{tokens}, heads, {d}], got {tuple(shape)}")
    heads = shape[1]
    ld = _kv_token_rows(shape, x.stride(), heads, d, name)
    ptr = x.data_ptr()
    if x.dtype != dtype or x.get_device() != device:
        _rope_refuse(x, dtype, name)
    if out is None or out is x:
        return ptr, ld, heads, ptr, ld
    if out.shape != shape:
        raise GDNError(5, f"{name}_out must have {name}'s shape {tuple(shape)}")
    if out.dtype != dtype or out.get_device() != device:
        _rope_refuse(out, dtype, name)
    return ptr, ld, heads, out.data_ptr(), _kv_token_rows(shape, out.stride(), heads, d,
                                                          f"{name}_out")


def _rope_refuse(t, dtype, name):
    if t.dtype != dtype:
        raise GDNError(4, "q, k and their outputs must share one dtype")
    raise GDNError(1, f"{name} must be on the positions' device")


def gdn_rope(rope: Rope, positions: torch.Tensor, q: Optional[torch.Tensor],
             k: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
             k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotate q [tokens, h_q, d] and k [tokens, h_k, d] (float32 or bf16; either may be None; the
    token stride may exceed heads * d) to positions [tokens] int32, into q_out and k_out, or in
    place where these are not given.  Returns both."""
    first = k if q is None else q
    if first is None:
        raise GDNError(1, "q or k is needed")
    tokens, dtype, device = positions.numel(), first.dtype, positions.get_device()
    code = _KV_DTYPES.get(dtype)
    if code is None:
        raise GDNError(4, f"unsupported dtype {dtype}")
    if positions.dtype != torch.int32 or device != _only or not positions.is_contiguous() or \
            tokens > 0x7fffffff:
        _rope_positions(positions, tokens, device)
    if tokens:
        q_ptr = q_to = k_ptr = k_to = None
        ld_q = h_q = ld_q_to = ld_k = h_k = ld_k_to = 0
        if q is not None:
            q_ptr, ld_q, h_q, q_to, ld_q_to = _rope_rows(q, q_out, rope.d, tokens, dtype, device,
                                                         "q")
        if k is not None:
            k_ptr, ld_k, h_k, k_to, ld_k_to = _rope_rows(k, k_out, rope.d, tokens, dtype, device,
                                                         "k")
        status = _lib.gdn_rope(
            rope.handle, tokens, positions.data_ptr(), q_ptr, ld_q, h_q, k_ptr, ld_k, h_k, q_to,
            ld_q_to, k_to, ld_k_to, code, stream.cuda_stream if stream is not None else
            torch._C._cuda_getCurrentRawStream(device))
        if status:
            _check(status)
    return q if q_out is None else q_out, k if k_out is None else k_out


# ------------------------------------- low-rank adapters beside the projection

class Adapters:
    """The low-rank adapters of one projection: a [n, rank, hidden] and b [n, n_out, rank] bf16,
    scale [n] float32 (default: ones), rank <= 128.  Rows start 16-byte aligned; those of one
    adapter follow the other's.  The tensors may be rewritten between calls."""

    def __init__(self, a, b, scale=None, host_checks=False):
        if a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
            raise GDNError(4, "a and b must be bf16")
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise GDNError(5, "a must be [n, rank, hidden] and b [n, n_out, rank]")
        n, self.rank, self.hidden = a.shape
        self.n_out = b.shape[1]
        if max(n, self.rank, self.hidden, self.n_out) > _INT32:
            raise GDNError(6, "a and b have sizes of 2^31 and more")
        if scale is None:
            scale = torch.ones(n, dtype=torch.float32, device=a.device)
        if scale.dtype != torch.float32 or scale.shape != (n,) or not scale.is_contiguous():
            raise GDNError(1, f"scale must be contiguous float32 [{n}]")
        if b.device != a.device or scale.device != a.device:
            raise GDNError(1, "a, b and scale must be on one device")
        lds = []
        for name, t in (("a", a), ("b", b)):
            rows, width = t.shape[1], t.shape[2]
            ld = t.stride(1) if rows > 1 else t.stride(0) if n > 1 else width
            if (width > 1 and t.stride(2) != 1) or ld < width or \
                    (n > 1 and t.stride(0) != rows * ld):
                raise GDNError(1, f"{name}: one row stride for all rows needed, and unit column "
                                  f"stride (strides {t.stride()})")
            lds.append(ld)
        self.a, self.b, self.scale = a, b, scale
        self.device = a.get_device()
        self.desc = gdn_adapters_desc(n, self.rank, self.hidden, self.n_out,
                                      1 if host_checks else 0)
        self.handle = gdn_adapters_create(self.desc, a, lds[0], b, lds[1], scale)

    def close(self):
        if getattr(self, "handle", None):
            gdn_adapters_destroy(self)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gdn_adapters_create(desc: gdn_adapters_desc, a, ld_a, b, ld_b, scale):
    # (the handle belongs to the current device, and its calls read a and b there)
    if a.get_device() < 0 or a.get_device() != torch.cuda.current_device():
        raise GDNError(1, "a, b and scale must be on the current GPU")
    out = ctypes.c_void_p()
    _check(load_library().gdn_adapters_create(ctypes.byref(desc), _ptr(a), ld_a, _ptr(b), ld_b,
                                              _ptr(scale), ctypes.byref(out)))
    return out


def gdn_adapters_destroy(adapters: Adapters):
    _check(load_library().gdn_adapters_destroy(_released(adapters)))


def _proj_rows(t, rows, width, device, name):
    """Row stride of t [rows, width] with unit column stride (0: one row or none)."""
    if t.shape != (rows, width):
        raise GDNError(5, f"{name} must be [{rows}, {width}], got {tuple(t.shape)}")
    if _elsewhere(t, device):
        raise GDNError(1, f"{name} must be on the adapters' device")
    if rows == 0:
        return 0
    ld, unit = t.stride()
    if unit != 1 and width > 1:
        raise GDNError(1, f"{name} must have a unit column stride (strides {t.stride()})")
    if rows == 1:
        return 0
    if ld < width:  # an expanded row (stride 0) is not the library's "packed" (0)
        raise GDNError(1, f"{name}: row stride {ld} smaller than a row of {width}")
    return ld


def gdn_in_proj_adapted(pool: Pool, adapters: Adapters, x: torch.Tensor, w: torch.Tensor,
                        ids: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None):
    """y[t] = W x[t] + scale[a] B[a] (A[a] x[t]) with a = ids[t] (-1: none): x [tokens, hidden]
    and w [n_out, hidden] bf16, ids [tokens] int32, y [tokens, n_out] float32 or bf16 (default
    float32)."""
    tokens, device = ids.numel(), adapters.device
    hidden, n_out = adapters.hidden, adapters.n_out
    bf16 = torch.bfloat16
    if x.dtype != bf16 or w.dtype != bf16:
        raise GDNError(4, "x and w must be bf16")
    if ids.dtype != torch.int32 or _elsewhere(ids, device) or not ids.is_contiguous():
        raise GDNError(1, "ids must be a contiguous int32 tensor on the adapters' device")
    ld_x = _proj_rows(x, tokens, hidden, device, "x")
    ld_w = _proj_rows(w, n_out, hidden, device, "w")
    if y is None:
        y = torch.empty(tokens, n_out, dtype=torch.float32, device=ids.device)
    ld_y = _proj_rows(y, tokens, n_out, device, "y")
    status = _lib.gdn_in_proj_adapted(
        pool.handle, adapters.handle, tokens, x.data_ptr(), ld_x, w.data_ptr(), ld_w,
        ids.data_ptr(), y.data_ptr(), ld_y, _kv_dtype(y), stream.cuda_stream if stream is not None
        else torch._C._cuda_getCurrentRawStream(device))
    if status:
        _check(status)
    return y

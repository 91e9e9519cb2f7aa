"""Python binding of libdsaidx: argument marshalling only.

Every step of the indexer, and of the attention after it, runs in the library's CUDA kernels; this module
checks tensor shapes/dtypes, passes device pointers and the current CUDA
stream through the C ABI declared in include/dsaidx.h, and raises on a
non-zero status. There is no fallback: without the built library every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

FMT_BF16 = 0
FMT_FP8 = 1
FMT_FP4 = 2
KERNEL_KINDS = ("store", "plan", "score_bf16", "score_fp8", "score_fp4", "rope", "kv_store", "kv_load",
                "attn", "attn_join", "span_plan", "batch_plan")
HEADS = 64
HEAD_DIM = 128
PAGE_SIZE = 64

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsaidx.so")
_lib = None

_c_int = ctypes.c_int32
_c_i64 = ctypes.c_int64
_c_ptr = ctypes.c_void_p
_c_size = ctypes.c_size_t
_c_f64 = ctypes.c_double

ROPE_LAYOUTS = ("half", "interleaved")
ROPE_SCALINGS = ("none", "linear", "by_parts")


class _RopeDesc(ctypes.Structure):  # dsa_rope_desc
    _fields_ = [("theta", _c_f64), ("rot_dim", _c_int), ("max_pos", _c_int), ("layout", _c_int),
                ("scaling", _c_int), ("factor", _c_f64), ("orig_max_pos", _c_f64), ("beta_slow", _c_f64),
                ("beta_fast", _c_f64), ("mscale", _c_f64)]


# dsa_attn_args, field by field with the C padding
_ATTN_PACK = struct.Struct("@PqqPqqPPiiiiiPiPPiiPidPN").pack
_SPAN_PACK = struct.Struct("@PPPdi4x").pack  # dsa_span
_BATCH_PACK = struct.Struct("@12P5i4x").pack   # dsa_batch_args
_KV_PAGE_BYTES = {}  # of (kv_heads, head_dim, fmt)


class DsaError(RuntimeError):
    def __init__(self, where: str, status: int):
        super().__init__(f"{where}: {status_str(status)} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libdsaidx.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.dsa_ctx_create.argtypes = [ctypes.POINTER(_c_ptr), ctypes.c_float, ctypes.c_float, _c_int, _c_ptr]
        L.dsa_ctx_create.restype = ctypes.c_int
        L.dsa_ctx_destroy.argtypes = [_c_ptr]
        L.dsa_ctx_destroy.restype = ctypes.c_int
        L.dsa_cache_page_bytes.argtypes = [ctypes.c_int]
        L.dsa_cache_page_bytes.restype = _c_size
        L.dsa_index_store.argtypes = [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, _c_int, _c_int,
                                      _c_ptr, _c_int, ctypes.c_int, _c_ptr]
        L.dsa_index_store.restype = ctypes.c_int
        L.dsa_index_topk_workspace_size.argtypes = [_c_ptr, _c_int, _c_int, _c_int, ctypes.c_int]
        L.dsa_index_topk_workspace_size.restype = _c_size
        L.dsa_index_topk.argtypes = [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, ctypes.c_int, _c_ptr, _c_int,
                                     _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int, _c_ptr, _c_ptr,
                                     _c_ptr, _c_size, _c_ptr]
        L.dsa_index_topk.restype = ctypes.c_int
        L.dsa_index_topk_static.argtypes = [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_int, ctypes.c_int, _c_ptr,
                                            _c_int, _c_ptr, _c_ptr, _c_int, _c_int, _c_int, _c_int,
                                            _c_ptr, _c_ptr, _c_ptr]
        L.dsa_index_topk_static.restype = ctypes.c_int
        L.dsa_get_device_status.argtypes = [_c_ptr, _c_ptr]
        L.dsa_get_device_status.restype = ctypes.c_int
        L.dsa_selftest_bounded_wait.argtypes = [_c_ptr, _c_ptr]
        L.dsa_selftest_bounded_wait.restype = ctypes.c_int
        L.dsa_ctx_set_slot_output.argtypes = [_c_ptr, _c_int]
        L.dsa_ctx_set_slot_output.restype = ctypes.c_int
        L.dsa_ctx_set_hadamard.argtypes = [_c_ptr, _c_int]
        L.dsa_ctx_set_hadamard.restype = ctypes.c_int
        L.dsa_profile_enable.argtypes = [_c_ptr, ctypes.c_int]
        L.dsa_profile_enable.restype = ctypes.c_int
        L.dsa_profile_read.argtypes = [_c_ptr, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_c_int)]
        L.dsa_profile_read.restype = ctypes.c_int
        L.dsa_profile_read_kinds.argtypes = [_c_ptr, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_c_int), _c_int]
        L.dsa_profile_read_kinds.restype = ctypes.c_int
        L.dsa_rope_create.argtypes = [_c_ptr, ctypes.POINTER(_c_ptr), ctypes.POINTER(_RopeDesc)]
        L.dsa_rope_destroy.argtypes = [_c_ptr]
        L.dsa_rope_apply.argtypes = [_c_ptr, _c_ptr, _c_ptr, _c_ptr, ctypes.c_int, _c_ptr, _c_int, _c_int,
                                     _c_int, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_ptr]
        L.dsa_kv_page_bytes.argtypes = [_c_int, _c_int, ctypes.c_int]
        L.dsa_kv_page_bytes.restype = _c_size
        L.dsa_kv_store.argtypes = [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64, _c_ptr, _c_ptr, _c_ptr,
                                   _c_int, _c_int, _c_int, _c_int, _c_int, _c_ptr, _c_int, ctypes.c_int, _c_ptr,
                                   _c_ptr, _c_int, _c_ptr]
        L.dsa_kv_load.argtypes = [_c_ptr, _c_ptr, _c_int, ctypes.c_int, _c_int, _c_int, _c_ptr, _c_ptr, _c_ptr,
                                  _c_int, _c_int, _c_int, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64, _c_i64, _c_ptr]
        L.dsa_attn_workspace_size.argtypes = [_c_ptr, _c_int]
        L.dsa_attn_workspace_size.restype = _c_size
        L.dsa_tree_attn.argtypes = [_c_ptr, ctypes.c_char_p, _c_ptr]
        L.dsa_sparse_attn.argtypes = [_c_ptr, ctypes.c_char_p, _c_ptr, _c_int, _c_ptr]
        L.dsa_span_attn_workspace_size.argtypes = [_c_ptr] + [_c_int] * 5
        L.dsa_span_attn_workspace_size.restype = _c_size
        L.dsa_shared_attn_workspace_size.argtypes = [_c_ptr] + [_c_int] * 6
        L.dsa_shared_attn_workspace_size.restype = _c_size
        L.dsa_span_attn.argtypes = [_c_ptr, ctypes.c_char_p, ctypes.c_char_p, _c_ptr]
        L.dsa_shared_attn.argtypes = [_c_ptr, ctypes.c_char_p, ctypes.c_char_p, _c_ptr, _c_ptr, _c_int, _c_ptr]
        L.dsa_batch_plan.argtypes = [_c_ptr, ctypes.c_char_p, _c_ptr]
        for f in (L.dsa_rope_create, L.dsa_rope_destroy, L.dsa_rope_apply, L.dsa_kv_store, L.dsa_kv_load,
                  L.dsa_tree_attn, L.dsa_sparse_attn, L.dsa_span_attn, L.dsa_shared_attn, L.dsa_batch_plan):
            f.restype = ctypes.c_int
        L.dsa_status_str.argtypes = [ctypes.c_int]
        L.dsa_status_str.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_str(s: int) -> str:
    try:
        return lib().dsa_status_str(int(s)).decode()
    except RuntimeError:
        return f"status {s}"


def page_bytes(fmt: int) -> int:
    return int(lib().dsa_cache_page_bytes(int(fmt)))


def kv_page_bytes(kv_heads: int, head_dim: int, fmt: int) -> int:
    """Bytes of a K/V cache page (64 tokens, every kv head)."""
    return int(lib().dsa_kv_page_bytes(_c_int(kv_heads), _c_int(head_dim), int(fmt)))


def _stream_ptr(stream):
    if stream is None:
        import torch
        return _c_ptr(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return _c_ptr(stream)
    return _c_ptr(stream.cuda_stream)


def _dev(t, dtype, shape=None, name="tensor"):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _c_ptr(t.data_ptr())


# The calls below are made once a layer of a decode step, so their checks are
# written to cost little where nothing is wrong: plain integers instead of
# ctypes objects, one comparison per property, messages only on the way out.

_current_device = None


def _device():
    """The current device's index: the calls enqueue there, and the library
    compares it with the context's."""
    global _current_device
    if _current_device is None:
        import torch
        _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


def _ptr(t, dtype, shape, name, dev):
    """data_ptr of a contiguous tensor of that type and shape (None: any) on
    device `dev`."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, shape, name)       # says what is wrong
    raise ValueError(f"{name} is on another device than the current one")


def _rows(t, dtype, shape, name, dev):
    """Pointer and (token, head) strides of a [tokens, heads, dims] tensor on
    device `dev` whose dims are contiguous."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the current one")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    st, sh, sd = t.stride()
    T, H, D = shape
    if sd != 1 and D > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # a dimension of one element has no stride to speak of
    return t.data_ptr(), 0 if T <= 1 else st, 0 if H <= 1 else sh


_current_stream = None


def _raw_stream(stream):
    """The stream's address; the current one of the current device for None."""
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            # what torch.cuda.current_stream() asks, without the Stream object around the answer
            raw, dev = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            _current_stream = (lambda: raw(dev())) if raw and dev else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


class Rope:
    """A rotary plan (dsa_rope): the cos/sin table of one set of parameters.

    layout: "half" pairs (i, i + rot_dim/2), "interleaved" (2i, 2i+1).
    scaling: "none", "linear" (frequencies / factor) or "by_parts" (divided
    where a pair turns fewer than beta_slow times over orig_max_pos, kept where
    more than beta_fast times, blended between). mscale multiplies cos and sin.
    """

    def __init__(self, ctx: "Context", rot_dim: int, max_pos: int, theta: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, orig_max_pos: float = 32768, beta_slow: float = 1.0,
                 beta_fast: float = 32.0, mscale: float = 1.0):
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {ROPE_LAYOUTS}")
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {ROPE_SCALINGS}")
        self.rot_dim, self.max_pos = int(rot_dim), int(max_pos)
        d = _RopeDesc(float(theta), self.rot_dim, self.max_pos, ROPE_LAYOUTS.index(layout),
                      ROPE_SCALINGS.index(scaling), float(factor), float(orig_max_pos), float(beta_slow),
                      float(beta_fast), float(mscale))
        h = _c_ptr()
        st = lib().dsa_rope_create(ctx.handle, ctypes.byref(h), ctypes.byref(d))
        if st != 0:
            raise DsaError("dsa_rope_create", st)
        self._h = h

    @property
    def handle(self):
        return self._h

    def _open(self):
        if self._h is None:
            raise ValueError("the rotary plan is closed")
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().dsa_rope_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Context:
    """A library context on the current CUDA device (RoPE table, gamma,
    device status word)."""

    def __init__(self, theta: float = 10000.0, eps: float = 1e-6, max_pos: int = 131072,
                 gamma_bf16=None):
        self.theta = float(theta)
        self.eps = float(eps)
        self.max_pos = int(max_pos)
        h = _c_ptr()
        g = None
        if gamma_bf16 is not None:
            import numpy as np
            garr = np.ascontiguousarray(gamma_bf16, dtype=np.uint16)
            if garr.shape != (128,):
                raise ValueError("gamma_bf16 must be 128 bf16 bit patterns")
            self._gamma = garr
            g = _c_ptr(garr.ctypes.data)
        st = lib().dsa_ctx_create(ctypes.byref(h), ctypes.c_float(theta), ctypes.c_float(eps),
                                  _c_int(max_pos), g)
        if st != 0:
            raise DsaError("dsa_ctx_create", st)
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            lib().dsa_ctx_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def store(self, k_raw, rope_pos, seq_id, page_table, cache, num_pages: int, fmt: int,
              stream=None):
        """dsa_index_store: write RMSNorm+RoPE'd index keys into the paged cache."""
        import torch
        T = int(k_raw.shape[0]) if k_raw.dim() == 2 else -1
        B, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
        st = lib().dsa_index_store(
            self._h, _dev(k_raw, torch.bfloat16, (T, HEAD_DIM), "k_raw"),
            _dev(rope_pos, torch.int32, (T,), "rope_pos"), _dev(seq_id, torch.int32, (T,), "seq_id"),
            _dev(page_table, torch.int32, None, "page_table"), _c_int(T), _c_int(B), _c_int(max_pages),
            _dev(cache, torch.uint8, None, "cache"), _c_int(num_pages), int(fmt), _stream_ptr(stream))
        if st != 0:
            raise DsaError("dsa_index_store", st)

    def topk_workspace_size(self, Tq: int, B: int, k: int, fmt: int) -> int:
        return int(lib().dsa_index_topk_workspace_size(self._h, _c_int(Tq), _c_int(B), _c_int(k), int(fmt)))

    def topk(self, q, head_w, cache, num_pages: int, fmt: int, page_table, seq_lens, cu_q,
             causal: bool, k: int, out_idx, out_score, workspace, stream=None):
        """dsa_index_topk: per-query top-k key positions and scores."""
        import torch
        Tq = int(q.shape[0])
        B, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
        st = lib().dsa_index_topk(
            self._h, _dev(q, torch.bfloat16, (Tq, HEADS, HEAD_DIM), "q"),
            _dev(head_w, torch.float32, (Tq, HEADS), "head_w"), _dev(cache, torch.uint8, None, "cache"),
            _c_int(num_pages), int(fmt), _dev(page_table, torch.int32, None, "page_table"),
            _c_int(max_pages), _dev(seq_lens, torch.int32, (B,), "seq_lens"),
            _dev(cu_q, torch.int32, (B + 1,), "cu_q"), _c_int(B), _c_int(Tq), _c_int(1 if causal else 0),
            _c_int(k), _dev(out_idx, torch.int32, (Tq, k), "out_idx"),
            _dev(out_score, torch.float32, (Tq, k), "out_score"),
            _dev(workspace, torch.uint8, None, "workspace"), _c_size(workspace.numel()),
            _stream_ptr(stream))
        if st != 0:
            raise DsaError("dsa_index_topk", st)

    def topk_static(self, q, head_w, cache, num_pages: int, fmt: int, page_table, seq_lens, cu_q,
                    causal: bool, k: int, out_idx, out_score, stream=None):
        """dsa_index_topk_static: as topk(), with the library's fixed scratch
        array instead of a caller workspace (allocates nothing)."""
        import torch
        Tq = int(q.shape[0])
        B, max_pages = int(page_table.shape[0]), int(page_table.shape[1])
        st = lib().dsa_index_topk_static(
            self._h, _dev(q, torch.bfloat16, (Tq, HEADS, HEAD_DIM), "q"),
            _dev(head_w, torch.float32, (Tq, HEADS), "head_w"), _dev(cache, torch.uint8, None, "cache"),
            _c_int(num_pages), int(fmt), _dev(page_table, torch.int32, None, "page_table"),
            _c_int(max_pages), _dev(seq_lens, torch.int32, (B,), "seq_lens"),
            _dev(cu_q, torch.int32, (B + 1,), "cu_q"), _c_int(B), _c_int(Tq), _c_int(1 if causal else 0),
            _c_int(k), _dev(out_idx, torch.int32, (Tq, k), "out_idx"),
            _dev(out_score, torch.float32, (Tq, k), "out_score"), _stream_ptr(stream))
        if st != 0:
            raise DsaError("dsa_index_topk_static", st)

    def rope_apply(self, x, pos, rope: Rope, out=None, rot_start: int = 0, inverse: bool = False, stream=None):
        """dsa_rope_apply: rotate [T, H, D] rows (bf16, fp16 or fp32) to their
        positions, into `out` or in place. `inverse` turns back (the gradient)."""
        import torch
        dt = x.dtype if isinstance(x, torch.Tensor) else None
        code = 0 if dt is torch.bfloat16 else 1 if dt is torch.float16 else 2 if dt is torch.float32 else -1
        if code < 0:
            raise TypeError("x must be a bf16, fp16 or fp32 CUDA tensor")
        shape = x.shape
        if len(shape) != 3:
            raise ValueError(f"x must be [T, H, D], got {tuple(shape)}")
        T, H, D = shape
        dev = _device()
        xp, xt, xh = _rows(x, dt, shape, "x", dev)
        yp, yt, yh = (xp, xt, xh) if out is None else _rows(out, dt, shape, "out", dev)
        st = lib().dsa_rope_apply(self._h, rope._open(), xp, yp, code, _ptr(pos, torch.int32, (T,), "pos", dev), T, H, D,
                                  rot_start, xt, xh, yt, yh, 1 if inverse else 0, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_rope_apply", st)

    def kv_store(self, k, v, cache_pos, seq_id, page_table, cache, num_pages: int, fmt: int, rope=None,
                 rope_pos=None, rot_start: int = 0, stream=None):
        """dsa_kv_store: write [T, kv_heads, head_dim] bf16 keys (rotated when a
        plan is given) and values into the paged K/V cache."""
        import torch
        i32, shape, dev = torch.int32, k.shape, _device()
        kp, kt, kh = _rows(k, torch.bfloat16, shape, "k", dev)
        vp, vt, vh = _rows(v, torch.bfloat16, shape, "v", dev)
        T, n, D = shape
        B, max_pages = page_table.shape
        st = lib().dsa_kv_store(
            self._h, kp, vp, kt, kh, vt, vh, _ptr(cache_pos, i32, (T,), "cache_pos", dev), _ptr(seq_id, i32, (T,), "seq_id", dev),
            _ptr(page_table, i32, None, "page_table", dev), T, B, max_pages, n, D,
            self._kv_cache(cache, num_pages, n, D, fmt, dev), num_pages, fmt, None if rope is None else rope._open(),
            None if rope_pos is None else _ptr(rope_pos, i32, (T,), "rope_pos", dev), rot_start, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_kv_store", st)

    def kv_load(self, cache, num_pages: int, fmt: int, cache_pos, seq_id, page_table, k, v, stream=None):
        """dsa_kv_load: read tokens of the K/V cache back into k and v, [T,
        kv_heads, head_dim] bf16."""
        import torch
        i32, shape, dev = torch.int32, k.shape, _device()
        kp, kt, kh = _rows(k, torch.bfloat16, shape, "k", dev)
        vp, vt, vh = _rows(v, torch.bfloat16, shape, "v", dev)
        T, n, D = shape
        B, max_pages = page_table.shape
        st = lib().dsa_kv_load(
            self._h, self._kv_cache(cache, num_pages, n, D, fmt, dev), num_pages, fmt, n, D,
            _ptr(cache_pos, i32, (T,), "cache_pos", dev), _ptr(seq_id, i32, (T,), "seq_id", dev),
            _ptr(page_table, i32, None, "page_table", dev), T, B, max_pages, kp, vp, kt, kh, vt, vh, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_kv_load", st)

    @staticmethod
    def _kv_cache(cache, num_pages, kv_heads, head_dim, fmt, dev):
        """The cache's pointer, once it is known to hold that many pages."""
        import torch
        p = _ptr(cache, torch.uint8, None, "cache", dev)
        key = (kv_heads, head_dim, fmt)
        size = _KV_PAGE_BYTES.get(key)
        if size is None:
            size = _KV_PAGE_BYTES[key] = kv_page_bytes(*key)
        if cache.numel() < num_pages * size:
            raise ValueError(f"cache must have at least {num_pages * size} bytes, got {cache.numel()}")
        return p

    def attn_workspace_size(self, head_dim: int) -> int:
        return int(lib().dsa_attn_workspace_size(self._h, _c_int(head_dim)))

    def _attn_args(self, q, cache, num_pages, fmt, kv_heads, page_table, seq_lens, cu_q, out, workspace, mask, lse,
                   scale):
        """A dsa_attn_args as bytes."""
        import torch
        i32, bf16 = torch.int32, torch.bfloat16
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be a [Tq, heads, head_dim] tensor")
        shape = q.shape
        Tq, H, D = shape
        dev = _device()
        qp, qt, qh = _rows(q, bf16, shape, "q", dev)
        op, ot, oh = _rows(out, bf16, shape, "out", dev)
        B, max_pages = page_table.shape
        mp = words = 0
        if mask is not None:
            if mask.dim() != 2:
                raise ValueError("mask must be [Tq, words]")
            words = mask.shape[1]
            mp = _ptr(mask, i32, (Tq, words), "mask", dev)
        return _ATTN_PACK(
            qp, qt, qh, op, ot, oh, 0 if lse is None else _ptr(lse, torch.float32, (Tq, H), "lse", dev),
            self._kv_cache(cache, num_pages, kv_heads, D, fmt, dev), num_pages, fmt, H, kv_heads, D,
            _ptr(page_table, i32, None, "page_table", dev), max_pages, _ptr(seq_lens, i32, (B,), "seq_lens", dev),
            _ptr(cu_q, i32, (B + 1,), "cu_q", dev), B, Tq, mp, words, D ** -0.5 if scale is None else scale,
            _ptr(workspace, torch.uint8, None, "workspace", dev), workspace.numel())

    def tree_attn(self, q, cache, num_pages: int, fmt: int, kv_heads: int, page_table, seq_lens, cu_q, out,
                  workspace, mask=None, lse=None, scale=None, stream=None):
        """dsa_tree_attn: attention of each sequence's new tokens over its cache.
        mask: int32 [Tq, words], bit j of a row: it sees the sequence's j-th new
        token; None: token i sees the new tokens up to i."""
        a = self._attn_args(q, cache, num_pages, fmt, kv_heads, page_table, seq_lens, cu_q, out, workspace, mask,
                            lse, scale)
        st = lib().dsa_tree_attn(self._h, a, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_tree_attn", st)

    def sparse_attn(self, q, sel, cache, num_pages: int, fmt: int, kv_heads: int, page_table, seq_lens, cu_q, out,
                    workspace, mask=None, lse=None, scale=None, stream=None):
        """dsa_sparse_attn: attention of each query over its selected keys (topk()'s
        out_idx) and, with a mask, over the new tokens whose bits are set."""
        import torch
        if not isinstance(sel, torch.Tensor) or sel.dim() != 2:
            raise ValueError("sel must be a [Tq, k] tensor")
        k = sel.shape[1]
        a = self._attn_args(q, cache, num_pages, fmt, kv_heads, page_table, seq_lens, cu_q, out, workspace, mask,
                            lse, scale)
        st = lib().dsa_sparse_attn(self._h, a, _ptr(sel, torch.int32, (q.shape[0], k), "sel", q.get_device()), k, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_sparse_attn", st)

    def span_attn_workspace_size(self, Tq: int, B: int, heads: int, kv_heads: int, head_dim: int) -> int:
        return int(lib().dsa_span_attn_workspace_size(self._h, Tq, B, heads, kv_heads, head_dim))

    def shared_attn_workspace_size(self, Tq: int, B: int, n_groups: int, heads: int, kv_heads: int, head_dim: int) -> int:
        return int(lib().dsa_shared_attn_workspace_size(self._h, Tq, B, n_groups, heads, kv_heads, head_dim))

    @staticmethod
    def _span(q, cap, slopes, window, first, last):
        """A dsa_span as bytes."""
        import torch
        Tq, H, _ = q.shape
        dev = q.get_device()
        return _SPAN_PACK(0 if first is None else _ptr(first, torch.int32, (Tq,), "first", dev),
                          0 if last is None else _ptr(last, torch.int32, (Tq,), "last", dev),
                          0 if slopes is None else _ptr(slopes, torch.float32, (H,), "slopes", dev), cap, window)

    def span_attn(self, q, cache, num_pages: int, fmt: int, kv_heads: int, page_table, seq_lens, cu_q, out, workspace,
                  mask=None, lse=None, scale=None, cap: float = 0.0, slopes=None, window: int = 0, first=None, last=None,
                  stream=None):
        """dsa_span_attn: as tree_attn(), each new token over a span of places.
        first, last: int32 [Tq], the first place and one past the last one that
        a token sees; window: how many places it looks back over, itself
        included (of places, with a mask too: a drafted token's depth is not
        counted); cap: scores become cap * tanh(score / cap); slopes: fp32
        [heads], times the distance in places, taken off the scores."""
        a = self._attn_args(q, cache, num_pages, fmt, kv_heads, page_table, seq_lens, cu_q, out, workspace, mask,
                            lse, scale)
        st = lib().dsa_span_attn(self._h, a, self._span(q, cap, slopes, window, first, last), _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_span_attn", st)

    def shared_attn(self, q, cache, num_pages: int, fmt: int, kv_heads: int, page_table, seq_lens, cu_q, out, workspace,
                    cu_groups, shared_lens, mask=None, lse=None, scale=None, cap: float = 0.0, slopes=None,
                    window: int = 0, first=None, last=None, stream=None):
        """dsa_shared_attn: span_attn() for a batch whose sequences cu_groups[g] ..
        cu_groups[g+1]-1 have their first shared_lens[g] tokens in common, in the
        same pages: those are read once a group."""
        import torch
        a = self._attn_args(q, cache, num_pages, fmt, kv_heads, page_table, seq_lens, cu_q, out, workspace, mask,
                            lse, scale)
        n, dev = shared_lens.shape[0], q.get_device()
        st = lib().dsa_shared_attn(self._h, a, self._span(q, cap, slopes, window, first, last),
                                   _ptr(cu_groups, torch.int32, (n + 1,), "cu_groups", dev),
                                   _ptr(shared_lens, torch.int32, (n,), "shared_lens", dev), n, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_shared_attn", st)

    def batch_plan(self, old_lens, new_lens, page_table, num_pages: int, free_pages, free_count, free_left, seq_lens,
                   cu_q, seq_id, cache_pos, slots=None, own_from=None, stream=None):
        """dsa_batch_plan: a step's page tables and slot maps from its requests'
        lengths. Sequence b's new_lens[b] tokens follow the old_lens[b] in the
        cache (negative: it ends and its pages from own_from[b] on come back);
        pages come off the stack free_pages[:free_count]. Writes page_table,
        free_pages, free_left [1], seq_lens [B], cu_q [B+1] and seq_id,
        cache_pos, slots [T], which are -1 past the last token."""
        import torch
        i32, dev = torch.int32, _device()
        B, max_pages = page_table.shape
        T = seq_id.shape[0]
        a = _BATCH_PACK(
            _ptr(old_lens, i32, (B,), "old_lens", dev), _ptr(new_lens, i32, (B,), "new_lens", dev),
            0 if own_from is None else _ptr(own_from, i32, (B,), "own_from", dev), _ptr(free_count, i32, (1,), "free_count", dev),
            _ptr(page_table, i32, None, "page_table", dev), _ptr(free_pages, i32, None, "free_pages", dev),
            _ptr(free_left, i32, (1,), "free_left", dev), _ptr(seq_lens, i32, (B,), "seq_lens", dev),
            _ptr(cu_q, i32, (B + 1,), "cu_q", dev), _ptr(seq_id, i32, (T,), "seq_id", dev),
            _ptr(cache_pos, i32, (T,), "cache_pos", dev), 0 if slots is None else _ptr(slots, i32, (T,), "slots", dev),
            B, T, max_pages, num_pages, free_pages.numel())
        st = lib().dsa_batch_plan(self._h, a, _raw_stream(stream))
        if st != 0:
            raise DsaError("dsa_batch_plan", st)

    def set_hadamard(self, on: bool = True):
        """Store keys (and rotate queries) with the 128-point Walsh-Hadamard transform."""
        st = lib().dsa_ctx_set_hadamard(self._h, 1 if on else 0)
        if st != 0:
            raise DsaError("dsa_ctx_set_hadamard", st)

    def selftest_bounded_wait(self, stream=None):
        """Enqueue the bounded-wait self-test (records a timeout in the status)."""
        st = lib().dsa_selftest_bounded_wait(self._h, _stream_ptr(stream))
        if st != 0:
            raise DsaError("dsa_selftest_bounded_wait", st)

    def set_slot_output(self, on: bool = True):
        """Top-k returns cache slots (page * 64 + offset) instead of positions, and
        sparse_attn() reads its selection as slots."""
        st = lib().dsa_ctx_set_slot_output(self._h, 1 if on else 0)
        if st != 0:
            raise DsaError("dsa_ctx_set_slot_output", st)

    def profile_enable(self, on: bool = True):
        st = lib().dsa_profile_enable(self._h, 1 if on else 0)
        if st != 0:
            raise DsaError("dsa_profile_enable", st)

    def profile_read(self):
        """{kind: (total ms, launches)} since the previous read (synchronises)."""
        ms = (ctypes.c_float * len(KERNEL_KINDS))()
        n = (_c_int * len(KERNEL_KINDS))()
        st = lib().dsa_profile_read_kinds(self._h, ms, n, len(KERNEL_KINDS))
        if st != 0:
            raise DsaError("dsa_profile_read_kinds", st)
        return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(KERNEL_KINDS)}

    def device_status(self, stream=None) -> int:
        """Synchronise the stream; read and clear the device status word."""
        return int(lib().dsa_get_device_status(self._h, _stream_ptr(stream)))

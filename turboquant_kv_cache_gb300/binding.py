"""Thin Python binding of libtq (the C ABI in include/tq.h).

Argument marshalling only: every function here checks shapes, takes raw
pointers from torch tensors, calls the C entry point of the same name on the
caller's current CUDA stream, or on `stream` (a torch.cuda.Stream), and raises
TQError on a non-zero status.  What a call makes for itself or returns anew is
made on that stream and is its memory, as if it were the current one.  All
computation happens in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libtq.so")
_lib = None

TQ_F16, TQ_F32 = 0, 1


class TQError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _load().tq_strerror(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: tq status {status} ({msg})")


class tq_layout(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("block", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("qjl_m", ctypes.c_int32), ("norm_correct", ctypes.c_int32), ("codebook", ctypes.c_int32),
                ("sign_seed", ctypes.c_uint64)]


class tq_kv_view(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("qjl_bits", ctypes.c_void_p),
                ("qjl_rnorm", ctypes.c_void_p), ("S", ctypes.c_void_p), ("layout", tq_layout),
                ("page_table", ctypes.c_void_p), ("page_size", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32)]


class tq_page_pool(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_void_p), ("ref", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libtq.so not built at {_LIB_PATH}: run `python -m turboquant_kv_cache_gb300.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "tq_codebook": (I, [I, I, P, P]),
        "tq_codebook_f64": (I, [I, I, P, P]),
        "tq_codebook_kind": (I, [I, I, I, P, P]),
        "tq_signs": (I, [ctypes.c_uint64, I, P]),
        "tq_layout_sizes": (I, [P, P, P, P]),
        "tq_quantize_kv": (I, [P, P, I, I64, I64, P, P, P, P, P, P]),
        "tq_append_kv": (I, [P, P, I, I, I, I, I64, P, I64, P, I, I, P, P, P, P, P, P]),
        "tq_dequantize_kv": (I, [P, P, P, P, P, P, I64, P, I, P]),
        "tq_decode_attn": (I, [P, P, P, I, I, I, I64, P, I64, ctypes.c_float, P, P, SZ, I, P]),
        "tq_decode_workspace_bytes": (I, [I, I, I, I, I64, I, P, P]),
        "tq_decode_attn_window": (I, [P, P, P, I, I, I, I64, P, I64, P, P, I, P, I, ctypes.c_float, P, P, SZ, I, P]),
        "tq_decode_window_workspace_bytes": (I, [I, I, I, I, I64, I, P]),
        "tq_polar_code_bytes": (I, [I, I, P]),
        "tq_to_blocks": (I, [P, P, P, I64, P, P]),
        "tq_from_blocks": (I, [P, P, I64, P, P, P]),
        "tq_decode_attn_blocks": (I, [P, P, P, P, P, I, I, I, I64, P, I64, ctypes.c_float, P, P, SZ, I, P]),
        "tq_polar_quantize": (I, [P, I, I64, I, I64, I, P, P, P]),
        "tq_polar_dequantize": (I, [P, P, I64, I, I, P, I, P]),
        "tq_decode_attn_static": (I, [P, P, P, I, I, I, I64, P, I64, ctypes.c_float, P, I, P]),
        "tq_prefill_attn": (I, [P, P, P, I, I, I, I, I64, I64, I, ctypes.c_float, P, P, SZ, P]),
        "tq_prefill_workspace_bytes": (I, [I, I, I, I, I, I64, P]),
        "tq_decode_attn_shared": (I, [P, P, I64, P, I64, P, P, P, I, I, I, I64, P, I64, ctypes.c_float, P, P, SZ, I, P]),
        "tq_decode_shared_workspace_bytes": (I, [I, I, I, I, I64, I64, I, P]),
        "tq_qkv_norm_rope": (I, [P, I, I, I, I, I, I, I64, P, P, ctypes.c_float, P, I64, I, I, P, P, P, P, P, I64, P, P]),
        "tq_pages_fork": (I, [P, P, I, I, P, P, P, P, I, P, P, SZ, P]),
        "tq_pages_free": (I, [P, P, P, I, P]),
        "tq_pages_compact": (I, [P, P, I, I, P, P, SZ, P]),
        "tq_pages_workspace_bytes": (I, [I, I, I, P]),
        "tq_set_wait_limit_ns": (I, [ctypes.c_uint64]),
        "tq_device_status": (I, [I, I, P]),
        "tq_strerror": (ctypes.c_char_p, [I]),
        "tq_version": (I, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def library():
    """The loaded ctypes library (raises if libtq.so is missing)."""
    return _load()


# ------------------------------------------------------------------ helpers
CODEBOOK_GAUSSIAN, CODEBOOK_BETA = 0, 1


def make_layout(head_dim, block, bits, qjl_m=0, norm_correct=0, sign_seed=1, codebook=CODEBOOK_GAUSSIAN):
    return tq_layout(head_dim, block, bits, qjl_m, norm_correct, codebook, sign_seed)


def _ptr(t):
    return t.data_ptr() if t is not None else None


# the current stream's handle without building a Stream object (3 us of host
# time a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# the current device without the check that CUDA has been initialised (a CUDA
# tensor is at hand where it is used)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _stream_on(stream, dev):
    """The same where dev is the current device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    if stream is not None and stream.device_index != dev:
        raise ValueError("stream must be a stream of the call's CUDA device")
    return _stream(stream)


def _new(stream, make, *args, **kw):
    """A tensor that a call makes for itself or returns, made on the call's
    stream: fills and copies are in the kernels' order, and the memory, once
    let go, is that stream's to use again."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


class _on:
    """Makes a tensor's device current for the calls inside."""

    def __init__(self, dev):
        self.dev = dev

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        torch.cuda.set_device(self.dev)

    def __exit__(self, *exc):
        torch.cuda.set_device(self.prev)


def _is(t, dtype, shape, dev):
    """Whether t is a contiguous tensor of this type and shape on CUDA device dev."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _i32(t, n, name, dev):
    """Checks a contiguous int32 tensor of n values (or None) on device dev."""
    if t is not None and not (t.dtype is torch.int32 and t.numel() == n and t.get_device() == dev
                              and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} values on the call's CUDA device")


def _check_workspace(w, dev):
    if w.get_device() != dev or not w.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the call's CUDA device")


def _check(st, where):
    if st != 0:
        raise TQError(st, where)


def _dtype_code(dt):
    if dt == torch.float16:
        return TQ_F16
    if dt == torch.float32:
        return TQ_F32
    raise TypeError(f"unsupported dtype {dt}")


# ------------------------------------------------------------------ host calls
def tq_codebook(bits, block, f64=False):
    """(centroids, boundaries) as Python lists (host call)."""
    lib = _load()
    K = 1 << bits
    T = ctypes.c_double if f64 else ctypes.c_float
    c = (T * K)()
    b = (T * max(K - 1, 1))()
    _check((lib.tq_codebook_f64 if f64 else lib.tq_codebook)(bits, block, c, b), "tq_codebook")
    return list(c), list(b)[:K - 1]


def tq_codebook_kind(bits, block, kind):
    """(centroids, boundaries) in double precision for a codebook kind
    (CODEBOOK_GAUSSIAN or CODEBOOK_BETA)."""
    lib = _load()
    K = 1 << bits
    c = (ctypes.c_double * K)()
    b = (ctypes.c_double * max(K - 1, 1))()
    _check(lib.tq_codebook_kind(bits, block, kind, c, b), "tq_codebook_kind")
    return list(c), list(b)[:K - 1]


def tq_signs(sign_seed, d):
    lib = _load()
    out = (ctypes.c_int8 * d)()
    _check(lib.tq_signs(ctypes.c_uint64(sign_seed), d, out), "tq_signs")
    return list(out)


def tq_layout_sizes(layout):
    lib = _load()
    cb, ns, qb = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib.tq_layout_sizes(ctypes.byref(layout), ctypes.byref(cb), ctypes.byref(ns), ctypes.byref(qb)),
           "tq_layout_sizes")
    return cb.value, ns.value, qb.value


def tq_decode_workspace_bytes(B, Hq, Hkv, head_dim, ctx, n_split=0):
    lib = _load()
    nb, ns = ctypes.c_size_t(), ctypes.c_int()
    _check(lib.tq_decode_workspace_bytes(B, Hq, Hkv, head_dim, ctx, n_split, ctypes.byref(nb), ctypes.byref(ns)),
           "tq_decode_workspace_bytes")
    return nb.value, ns.value


def tq_prefill_workspace_bytes(B, Hq, Hkv, head_dim, Tq, ctx):
    lib = _load()
    nb = ctypes.c_size_t()
    _check(lib.tq_prefill_workspace_bytes(B, Hq, Hkv, head_dim, Tq, ctx, ctypes.byref(nb)),
           "tq_prefill_workspace_bytes")
    return nb.value


# ------------------------------------------------------------------ packed cache
class PackedKV:
    """Device buffers of one packed cache (K or V): codes [N, code_bytes]
    uint8, scales [N, d/block] fp16, and with QJL qjl [N, m/8] uint8, rnorm
    [N] fp16 and the projection S [m, d] fp32.  N may carry leading dims.

    As an attention cache the lead shape is [B, Hkv, S_cap] (contiguous), or
    [num_pages, Hkv, page_size] with page_table an int32 CUDA tensor
    [B, pages_per_seq] (paged: token t of batch b is row t % page_size of
    page page_table[b, t // page_size])."""

    def __init__(self, layout, lead_shape, device="cuda", S=None, page_table=None):
        cb, ns, qb = tq_layout_sizes(layout)
        self.layout = layout
        self.lead_shape = tuple(lead_shape)
        self.page_table = page_table
        if page_table is not None:
            if (page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_cuda
                    or len(self.lead_shape) != 3):
                raise ValueError("paged cache: lead shape [num_pages, Hkv, page_size] and an int32 CUDA "
                                 "page table [B, pages_per_seq]")
        self.codes = torch.empty(self.lead_shape + (cb,), dtype=torch.uint8, device=device)
        self.scales = torch.empty(self.lead_shape + (ns,), dtype=torch.float16, device=device)
        self.qjl = torch.empty(self.lead_shape + (qb,), dtype=torch.uint8, device=device) if qb else None
        self.rnorm = torch.empty(self.lead_shape, dtype=torch.float16, device=device) if qb else None
        self.S = S

    @classmethod
    def of(cls, layout, codes, scales, qjl=None, rnorm=None, S=None, page_table=None):
        """A PackedKV over arrays that exist already (contiguous; the lead
        shape is codes.shape[:-1]).  A table may be part of a wider one (its
        rows then lie further apart than they are long)."""
        lead = tuple(codes.shape[:-1])
        if page_table is not None and (page_table.dtype != torch.int32 or page_table.dim() != 2 or len(lead) != 3
                                       or page_table.device != codes.device or page_table.stride(1) != 1):
            raise ValueError("paged cache: lead shape [num_pages, Hkv, page_size] and an int32 page table "
                             "[B, pages_per_seq] on its device")
        self = cls.__new__(cls)
        self.layout, self.lead_shape, self.page_table, self.S = layout, lead, page_table, S
        self.codes, self.scales, self.qjl, self.rnorm = codes, scales, qjl, rnorm
        self.check_arrays()
        return self

    def check_arrays(self):
        """Raises ValueError where an array is not what the layout and the lead
        shape say."""
        cb, ns, qb = tq_layout_sizes(self.layout)
        if qb and (self.qjl is None or self.rnorm is None):
            raise ValueError("a layout with QJL has its sign bits and residual norms")
        for t, dt, tail in ((self.codes, torch.uint8, (cb,)), (self.scales, torch.float16, (ns,)),
                            (self.qjl if qb else None, torch.uint8, (qb,)), (self.rnorm if qb else None, torch.float16, ())):
            if t is not None and (t.dtype != dt or tuple(t.shape) != self.lead_shape + tail or not t.is_contiguous()
                                  or t.device != self.codes.device):
                raise ValueError("arrays must be contiguous, of one lead shape and device, as the layout has them")

    @property
    def n_vec(self):
        n = 1
        for s in self.lead_shape:
            n *= s
        return n

    @property
    def heads(self):
        return self.lead_shape[1]

    @property
    def batch(self):
        return self.page_table.shape[0] if self.page_table is not None else self.lead_shape[0]

    @property
    def capacity(self):
        """Slots per (batch, head): S_cap."""
        if self.page_table is not None:
            return self.page_table.shape[1] * self.lead_shape[2]
        return self.lead_shape[2]

    def view(self):
        """The C view of the cache as it is now, the caller's own."""
        v = tq_kv_view(self.codes.data_ptr(), self.scales.data_ptr())
        v.layout = self.layout
        if self.qjl is not None:
            v.qjl_bits, v.qjl_rnorm = self.qjl.data_ptr(), _ptr(self.rnorm)
        if self.S is not None:
            v.S = self.S.data_ptr()
        if self.page_table is not None:
            v.page_table, v.page_size = self.page_table.data_ptr(), self.lead_shape[2]
            v.pages_per_seq = self._table_stride()
        return v

    _kept = (None, None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_kept"}   # addresses are not copied or pickled

    def _view_ref(self):
        """view() by reference, for a C call of this module: nobody changes it,
        so it is kept while all that it is made of is what it was."""
        of = self.codes.data_ptr(), self.scales.data_ptr(), bytes(self.layout)
        pt = self.page_table
        if pt is not None:
            of += pt.data_ptr(), self.lead_shape[2], pt.shape, pt.stride()
        if self.qjl is not None or self.S is not None:
            of += _ptr(self.qjl), _ptr(self.rnorm), _ptr(self.S)
        if of != self._kept[0]:
            self._kept = of, ctypes.byref(self.view())
        return self._kept[1]

    def _table_stride(self):
        """Entries between two rows of the table (its width unless it is part of a wider one)."""
        pt = self.page_table
        if pt is None:
            return 0
        if pt.shape[1] > 1 and pt.stride(1) != 1:
            raise ValueError("a page table's rows must be contiguous")
        return pt.stride(0) if pt.shape[0] > 1 else pt.shape[1]

    def nbytes(self):
        n = self.codes.numel() + 2 * self.scales.numel()
        if self.qjl is not None:
            n += self.qjl.numel() + 2 * self.rnorm.numel()
        return n


# ------------------------------------------------------------------ device calls
def tq_quantize_kv(layout, x, S=None, out=None, stream=None):
    """Quantise x [..., d] (fp16/fp32, CUDA, last dim contiguous) into a
    PackedKV with leading shape x.shape[:-1]."""
    lib = _load()
    d = layout.head_dim
    if x.shape[-1] != d or x.stride(-1) != 1:
        raise ValueError("x must have a contiguous last dimension of head_dim")
    lead = tuple(x.shape[:-1])
    x2 = _new(stream, x.reshape, -1, d)
    if out is None:
        out = _new(stream, PackedKV, layout, lead, device=x.device, S=S)
    n = x2.shape[0]
    st = lib.tq_quantize_kv(ctypes.byref(layout), _ptr(x2), _dtype_code(x.dtype), n, x2.stride(0), _ptr(S),
                            _ptr(out.codes), _ptr(out.scales), _ptr(out.qjl), _ptr(out.rnorm), _stream(stream))
    _check(st, "tq_quantize_kv")
    return out


def tq_append_kv(cache, x, pos, stream=None):
    """Quantise new tokens x [B, H, n_new, d] (fp16/fp32, CUDA, last dim
    contiguous, rows of one (b, h) contiguous) into a PackedKV cache of
    leading shape [B, H, S_cap]: token j of (b, h) lands in slot pos[b] + j
    (pos: int32 CUDA tensor [B]); slots outside [0, S_cap) are skipped."""
    lib = _load()
    layout = cache.layout
    d = layout.head_dim
    if x.dim() != 4 or x.shape[-1] != d or x.stride(-1) != 1:
        raise ValueError("x must be [B, H, n_new, head_dim] with a contiguous last dimension")
    B, H, n_new, _ = x.shape
    if len(cache.lead_shape) != 3 or (cache.batch, cache.heads) != (B, H):
        raise ValueError("cache must have leading shape [B, H, S_cap] (or be paged for B sequences) matching x")
    if pos.dtype != torch.int32 or pos.numel() != B or not pos.is_cuda:
        raise ValueError("pos must be an int32 CUDA tensor of B slot offsets")
    x2 = _new(stream, x.reshape, -1, d)
    pos = _new(stream, pos.contiguous)
    pt = cache.page_table
    st = lib.tq_append_kv(ctypes.byref(layout), _ptr(x2), _dtype_code(x.dtype), B, H, n_new, x2.stride(0),
                          _ptr(pos), cache.capacity, _ptr(pt),
                          cache.lead_shape[2] if pt is not None else 0, cache._table_stride(),
                          _ptr(cache.S), _ptr(cache.codes), _ptr(cache.scales), _ptr(cache.qjl), _ptr(cache.rnorm),
                          _stream(stream))
    _check(st, "tq_append_kv")
    return cache


def tq_dequantize_kv(packed, out_dtype=torch.float16, stream=None, out=None):
    lib = _load()
    d = packed.layout.head_dim
    if out is None:
        out = _new(stream, torch.empty, packed.lead_shape + (d,), dtype=out_dtype, device=packed.codes.device)
    elif out.dtype != out_dtype or out.numel() != packed.n_vec * d or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of n_vec x head_dim elements of out_dtype")
    st = lib.tq_dequantize_kv(ctypes.byref(packed.layout), _ptr(packed.codes), _ptr(packed.scales),
                              _ptr(packed.qjl), _ptr(packed.rnorm), _ptr(packed.S), packed.n_vec, _ptr(out),
                              _dtype_code(out_dtype), _stream(stream))
    _check(st, "tq_dequantize_kv")
    return out


def _cache_for(K, V, B):
    """Heads and S_cap of a K/V cache pair read by B sequences."""
    k, v, table = K.lead_shape, V.lead_shape, K.page_table
    if table is V.page_table and len(k) == 3 and k[1:] == v[1:]:   # the usual pair
        if table is not None:
            n, pages = table.shape
            if n >= B:
                return k[1], pages * k[2]
        elif k[0] >= B and v[0] >= B:
            return k[1], k[2]
    if K.batch < B or V.batch < B or (K.heads, K.capacity) != (V.heads, V.capacity):
        raise ValueError("K and V caches must hold the same heads and slots for at least B sequences")
    return K.heads, K.capacity


def tq_decode_attn(K, V, q, ctx=None, kv_len=None, softmax_scale=0.0, n_split=0, workspace=None, out=None,
                   stream=None):
    """q [B, Hq, d] fp16; K, V PackedKV caches (contiguous [B, Hkv, S_cap]
    or paged with one page table)."""
    lib = _load()
    B, Hq, d = q.shape
    Hkv, S_cap = _cache_for(K, V, B)
    ctx = S_cap if ctx is None else ctx
    need, ns = tq_decode_workspace_bytes(B, Hq, Hkv, d, ctx, n_split)
    if workspace is None:
        workspace = _new(stream, torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    kv, vv = K._view_ref(), V._view_ref()
    st = lib.tq_decode_attn(kv, vv, _ptr(q), B, Hq, Hkv, S_cap, _ptr(kv_len), ctx,
                            float(softmax_scale), _ptr(out), _ptr(workspace), workspace.numel(), n_split,
                            _stream(stream))
    _check(st, "tq_decode_attn")
    return out


def tq_decode_attn_static(K, V, q, ctx=None, kv_len=None, softmax_scale=0.0, n_split=0, out=None, stream=None):
    """tq_decode_attn without a workspace: the library's own fixed device
    array holds the split partials (for callers that cannot allocate)."""
    lib = _load()
    B, Hq, d = q.shape
    Hkv, S_cap = _cache_for(K, V, B)
    ctx = S_cap if ctx is None else ctx
    if out is None:
        out = _new(stream, torch.empty_like, q)
    kv, vv = K._view_ref(), V._view_ref()
    st = lib.tq_decode_attn_static(kv, vv, _ptr(q), B, Hq, Hkv, S_cap, _ptr(kv_len),
                                   ctx, float(softmax_scale), _ptr(out), n_split, _stream(stream))
    _check(st, "tq_decode_attn_static")
    return out


def tq_decode_window_workspace_bytes(B, Hq, Hkv, head_dim, ctx, n_split=0):
    lib = _load()
    nb = ctypes.c_size_t()
    _check(lib.tq_decode_window_workspace_bytes(B, Hq, Hkv, head_dim, ctx, n_split, ctypes.byref(nb)),
           "tq_decode_window_workspace_bytes")
    return nb.value


def tq_decode_attn_window(K, V, q, k_win, v_win, ctx=None, kv_len=None, win_len=None, win=None, softmax_scale=0.0,
                          n_split=0, workspace=None, out=None, stream=None):
    """Decode over the packed cache plus an fp16 residual window: k_win,
    v_win [B, Hkv, W_cap, d] fp16 CUDA (contiguous, unrotated); win_len an
    int32 CUDA tensor [B] of window tokens, or win for every batch (default
    W_cap)."""
    lib = _load()
    B, Hq, d = q.shape
    Hkv, S_cap = _cache_for(K, V, B)
    ctx = S_cap if ctx is None else ctx
    if k_win.shape != v_win.shape or k_win.dim() != 4 or tuple(k_win.shape[:2]) != (B, Hkv) or k_win.shape[3] != d:
        raise ValueError("k_win, v_win must be [B, Hkv, W_cap, head_dim]")
    if k_win.dtype != torch.float16 or v_win.dtype != torch.float16:
        raise ValueError("the window is fp16")
    k_win, v_win = _new(stream, k_win.contiguous), _new(stream, v_win.contiguous)
    W_cap = k_win.shape[2]
    if win_len is not None and (win_len.dtype != torch.int32 or win_len.numel() != B or not win_len.is_cuda):
        raise ValueError("win_len must be an int32 CUDA tensor of B window lengths")
    win = W_cap if win is None else win
    need = tq_decode_window_workspace_bytes(B, Hq, Hkv, d, ctx, n_split)
    if workspace is None:
        workspace = _new(stream, torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    kv, vv = K._view_ref(), V._view_ref()
    st = lib.tq_decode_attn_window(kv, vv, _ptr(q), B, Hq, Hkv, S_cap, _ptr(kv_len), ctx,
                                   _ptr(k_win), _ptr(v_win), W_cap, _ptr(win_len), win, float(softmax_scale),
                                   _ptr(out), _ptr(workspace), workspace.numel(), n_split, _stream(stream))
    _check(st, "tq_decode_attn_window")
    return out


def tq_decode_shared_workspace_bytes(B, Hq, Hkv, head_dim, prefix_ctx, ctx, n_split=0):
    lib = _load()
    nb = ctypes.c_size_t()
    _check(lib.tq_decode_shared_workspace_bytes(B, Hq, Hkv, head_dim, prefix_ctx, ctx, n_split, ctypes.byref(nb)),
           "tq_decode_shared_workspace_bytes")
    return nb.value


def tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx=None, prefix_len=None, ctx=None, kv_len=None, softmax_scale=0.0,
                          n_split=0, workspace=None, out=None, stream=None):
    """Decode attention of q [B, Hq, d] fp16 over a prefix that all B
    sequences share (Kp, Vp: PackedKV caches of one sequence) and each
    sequence's own tokens behind it (K, V: caches as in tq_decode_attn, or
    None when there are none yet).  prefix_len: int32 CUDA tensor of one
    value, kv_len: int32 CUDA tensor [B]; prefix_ctx and ctx bound them."""
    dev, shape = q.get_device(), q.shape
    if len(shape) != 3 or dev < 0 or q.dtype is not torch.float16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous fp16 CUDA tensor [B, Hq, head_dim]")
    if dev != _current_device():
        with _on(dev):
            return tq_decode_attn_shared(Kp, Vp, K, V, q, prefix_ctx, prefix_len, ctx, kv_len, softmax_scale, n_split,
                                         workspace, out, stream)
    B, Hq, d = shape
    Hkv, P_cap = _cache_for(Kp, Vp, 1)
    if prefix_ctx is None:
        prefix_ctx = P_cap
    if (K is None) != (V is None):
        raise ValueError("K and V, the sequences' own caches, are given together or left out together")
    if K is not None:
        heads, S_cap = _cache_for(K, V, B)
        if heads != Hkv:
            raise ValueError("prefix and own caches must hold the same heads")
        if K.codes.get_device() != dev or V.codes.get_device() != dev:
            raise ValueError("caches must have q's head_dim and device")
        kv, vv = K._view_ref(), V._view_ref()
    else:
        S_cap = 0
        kv = vv = None
    if ctx is None:
        ctx = S_cap
    # the call itself checks that all layouts agree
    if Kp.layout.head_dim != d or Kp.codes.get_device() != dev or Vp.codes.get_device() != dev:
        raise ValueError("caches must have q's head_dim and device")
    if prefix_len is not None:
        _i32(prefix_len, 1, "prefix_len", dev)
    if kv_len is not None:
        _i32(kv_len, B, "kv_len", dev)
    if workspace is None:
        need = tq_decode_shared_workspace_bytes(B, Hq, Hkv, d, prefix_ctx, ctx, n_split)
        workspace = _new(stream, torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    else:
        _check_workspace(workspace, dev)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    elif not _is(out, torch.float16, shape, dev):
        raise ValueError("out must be a contiguous tensor like q")
    st = _load().tq_decode_attn_shared(Kp._view_ref(), Vp._view_ref(), P_cap, _ptr(prefix_len),
                                       prefix_ctx, kv, vv, q.data_ptr(), B, Hq, Hkv, S_cap, _ptr(kv_len), ctx, softmax_scale,
                                       out.data_ptr(), workspace.data_ptr(), workspace.nbytes, n_split,
                                       _stream_on(stream, dev))
    if st:
        _check(st, "tq_decode_attn_shared")
    return out


def tq_qkv_norm_rope(qkv, Hq, Hkv, head_dim, q_weight=None, k_weight=None, eps=1e-6, rope=None, interleaved=False,
                     pos=None, new_len=None, slot=None, q_out=None, k_out=None, v_out=None, stream=None):
    """Projection rows qkv [B, T, (Hq + 2 Hkv) head_dim] (fp16/fp32, CUDA; rows
    may lie further apart than they are long) to normalised, rotated queries
    [B, Hq, T, d] and keys, and values, [B, Hkv, cap, d], all fp16.  q_weight,
    k_weight: fp32 [d] or None; rope: fp32 [n_pos, rot_dim] (cosines, then
    sines) or None; pos, new_len, slot: int32 [B] or None.  k_out and v_out
    default to new arrays of cap = T (cap: their third dimension).  In an
    output that is given, what no token goes to is left as it was; in a new
    one it is zero."""
    d = head_dim
    dev, shape = qkv.get_device(), qkv.shape
    if len(shape) != 3 or shape[2] != (Hq + 2 * Hkv) * d or dev < 0:
        raise ValueError("qkv must be a CUDA tensor [B, T, (Hq + 2 Hkv) head_dim] with a contiguous last dimension")
    if dev != _current_device():
        with _on(dev):
            return tq_qkv_norm_rope(qkv, Hq, Hkv, d, q_weight, k_weight, eps, rope, interleaved, pos, new_len, slot,
                                    q_out, k_out, v_out, stream)
    B, T, row = shape
    if not qkv.is_contiguous():
        sb, st, one = qkv.stride()
        if one != 1:
            raise ValueError("qkv must be a CUDA tensor [B, T, (Hq + 2 Hkv) head_dim] with a contiguous last dimension")
        if T > 1 and B > 1 and sb != T * st:
            qkv = _new(stream, qkv.contiguous)
        elif T > 1:
            row = st
        elif B > 1:
            row = sb
    f32, f16 = torch.float32, torch.float16
    if q_weight is not None:
        if not _is(q_weight, f32, (d,), dev):
            raise ValueError("norm weights must be contiguous fp32 tensors [head_dim] on qkv's device")
    if k_weight is not None:
        if not _is(k_weight, f32, (d,), dev):
            raise ValueError("norm weights must be contiguous fp32 tensors [head_dim] on qkv's device")
    n_pos = rot = 0
    if rope is not None:
        table = rope.shape
        if len(table) != 2 or rope.dtype is not f32 or rope.get_device() != dev or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous fp32 tensor [n_pos, rot_dim] on qkv's device")
        n_pos, rot = table
    # zeros in new outputs that some token may leave out
    whole = new_len is None and pos is None and slot is None and (rot == 0 or n_pos >= T)
    fresh = torch.empty if whole else torch.zeros
    if pos is not None:
        _i32(pos, B, "pos", dev)
    if new_len is not None:
        _i32(new_len, B, "new_len", dev)
    if slot is not None:
        _i32(slot, B, "slot", dev)
    if q_out is None or k_out is None or v_out is None:
        if q_out is None:
            q_out = _new(stream, fresh, (B, Hq, T, d), dtype=f16, device=qkv.device)
        if k_out is None:
            k_out = _new(stream, fresh, (B, Hkv, T, d), dtype=f16, device=qkv.device)
        if v_out is None:
            if k_out.shape[2:3] != (T,):
                fresh = torch.zeros
            v_out = _new(stream, fresh, tuple(k_out.shape), dtype=f16, device=qkv.device)
    kv_shape = k_out.shape
    cap = kv_shape[2] if len(kv_shape) == 4 else -1
    if (kv_shape != (B, Hkv, cap, d) or not _is(q_out, f16, (B, Hq, T, d), dev) or not _is(k_out, f16, kv_shape, dev)
            or not _is(v_out, f16, kv_shape, dev)):
        raise ValueError("outputs must be contiguous fp16 tensors [B, Hq, T, d], [B, Hkv, cap, d] on qkv's device")
    st = _load().tq_qkv_norm_rope(qkv.data_ptr(), _dtype_code(qkv.dtype), B, T, Hq, Hkv, d, row, _ptr(q_weight),
                                  _ptr(k_weight), eps, _ptr(rope), n_pos, rot, 1 if interleaved else 0, _ptr(pos),
                                  _ptr(new_len), q_out.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), cap, _ptr(slot),
                                  _stream_on(stream, dev))
    if st:
        _check(st, "tq_qkv_norm_rope")
    return q_out, k_out, v_out


# ------------------------------------------------------------------ page pool
class PagePool:
    """The page table of a paged cache and its books: page_table int32
    [n_seqs, pages_per_seq], n_pages int32 [n_seqs] (pages each sequence
    holds), ref int32 [num_pages] (sequences that hold each page), and the
    caches whose pages they name (PackedKV of lead shape [num_pages, Hkv,
    page_size]: every layer's K and V).  A new pool has zeros in n_pages and
    ref (PagePool.new).  The calls follow when one of these arrays is replaced
    by another; none of them must be given another storage in place (set_,
    resize_)."""

    def __init__(self, page_table, n_pages, ref, page_size, caches=()):
        self.page_table, self.n_pages, self.ref, self.page_size = page_table, n_pages, ref, page_size
        self.caches = tuple(caches)
        self._books_of = (None, None, None, 0)
        self.bound()

    def books(self):
        """The C struct of the table and its books, checked and built anew
        where one of them has been replaced."""
        was = self._books_of    # the tensors themselves: none of them is freed while the struct names it
        if (self.page_table is not was[0] or self.n_pages is not was[1] or self.ref is not was[2]
                or self.page_size != was[3]):
            table, n_pages, ref = t = self.page_table, self.n_pages, self.ref
            for x, dim in zip(t, (2, 1, 1)):
                if x.dtype != torch.int32 or x.dim() != dim or not x.is_contiguous() or x.device != table.device:
                    raise ValueError("page_table [n_seqs, pages_per_seq], n_pages [n_seqs] and ref [num_pages] must be "
                                     "contiguous int32 tensors on one device")
            if n_pages.shape[0] != table.shape[0]:
                raise ValueError("n_pages must have an entry for every row of page_table")
            if ref.get_device() < 0:
                raise ValueError("a page pool lies on a CUDA device")
            self.dev = ref.get_device()
            self.struct = tq_page_pool(table.data_ptr(), n_pages.data_ptr(), ref.data_ptr(), table.shape[0],
                                       table.shape[1], ref.shape[0], self.page_size)
            self.ref_struct = ctypes.byref(self.struct)
            self._books_of, self._caches_of = t + (self.page_size,), None
        return self.ref_struct

    def bound(self):
        """books(), and the same for the caches' C views."""
        struct, was = self.books(), self._caches_of
        if was is not None and len(was) == len(self.caches):
            for c, k in zip(self.caches, was):
                if c.codes is not k[0] or c.scales is not k[1] or c.qjl is not k[2] or c.rnorm is not k[3]:
                    break
            else:
                return struct
        self._caches_of = None
        self.heads = self.caches[0].lead_shape[1] if self.caches else 0
        lead = (self.ref.shape[0], self.heads, self.page_size)
        for c in self.caches:
            if c.lead_shape != lead or c.codes.device != self.ref.device:
                raise ValueError("caches must have lead shape [num_pages, Hkv, page_size] on the pool's device")
            c.check_arrays()
        self.views = (tq_kv_view * max(1, len(self.caches)))(*[c.view() for c in self.caches])
        self._caches_of = [(c.codes, c.scales, c.qjl, c.rnorm) for c in self.caches]
        return struct

    @classmethod
    def new(cls, n_seqs, pages_per_seq, num_pages, page_size, caches=(), device="cuda"):
        z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        return cls(z(n_seqs, pages_per_seq), z(n_seqs), z(num_pages), page_size, caches)


def tq_pages_workspace_bytes(n_seqs, num_pages, n):
    nb = ctypes.c_size_t()
    _check(_load().tq_pages_workspace_bytes(n_seqs, num_pages, n, ctypes.byref(nb)), "tq_pages_workspace_bytes")
    return nb.value


def _pool_call(pool, n, workspace, result, stream):
    if workspace is None:
        workspace = _new(stream, torch.empty, tq_pages_workspace_bytes(pool.n_pages.shape[0], pool.ref.shape[0], n),
                         dtype=torch.uint8, device=pool.ref.device)
    else:
        _check_workspace(workspace, pool.dev)
    if result is None:
        result = _new(stream, torch.empty, 4, dtype=torch.int32, device=pool.ref.device)
    else:
        _i32(result, 4, "result", pool.dev)
    return workspace, result


def tq_pages_fork(pool, parent, child, share_len, new_len, workspace=None, result=None, stream=None):
    """Sequences begin (parent -1), fork (share the full pages of the parent's
    first share_len tokens, copy the part-filled one) and grow (parent equal
    to child: pages that tokens from share_len on go to and that others hold
    too are replaced), so that child[i] holds pages for new_len[i] tokens.
    int32 CUDA tensors of one length.  Returns the result tensor {status, pages taken,
    pages copied, 0}: status 0 done, > 0 pages missing, -1 an entry is not
    valid; unless it is 0 nothing has changed."""
    struct, n, dev = pool.bound(), child.numel(), pool.dev
    _i32(parent, n, "parent", dev)
    _i32(child, n, "child", dev)
    _i32(share_len, n, "share_len", dev)
    _i32(new_len, n, "new_len", dev)
    if dev != _current_device():
        with _on(dev):
            return tq_pages_fork(pool, parent, child, share_len, new_len, workspace, result, stream)
    workspace, result = _pool_call(pool, n, workspace, result, stream)
    st = _load().tq_pages_fork(struct, pool.views, len(pool.caches), pool.heads, parent.data_ptr(),
                               child.data_ptr(), share_len.data_ptr(), new_len.data_ptr(), n, result.data_ptr(), workspace.data_ptr(),
                               workspace.nbytes, _stream_on(stream, pool.dev))
    if st:
        _check(st, "tq_pages_fork")
    return result


def tq_pages_free(pool, seqs, keep_len=None, stream=None):
    """The sequences named (int32 CUDA tensor) give up their pages, or those
    behind their first keep_len tokens."""
    struct, n, dev = pool.books(), seqs.numel(), pool.dev
    _i32(seqs, n, "seqs", dev)
    _i32(keep_len, n, "keep_len", dev)
    if dev != _current_device():
        with _on(dev):
            return tq_pages_free(pool, seqs, keep_len, stream)
    st = _load().tq_pages_free(struct, seqs.data_ptr(), _ptr(keep_len), n, _stream_on(stream, pool.dev))
    if st:
        _check(st, "tq_pages_free")


def tq_pages_compact(pool, workspace=None, result=None, stream=None):
    """Moves the pages in use to the front of the pool in all of its caches.
    Returns the result tensor {0, pages in use, pages moved, 0}."""
    struct = pool.bound()
    if pool.dev != _current_device():
        with _on(pool.dev):
            return tq_pages_compact(pool, workspace, result, stream)
    workspace, result = _pool_call(pool, 0, workspace, result, stream)
    st = _load().tq_pages_compact(struct, pool.views, len(pool.caches), pool.heads, result.data_ptr(),
                                  workspace.data_ptr(), workspace.nbytes, _stream_on(stream, pool.dev))
    if st:
        _check(st, "tq_pages_compact")
    return result


def tq_to_blocks(pk, stream=None):
    """GGML-style blocks of a PackedKV without QJL: uint8 [..., d/32,
    2 + 4 bits] (fp16 norm of the rotation block, then the packed codes)."""
    lib = _load()
    L = pk.layout
    n = pk.scales.numel() // pk.scales.shape[-1]
    bb = 2 + 4 * L.bits
    out = _new(stream, torch.empty, tuple(pk.lead_shape) + (L.head_dim // 32, bb), dtype=torch.uint8,
               device=pk.codes.device)
    _check(lib.tq_to_blocks(ctypes.byref(L), _ptr(pk.codes), _ptr(pk.scales), n, _ptr(out), _stream(stream)),
           "tq_to_blocks")
    return out


def tq_decode_attn_blocks(Lk, k_blocks, Lv, v_blocks, q, ctx=None, kv_len=None, softmax_scale=0.0, n_split=0,
                          workspace=None, out=None, stream=None):
    """Decode attention read straight from block-form caches: q [B, Hq, d]
    fp16; k_blocks / v_blocks uint8 [B, Hkv, S_cap, d/32, 2 + 4 bits] (as
    tq_to_blocks gives for a contiguous cache) of layouts Lk / Lv."""
    lib = _load()
    B, Hq, d = q.shape
    for blk, L in ((k_blocks, Lk), (v_blocks, Lv)):
        if blk.dim() != 5 or blk.dtype != torch.uint8 or tuple(blk.shape[3:]) != (L.head_dim // 32, 2 + 4 * L.bits):
            raise ValueError("blocks must be uint8 [B, Hkv, S_cap, head_dim/32, 2 + 4 bits]")
        if not blk.is_contiguous():
            raise ValueError("blocks must be contiguous")
    if tuple(k_blocks.shape[:3]) != tuple(v_blocks.shape[:3]) or k_blocks.shape[0] != B:
        raise ValueError("K and V blocks must share [B, Hkv, S_cap] with q's batch")
    Hkv, S_cap = k_blocks.shape[1], k_blocks.shape[2]
    ctx = S_cap if ctx is None else ctx
    need, ns = tq_decode_workspace_bytes(B, Hq, Hkv, d, ctx, n_split)
    if workspace is None:
        workspace = _new(stream, torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    st = lib.tq_decode_attn_blocks(ctypes.byref(Lk), _ptr(k_blocks), ctypes.byref(Lv), _ptr(v_blocks), _ptr(q), B,
                                   Hq, Hkv, S_cap, _ptr(kv_len), ctx, float(softmax_scale), _ptr(out),
                                   _ptr(workspace), workspace.numel(), n_split, _stream(stream))
    _check(st, "tq_decode_attn_blocks")
    return out


def tq_from_blocks(layout, blocks, stream=None):
    """Inverse of tq_to_blocks: a PackedKV with leading shape blocks.shape[:-2]."""
    lib = _load()
    lead = tuple(blocks.shape[:-2])
    pk = _new(stream, PackedKV, layout, lead, device=blocks.device)
    n = pk.scales.numel() // pk.scales.shape[-1]
    _check(lib.tq_from_blocks(ctypes.byref(layout), _ptr(blocks), n, _ptr(pk.codes), _ptr(pk.scales),
                              _stream(stream)), "tq_from_blocks")
    return pk


def tq_polar_quantize(x, bits, stream=None):
    """Polar-angle quantise x [..., d] (fp16/fp32, CUDA, last dim
    contiguous): returns (codes uint8 [..., d*bits/8], radius fp16 [...])."""
    lib = _load()
    d = x.shape[-1]
    if x.stride(-1) != 1:
        raise ValueError("x must have a contiguous last dimension")
    lead = tuple(x.shape[:-1])
    x2 = _new(stream, x.reshape, -1, d)
    n = x2.shape[0]
    cb = ctypes.c_int64()
    _check(lib.tq_polar_code_bytes(d, bits, ctypes.byref(cb)), "tq_polar_code_bytes")
    codes = _new(stream, torch.empty, lead + (cb.value,), dtype=torch.uint8, device=x.device)
    radius = _new(stream, torch.empty, lead, dtype=torch.float16, device=x.device)
    st = lib.tq_polar_quantize(_ptr(x2), _dtype_code(x.dtype), n, d, x2.stride(0), bits, _ptr(codes), _ptr(radius),
                               _stream(stream))
    _check(st, "tq_polar_quantize")
    return codes, radius


def tq_polar_dequantize(codes, radius, head_dim, bits, out_dtype=torch.float16, out=None, stream=None):
    lib = _load()
    lead = tuple(radius.shape)
    n = radius.numel()
    if out is None:
        out = _new(stream, torch.empty, lead + (head_dim,), dtype=out_dtype, device=codes.device)
    st = lib.tq_polar_dequantize(_ptr(codes), _ptr(radius), n, head_dim, bits, _ptr(out), _dtype_code(out.dtype),
                                 _stream(stream))
    _check(st, "tq_polar_dequantize")
    return out


def tq_prefill_attn(K, V, q, ctx, causal=True, softmax_scale=0.0, workspace=None, out=None, stream=None):
    """q [B, Hq, Tq, d] fp16 at positions ctx-Tq .. ctx-1."""
    lib = _load()
    B, Hq, Tq, d = q.shape
    Hkv, S_cap = _cache_for(K, V, B)
    need = tq_prefill_workspace_bytes(B, Hq, Hkv, d, Tq, ctx)
    if workspace is None:
        workspace = _new(stream, torch.empty, max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = _new(stream, torch.empty_like, q)
    kv, vv = K._view_ref(), V._view_ref()
    st = lib.tq_prefill_attn(kv, vv, _ptr(q), B, Hq, Hkv, Tq, S_cap, ctx,
                             1 if causal else 0, float(softmax_scale), _ptr(out), _ptr(workspace),
                             workspace.numel(), _stream(stream))
    _check(st, "tq_prefill_attn")
    return out


def tq_set_wait_limit_ns(ns):
    """Wait limit (ns) of the library's bounded device-side waits for later
    launches; 0 restores the default (2 s)."""
    _check(_load().tq_set_wait_limit_ns(int(ns)), "tq_set_wait_limit_ns")


def tq_device_status(device=None, clear=False):
    """The library's device status word of `device` (default: the current
    one) after synchronising it: 0 when no launch recorded a failure since
    the last clear, else the first failure (TQ_ERR_TIMEOUT = -6)."""
    if device is None:
        device = torch.cuda.current_device()
    st = ctypes.c_int(0)
    _check(_load().tq_device_status(int(device), 1 if clear else 0, ctypes.byref(st)), "tq_device_status")
    return st.value


def tq_strerror(status):
    return _load().tq_strerror(status).decode()


def tq_version():
    return _load().tq_version()

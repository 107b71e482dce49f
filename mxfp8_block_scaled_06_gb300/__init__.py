"""Python binding of libmx, the low-batch MXFP8 block-scaled projection library.

Argument marshalling only: every step runs in the CUDA kernels behind the C ABI
declared in include/mx.h; PyTorch supplies device memory and the current
stream. There is no fallback: if libmx.so is missing or the device is not a
compute-capability 10.3 GPU, the calls raise. Since the C entry points see only
plain pointers, each wrapper first checks every tensor's element type, size,
layout and residency on the handle's GPU (TypeError / ValueError, nothing
launched). A call runs on `stream` (default: the current one); outputs that it
allocates belong to that stream, and the order with other streams is the caller's.

Names and argument order follow the C entry points: mx_create, mx_scale_bytes,
mx_quantize_rows, mx_gemm, mx_gemm_chain, wo_a_grouped, mx_device_status; for expert
layers with MXFP4 weights mx_quantize_rows_fp4, mx_gemm_fp4, mx_route,
mx_gemm_fp4_grouped, mx_combine; for attention over a cache in MXFP4 (MxCache) mx_rope_table,
mx_rope, mx_cache_write, mx_cache_read, mx_attend.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmx.so")

MX_OK, MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED, MX_ERR_DEVICE, MX_ERR_CUDA, MX_ERR_TIMEOUT = range(6)
MX_FLAG_PDL = 1

EXPORTS = ["mx_create", "mx_destroy", "mx_scale_bytes", "mx_quantize_rows",
           "mx_rmsnorm_quantize_rows", "mx_gemm", "mx_gemm_bf16", "mx_gemm_chain",
           "mx_gemm_chain_norm", "mx_gemm_chain_noalloc", "wo_a_grouped", "wo_a_grouped_unfused",
           "mx_warmup_bytes", "mx_warmup", "mx_plan_gemm", "mx_plan_gemm_fp4", "mx_plan_chain_push",
           "mx_device_status",
           "mx_wait_selftest", "mx_status_string", "mx_quantize_rows_fp4", "mx_gemm_fp4", "mx_gemm_fp4_grouped",
           "mx_route", "mx_combine", "mx_rope_table", "mx_rope", "mx_cache_write", "mx_cache_read",
           "mx_attend_bytes", "mx_attend"]

_vp, _i, _l, _u = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_uint


class MxWeight(ctypes.Structure):
    _fields_ = [("w", _vp), ("w_scales", _vp), ("n", _i), ("k", _i)]


# reduction forms and push receive areas of the plan queries (include/mx.h)
MX_REDUCE_ITEMS, MX_REDUCE_ROWS, MX_REDUCE_PUSH, MX_REDUCE_PUSH_COMPACT, MX_REDUCE_BULK = range(5)
MX_PUSH_NONE, MX_PUSH_COMPACT, MX_PUSH_FULL = range(3)
# element types and router scorings (include/mx.h)
MX_TYPE_BF16, MX_TYPE_F16, MX_TYPE_F32 = range(3)
MX_SCORE_SOFTMAX, MX_SCORE_SIGMOID = range(2)
MX_ROPE_PLAIN, MX_ROPE_LINEAR, MX_ROPE_YARN = range(3)


class MxPlanInfo(ctypes.Structure):
    _fields_ = [("splits", _i), ("stages", _i), ("mtile", _i), ("tmem_cols", _i), ("reduction", _i),
                ("smem", ctypes.c_size_t)]


class MxPlanFp4Info(ctypes.Structure):
    _fields_ = [(f, _i) for f in ("splits", "rows", "mtile", "slices", "scale_tiles", "stages", "min_stages",
                                  "tmem_cols", "reduction")] + [("smem", ctypes.c_size_t)]


class MxCacheInfo(ctypes.Structure):
    _fields_ = ([(f, _vp) for f in ("k", "k_scales", "v", "v_scales")]
                + [(f, _i) for f in ("pages", "page_size", "heads", "d")]
                + [(f, _l) for f in ("k_stride", "k_scales_stride", "v_stride", "v_scales_stride")])


class MxError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmx.so (built by build.build()); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libmx.so is not built ({path}); run mxfp8_block_scaled_06_gb300.build.build()")
    lib = ctypes.CDLL(path)
    lib.mx_create.argtypes = [ctypes.POINTER(_vp), _i]
    lib.mx_destroy.argtypes = [_vp]
    lib.mx_scale_bytes.argtypes = [_i, _i]
    lib.mx_scale_bytes.restype = ctypes.c_size_t
    lib.mx_quantize_rows.argtypes = [_vp, _i, _i, _vp, _l, _vp, _vp, _i, _vp]
    lib.mx_gemm.argtypes = [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _u, _vp]
    lib.mx_rmsnorm_quantize_rows.argtypes = [_vp, _i, _i, _vp, _l, _vp, ctypes.c_float, _vp, _vp,
                                             _vp, _i, _vp]
    lib.mx_gemm_chain_norm.argtypes = [_vp, _i, _vp, _vp, ctypes.POINTER(MxWeight), _i, _vp,
                                       ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.mx_gemm_bf16.argtypes = [_vp, _i, _i, _i, _vp, _l, _vp, _vp, _vp, _u, _vp]
    lib.mx_gemm_chain.argtypes = [_vp, _i, _vp, _vp, ctypes.POINTER(MxWeight), _i, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _vp]
    lib.mx_gemm_chain_noalloc.argtypes = [_vp, _i, _vp, _vp, ctypes.POINTER(MxWeight), _i, _vp, _vp]
    lib.mx_warmup_bytes.argtypes = [ctypes.POINTER(MxWeight), _i, ctypes.POINTER(_i), _i]
    lib.mx_warmup_bytes.restype = ctypes.c_size_t
    lib.mx_plan_gemm.argtypes = [_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(MxPlanInfo)]
    lib.mx_plan_gemm_fp4.argtypes = [_i, _i, _i, _i, _i, _u, _i, ctypes.POINTER(_i), ctypes.POINTER(MxPlanFp4Info)]
    lib.mx_plan_chain_push.argtypes = [_i, ctypes.POINTER(MxWeight), _i, _i, ctypes.c_size_t, ctypes.c_size_t,
                                       ctypes.POINTER(_i)]
    lib.mx_warmup.argtypes = [_vp, ctypes.POINTER(MxWeight), _i, ctypes.POINTER(_i), _i, _vp,
                              ctypes.c_size_t, _vp]
    lib.wo_a_grouped.argtypes = [_vp, _i, _vp, _l, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i,
                                 _vp, _vp, _vp, _vp, _vp, _i, _vp]
    lib.wo_a_grouped_unfused.argtypes = [_vp, _i, _vp, _l, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i,
                                         _i, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.mx_quantize_rows_fp4.argtypes = [_vp, _i, _i, _vp, _l, _i, _vp, _vp, _i, _vp, _vp]
    lib.mx_gemm_fp4.argtypes = [_vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _vp, _u, _vp]
    lib.mx_gemm_fp4_grouped.argtypes = [_vp, _i, _i, _i, _i, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp]
    lib.mx_route.argtypes = [_vp, _i, _i, _i, _vp, _l, _i, _vp, _i, _i, _i, _i, ctypes.c_float, _vp, _vp, _vp,
                             _vp, _vp, _vp]
    lib.mx_combine.argtypes = [_vp, _i, _i, _i, _vp, _i, _l, _vp, _vp, _vp, _vp, _vp]
    d = ctypes.c_double
    cache = ctypes.POINTER(MxCacheInfo)
    lib.mx_rope_table.argtypes = [_vp, _i, _i, d, _i, d, _i, d, d, ctypes.c_float, _vp, _vp]
    lib.mx_rope.argtypes = [_vp, _i, _i, _i, _i, _i, _vp, _l, _l, _i, _vp, _vp, _i, _i, _i, _vp, _l, _l, _vp]
    lib.mx_cache_write.argtypes = [_vp, cache, _i, _vp, _vp, _l, _l, _vp, _l, _l, _i, _vp, _vp, _vp]
    lib.mx_cache_read.argtypes = [_vp, cache, _i, _vp, _i, _vp, _vp, _vp]
    lib.mx_attend_bytes.argtypes = [_vp, _i, _i]
    lib.mx_attend_bytes.restype = ctypes.c_size_t
    lib.mx_attend.argtypes = [_vp, cache, _i, _i, _i, _vp, _l, _l, _i, _vp, _vp, _i, _l, _vp, ctypes.c_float, _i, _i,
                              _vp, _l, _l, _vp, _vp, ctypes.c_size_t, _vp]
    lib.mx_device_status.argtypes = [_vp, ctypes.POINTER(_i)]
    lib.mx_wait_selftest.argtypes = [_vp, _vp]
    lib.mx_status_string.argtypes = [_i]
    lib.mx_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().mx_status_string(code).decode()


def _check(rc: int, what: str) -> None:
    if rc != MX_OK:
        raise MxError(rc, what)


class Handle:
    """An mx_handle* bound to one device."""

    def __init__(self, ptr: int, device: int):
        self.ptr = ptr
        self.device = device

    def close(self) -> None:
        if self.ptr:
            load_library().mx_destroy(self.ptr)
            self.ptr = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mx_create(device: int = 0) -> Handle:
    p = _vp()
    _check(load_library().mx_create(ctypes.byref(p), device), "mx_create")
    return Handle(p.value, device)


def mx_scale_bytes(rows: int, k: int) -> int:
    return int(load_library().mx_scale_bytes(rows, k))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty_on(stream):
    """torch.empty, of tensors that belong to this stream: memory of the current one may still be
    in use there by work that was queued before it was freed."""
    import torch

    def empty(shape, dtype, device):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return empty


def _empty_u8(shape, device, stream):
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    return empty(shape, dtype=torch.uint8, device=device)


# The C entry points take plain pointers and cannot see what they point at, so
# the binding checks each tensor before the call: element type, size (so no
# kernel reads or writes past a tensor's end), layout, and that it lives on the
# handle's GPU. Violations raise TypeError / ValueError and launch nothing.
_CODES = _SCALES = _BF16 = None


def _types():
    """(codes, scales, bf16) element types, resolved once."""
    global _CODES, _SCALES, _BF16
    if _CODES is None:
        import torch
        _CODES = (torch.uint8, torch.float8_e4m3fn)
        _SCALES = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())
        _BF16 = (torch.bfloat16,)
    return _CODES, _SCALES, _BF16


def _codes_types():
    return _types()[0]


def _scale_types():
    return _types()[1]


def _bf16_type():
    return _types()[2]


def _sbytes(rows: int, k: int) -> int:
    """mx_scale_bytes without the library call: ceil128(rows) * ceil4(k / 32), 0 for bad k."""
    if rows < 0 or k <= 0 or k % 32:
        return 0
    return (rows + 127) // 128 * 128 * ((k // 32 + 3) // 4 * 4)


def _resident(h: Handle, host_ok=(), **tensors) -> None:
    """Every given tensor lives on the handle's GPU (checked after all the others,
    so a host tensor is only ever rejected here); those named in host_ok may also
    be pinned host memory, which the kernels address directly (zero-copy)."""
    for name, t in tensors.items():
        if t is None:
            continue
        if name in host_ok and t.device.type == "cpu" and t.is_pinned():
            continue
        if t.get_device() != h.device or not t.is_cuda:
            raise ValueError(f"{name}: on {t.device}, the handle's device is cuda:{h.device}"
                             + (" (or pinned host memory)" if name in host_ok else ""))


def _flat(name: str, t, dtypes, numel: int):
    """A contiguous buffer of one of dtypes holding at least numel elements."""
    if t is None:
        raise ValueError(f"{name}: a tensor is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {numel} needed")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t


def _matrix(name: str, t, dtypes, rows: int, cols: int, row_stride: bool = False):
    """A 2-D tensor of one of dtypes with at least rows rows of exactly cols
    elements; contiguous, or (row_stride) with unit column stride and any row stride."""
    if t is None:
        raise ValueError(f"{name}: a tensor is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    shape = t.shape
    if len(shape) != 2 or shape[0] < rows or shape[1] != cols:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [>= {rows}, {cols}]")
    if row_stride:
        st = t.stride()
        if st[1] != 1 or st[0] < cols:
            raise ValueError(f"{name}: layout {st} not supported")
    elif not t.is_contiguous():
        raise ValueError(f"{name}: layout {t.stride()} not supported")
    return t


def _weight(i, w, s):
    if w is None or w.dim() != 2:
        raise ValueError(f"weight {i}: a 2-D [N, K] tensor is required")
    n, k = w.shape
    _matrix(f"weight {i}", w, _codes_types(), n, k)
    _flat(f"weight {i} scales", s, _scale_types(), _sbytes(n, k))
    return n, k


def mx_quantize_rows(h: Handle, x, q=None, scales=None, swizzled: bool = True, stream=None):
    """bf16 [M, K] (row stride x.stride(0)) -> (E4M3 codes uint8 [M, K], scale bytes).
    x may be on the handle's GPU or in pinned host memory (read directly)."""
    import torch
    if x.dim() != 2:
        raise ValueError("x: a 2-D [M, K] tensor is required")
    m, k = x.shape
    _matrix("x", x, (torch.bfloat16,), m, k, row_stride=True)
    sbytes = _sbytes(m, k) if swizzled else m * (k // 32)
    shape = (sbytes,) if swizzled else (m, k // 32)
    if q is not None:
        _matrix("q", q, _codes_types(), m, k)
    if scales is not None:
        _flat("scales", scales, _scale_types(), sbytes)
    if q is None or scales is None:  # outputs to allocate: x must be usable first
        _resident(h, host_ok=("x",), x=x)
    dev = x.device if x.is_cuda else torch.device("cuda", h.device)  # x may be pinned host memory
    q = _empty_u8((m, k), dev, stream) if q is None else q
    scales = _empty_u8(shape, dev, stream) if scales is None else scales
    _resident(h, host_ok=("x",), x=x, q=q, scales=scales)
    _check(load_library().mx_quantize_rows(h.ptr, m, k, _ptr(x), x.stride(0), _ptr(q),
                                           _ptr(scales), int(swizzled), _stream(stream)),
           "mx_quantize_rows")
    return q, scales


def mx_gemm(h: Handle, a, a_scales, w, w_scales, out=None, m: int | None = None,
            pdl: bool = False, stream=None):
    """out[M, N] bf16 = dequant(a[M, K]) x dequant(w[N, K])^T (M = a's rows unless m is given);
    out may be on the handle's GPU or in pinned host memory (written directly). pdl: the
    weights are read before the kernels still running on the stream have ended, so none
    of these may write them (MX_FLAG_PDL in include/mx.h)."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    n, k = _weight(0, w, w_scales)
    m = a.shape[0] if m is None else m
    _matrix("a", a, _codes_types(), m, k)
    _flat("a_scales", a_scales, _scale_types(), _sbytes(m, k))
    if out is None:
        out = empty((m, n), dtype=torch.bfloat16, device=w.device)
    _matrix("out", out, (torch.bfloat16,), m, n)
    _resident(h, host_ok=("out",), a=a, a_scales=a_scales, w=w, w_scales=w_scales, out=out)
    _check(load_library().mx_gemm(h.ptr, m, n, k, _ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales),
                                  _ptr(out), MX_FLAG_PDL if pdl else 0, _stream(stream)), "mx_gemm")
    return out


def mx_gemm_bf16(h: Handle, x, w, w_scales, out=None, m: int | None = None, pdl: bool = False,
                 stream=None):
    """out[M, N] bf16 = dequant(MXFP8(x[M, K])) x dequant(w[N, K])^T, x bf16 with its
    quantization inside the GEMM kernel (row stride x.stride(0)). pdl as for mx_gemm."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    n, k = _weight(0, w, w_scales)
    m = x.shape[0] if m is None else m
    _matrix("x", x, (torch.bfloat16,), m, k, row_stride=True)
    if out is None:
        out = empty((m, n), dtype=torch.bfloat16, device=w.device)
    _matrix("out", out, (torch.bfloat16,), m, n)
    _resident(h, x=x, w=w, w_scales=w_scales, out=out)
    _check(load_library().mx_gemm_bf16(h.ptr, m, n, k, _ptr(x), x.stride(0), _ptr(w), _ptr(w_scales),
                                       _ptr(out), MX_FLAG_PDL if pdl else 0, _stream(stream)),
           "mx_gemm_bf16")
    return out


def _chain_buffers(a1, a1_scales, weights, g1_cols, a2, a2_scales, a3, a3_scales, out, stream):
    """Checks and allocations shared by the two chain entry points."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    if len(weights) != 3:
        raise ValueError("weights: three (w, w_scales) pairs are required")
    (n1, k1), (n2, _), (n3, _) = (_weight(i, w, s) for i, (w, s) in enumerate(weights))
    m = a1.shape[0]
    dev = a1.device
    _matrix("a1", a1, _codes_types(), m, k1)
    _flat("a1_scales", a1_scales, _scale_types(), _sbytes(m, k1))
    a2 = _empty_u8((m, g1_cols), dev, stream) if a2 is None else _matrix("a2", a2, _codes_types(), m, g1_cols)
    a2_scales = (_empty_u8((_sbytes(m, g1_cols),), dev, stream) if a2_scales is None else
                 _flat("a2_scales", a2_scales, _scale_types(), _sbytes(m, g1_cols)))
    a3 = _empty_u8((m, n2), dev, stream) if a3 is None else _matrix("a3", a3, _codes_types(), m, n2)
    a3_scales = (_empty_u8((_sbytes(m, n2),), dev, stream) if a3_scales is None else
                 _flat("a3_scales", a3_scales, _scale_types(), _sbytes(m, n2)))
    out = empty((m, n3), dtype=torch.bfloat16, device=dev) if out is None else out
    _matrix("out", out, (torch.bfloat16,), m, n3)
    ws = (MxWeight * 3)(*[MxWeight(_ptr(w), _ptr(s), w.shape[0], w.shape[1]) for w, s in weights])
    return m, dev, ws, (n1, n2, n3), a2, a2_scales, a3, a3_scales, out


def _chain_resident(h: Handle, a1, a1_scales, weights, a2, a2_scales, a3, a3_scales, out):
    _resident(h, a1=a1, a1_scales=a1_scales, a2=a2, a2_scales=a2_scales, a3=a3, a3_scales=a3_scales,
              out=out, **{f"weight {i}": w for i, (w, _) in enumerate(weights)},
              **{f"weight {i} scales": s for i, (_, s) in enumerate(weights)})


def mx_gemm_chain(h: Handle, a1, a1_scales, weights, g1_cols: int = 1536, out=None,
                  a2=None, a2_scales=None, a3=None, a3_scales=None, debug: bool = False,
                  stream=None) -> dict:
    """Three projections on one stream with PDL: G1 -> MXFP8 requant of its first
    g1_cols columns -> G2 -> requant -> G3. weights = [(w, w_scales)] * 3."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    m, dev, ws, (n1, n2, n3), a2, a2_scales, a3, a3_scales, out = _chain_buffers(
        a1, a1_scales, weights, g1_cols, a2, a2_scales, a3, a3_scales, out, stream)
    d1 = empty((m, n1), dtype=torch.bfloat16, device=dev) if debug else None
    d2 = empty((m, n2), dtype=torch.bfloat16, device=dev) if debug else None
    _chain_resident(h, a1, a1_scales, weights, a2, a2_scales, a3, a3_scales, out)
    _check(load_library().mx_gemm_chain(h.ptr, m, _ptr(a1), _ptr(a1_scales), ws, g1_cols, _ptr(a2),
                                        _ptr(a2_scales), _ptr(a3), _ptr(a3_scales), _ptr(out),
                                        _ptr(d1), _ptr(d2), _stream(stream)), "mx_gemm_chain")
    return dict(out=out, a2=a2, a2_scales=a2_scales, a3=a3, a3_scales=a3_scales, out1=d1, out2=d2)


def mx_gemm_chain_noalloc(h: Handle, a1, a1_scales, weights, g1_cols: int = 1536, out=None,
                          stream=None):
    """The chain for callers that cannot allocate device memory: only the inputs
    and the output are passed; the library keeps the two intermediates in a fixed
    1 MiB device array (see include/mx.h). Raises MxError (MX_ERR_UNSUPPORTED)
    when the intermediates do not fit; calls that overlap on the GPU race."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    if len(weights) != 3:
        raise ValueError("weights: three (w, w_scales) pairs are required")
    (_, k1), _, (n3, _) = (_weight(i, w, s) for i, (w, s) in enumerate(weights))
    m = a1.shape[0]
    _matrix("a1", a1, _codes_types(), m, k1)
    _flat("a1_scales", a1_scales, _scale_types(), _sbytes(m, k1))
    out = empty((m, n3), dtype=torch.bfloat16, device=a1.device) if out is None else out
    _matrix("out", out, (torch.bfloat16,), m, n3)
    ws = (MxWeight * 3)(*[MxWeight(_ptr(w), _ptr(s), w.shape[0], w.shape[1]) for w, s in weights])
    _resident(h, a1=a1, a1_scales=a1_scales, out=out,
              **{f"weight {i}": w for i, (w, _) in enumerate(weights)},
              **{f"weight {i} scales": s for i, (_, s) in enumerate(weights)})
    _check(load_library().mx_gemm_chain_noalloc(h.ptr, m, _ptr(a1), _ptr(a1_scales), ws, g1_cols,
                                                _ptr(out), _stream(stream)),
           "mx_gemm_chain_noalloc (the intermediates must fit in the library's 1 MiB array)")
    return out


def mx_rmsnorm_quantize_rows(h: Handle, x, norm_weight, eps: float, q=None, scales=None,
                             swizzled: bool = True, y: bool = False, stream=None):
    """bf16 [M, K] (row stride x.stride(0)) -> RMS-normalized with norm_weight [K] bf16 and
    eps, rounded to bf16 (returned as y when asked) and MX-quantized: (q, scales, y)."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    if x.dim() != 2:
        raise ValueError("x: a 2-D [M, K] tensor is required")
    m, k = x.shape
    _matrix("x", x, (torch.bfloat16,), m, k, row_stride=True)
    _flat("norm_weight", norm_weight, (torch.bfloat16,), k)
    sbytes = _sbytes(m, k) if swizzled else m * (k // 32)
    q = _empty_u8((m, k), x.device, stream) if q is None else _matrix("q", q, _codes_types(), m, k)
    shape = (sbytes,) if swizzled else (m, k // 32)
    scales = _empty_u8(shape, x.device, stream) if scales is None else _flat("scales", scales, _scale_types(), sbytes)
    yt = empty((m, k), dtype=torch.bfloat16, device=x.device) if y else None
    _resident(h, x=x, norm_weight=norm_weight, q=q, scales=scales)
    _check(load_library().mx_rmsnorm_quantize_rows(h.ptr, m, k, _ptr(x), x.stride(0),
                                                   _ptr(norm_weight), float(eps), _ptr(yt), _ptr(q),
                                                   _ptr(scales), int(swizzled), _stream(stream)),
           "mx_rmsnorm_quantize_rows")
    return q, scales, yt


def mx_gemm_chain_norm(h: Handle, a1, a1_scales, weights, norm_weight, eps: float,
                       g1_cols: int = 1536, out=None, out1=None, a2=None, a2_scales=None, a3=None,
                       a3_scales=None, debug: bool = False, stream=None) -> dict:
    """mx_gemm_chain with the RMS-norm split between G1 and G2: G1's bf16 output goes
    to out1 (qr | kv), qr is normalized and quantized for G2."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    m, dev, ws, (n1, n2, n3), a2, a2_scales, a3, a3_scales, out = _chain_buffers(
        a1, a1_scales, weights, g1_cols, a2, a2_scales, a3, a3_scales, out, stream)
    _flat("norm_weight", norm_weight, (torch.bfloat16,), g1_cols)
    out1 = empty((m, n1), dtype=torch.bfloat16, device=dev) if out1 is None else out1
    _matrix("out1", out1, (torch.bfloat16,), m, n1)
    dy = empty((m, g1_cols), dtype=torch.bfloat16, device=dev) if debug else None
    d2 = empty((m, n2), dtype=torch.bfloat16, device=dev) if debug else None
    _chain_resident(h, a1, a1_scales, weights, a2, a2_scales, a3, a3_scales, out)
    _resident(h, norm_weight=norm_weight, out1=out1)
    _check(load_library().mx_gemm_chain_norm(h.ptr, m, _ptr(a1), _ptr(a1_scales), ws, g1_cols,
                                             _ptr(norm_weight), float(eps), _ptr(out1), _ptr(a2),
                                             _ptr(a2_scales), _ptr(a3), _ptr(a3_scales), _ptr(out),
                                             _ptr(dy), _ptr(d2), _stream(stream)),
           "mx_gemm_chain_norm")
    return dict(out=out, out1=out1, a2=a2, a2_scales=a2_scales, a3=a3, a3_scales=a3_scales, y=dy,
                out2=d2)


def _wo_a_inputs(x, positions, cos_sin, w, w_scales, n_groups, heads_per_group,
                 o_lora_rank, d_nope, d_rope):
    """Checks shared by the two WO-A entry points; returns (T, K of all groups, columns)."""
    import torch
    t = x.shape[0]
    kall = n_groups * heads_per_group * (d_nope + d_rope)
    cols = n_groups * o_lora_rank
    if x.dtype != torch.bfloat16:
        raise TypeError(f"x: dtype {x.dtype}, expected torch.bfloat16")
    # each token's heads x dims are contiguous; tokens are x.stride(0) elements apart
    if x.dim() < 2 or x.stride(-1) != 1 or not x[0].is_contiguous() or x[0].numel() != kall:
        raise ValueError(f"x: each token must hold {kall} contiguous elements")
    if x.stride(0) < kall:
        raise ValueError(f"x: token stride {x.stride(0)} below {kall}")
    _flat("positions", positions, (torch.int64,), t)
    if cos_sin.dim() != 2 or cos_sin.shape[1] != d_rope:
        raise ValueError(f"cos_sin: shape {tuple(cos_sin.shape)}, expected [max_pos, {d_rope}]")
    _flat("cos_sin", cos_sin, (torch.float32,), 0)
    _matrix("w", w, _codes_types(), cols, heads_per_group * (d_nope + d_rope))
    _flat("w_scales", w_scales, _scale_types(), _sbytes(cols, heads_per_group * (d_nope + d_rope)))
    return t, kall, cols


def _wo_a_resident(h: Handle, x, positions, cos_sin, w, w_scales):
    _resident(h, x=x, positions=positions, cos_sin=cos_sin, w=w, w_scales=w_scales)


def wo_a_grouped(h: Handle, x, positions, cos_sin, w, w_scales, n_groups: int,
                 heads_per_group: int, o_lora_rank: int, d_nope: int = 448, d_rope: int = 64,
                 q=None, q_scales=None, debug: bool = False, early_trigger: bool = False,
                 z: bool = False, stream=None) -> dict:
    """x: bf16 [T, heads, d_nope + d_rope] (token stride x.stride(0)); returns the
    MXFP8 activation (q, q_scales) for wo_b, plus debug tensors if asked: z (bf16
    before requantization) with z or debug, the quantized activation with debug
    (which keeps the call on the fused kernel at every T)."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    t, kall, cols = _wo_a_inputs(x, positions, cos_sin, w, w_scales, n_groups, heads_per_group,
                                 o_lora_rank, d_nope, d_rope)
    dev = x.device
    q = _empty_u8((t, cols), dev, stream) if q is None else _matrix("q", q, _codes_types(), t, cols)
    q_scales = (_empty_u8((_sbytes(t, cols),), dev, stream) if q_scales is None else
                _flat("q_scales", q_scales, _scale_types(), _sbytes(t, cols)))
    dz = empty((t, cols), dtype=torch.bfloat16, device=dev) if debug or z else None
    dxq = _empty_u8((t, kall), dev, stream) if debug else None
    dxs = _empty_u8((t, kall // 32), dev, stream) if debug else None
    _wo_a_resident(h, x, positions, cos_sin, w, w_scales)
    _resident(h, q=q, q_scales=q_scales)
    _check(load_library().wo_a_grouped(h.ptr, t, _ptr(x), x.stride(0), _ptr(positions),
                                       _ptr(cos_sin), cos_sin.shape[0], _ptr(w), _ptr(w_scales),
                                       n_groups, heads_per_group, d_nope, d_rope, o_lora_rank,
                                       _ptr(q), _ptr(q_scales), _ptr(dz), _ptr(dxq), _ptr(dxs),
                                       int(early_trigger), _stream(stream)), "wo_a_grouped")
    return dict(q=q, q_scales=q_scales, z=dz, xq=dxq, xs=dxs)


def wo_a_grouped_unfused(h: Handle, x, positions, cos_sin, w, w_scales, n_groups: int,
                         heads_per_group: int, o_lora_rank: int, d_nope: int = 448,
                         d_rope: int = 64, q=None, q_scales=None, xq=None, xq_scales=None,
                         z: bool = False, stream=None) -> dict:
    """wo_a_grouped in two launches (RoPE + quantize into the caller-owned xq, then a
    grouped GEMM with the requantization fused); for token counts up to 256."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    t, kall, cols = _wo_a_inputs(x, positions, cos_sin, w, w_scales, n_groups, heads_per_group,
                                 o_lora_rank, d_nope, d_rope)
    dev = x.device
    q = _empty_u8((t, cols), dev, stream) if q is None else _matrix("q", q, _codes_types(), t, cols)
    q_scales = (_empty_u8((_sbytes(t, cols),), dev, stream) if q_scales is None else
                _flat("q_scales", q_scales, _scale_types(), _sbytes(t, cols)))
    xq = _empty_u8((t, kall), dev, stream) if xq is None else _matrix("xq", xq, _codes_types(), t, kall)
    xq_scales = (_empty_u8((_sbytes(t, kall),), dev, stream) if xq_scales is None else
                 _flat("xq_scales", xq_scales, _scale_types(), _sbytes(t, kall)))
    zt = empty((t, cols), dtype=torch.bfloat16, device=dev) if z else None
    _wo_a_resident(h, x, positions, cos_sin, w, w_scales)
    _resident(h, q=q, q_scales=q_scales, xq=xq, xq_scales=xq_scales)
    _check(load_library().wo_a_grouped_unfused(h.ptr, t, _ptr(x), x.stride(0), _ptr(positions),
                                               _ptr(cos_sin), cos_sin.shape[0], _ptr(w),
                                               _ptr(w_scales), n_groups, heads_per_group, d_nope,
                                               d_rope, o_lora_rank, _ptr(xq), _ptr(xq_scales),
                                               _ptr(zt), _ptr(q), _ptr(q_scales), _stream(stream)),
           "wo_a_grouped_unfused")
    return dict(q=q, q_scales=q_scales, z=zt, xq=xq, xq_scales=xq_scales)


# The five calls below run in a few microseconds of GPU time for a decode step, so
# their host path is kept short: element types resolved once, residency by device
# number, and the current stream's raw handle (2.8 us through torch.cuda.current_stream).
_TYPE_CODES = _U8 = _I32 = _F32 = _RAW_STREAM = None


def _setup():
    """Resolves what the calls below need of torch, once."""
    global _TYPE_CODES, _U8, _I32, _F32, _RAW_STREAM
    import torch
    _types()
    _U8, _I32, _F32 = (torch.uint8,), (torch.int32,), (torch.float32,)
    _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _TYPE_CODES = {torch.bfloat16: MX_TYPE_BF16, torch.float16: MX_TYPE_F16, torch.float32: MX_TYPE_F32}
    return torch


_torch = None


def _t():
    global _torch
    if _torch is None:
        _torch = _setup()
    return _torch


def _here(h: Handle, *named) -> None:
    """As _resident, of (name, tensor or None) pairs."""
    device = h.device
    for name, t in named:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{name}: on {t.device}, the handle's device is cuda:{device}")


def _stream_of(h: Handle, stream):
    """Raw handle of the given stream, or of the handle's device's current one."""
    if stream is None and _RAW_STREAM is not None:
        return _RAW_STREAM(h.device)
    return _stream(stream)


def _type_code(name: str, t, allowed):
    """MX_TYPE_* of a tensor, which has to be one of allowed."""
    code = _TYPE_CODES.get(t.dtype)
    if code is None or code not in allowed:
        raise TypeError(f"{name}: dtype {t.dtype} not supported")
    return code


def mx_quantize_rows_fp4(h: Handle, x, q=None, scales=None, swizzled: bool = True, y: bool = False,
                         stream=None):
    """bf16, fp16 or fp32 [M, K] (row stride x.stride(0)) -> (packed E2M1 codes uint8
    [M, K/2], scale bytes, y): y = the codes' values in bf16 [M, K] when asked, else None."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if x.dim() != 2:
        raise ValueError("x: a 2-D [M, K] tensor is required")
    m, k = x.shape
    code = _type_code("x", x, (MX_TYPE_BF16, MX_TYPE_F16, MX_TYPE_F32))
    _matrix("x", x, (x.dtype,), m, k, row_stride=True)
    if k % 32:
        raise ValueError(f"x: {k} columns, a multiple of 32 is required")
    sbytes = _sbytes(m, k) if swizzled else m * (k // 32)
    if q is not None:
        _matrix("q", q, _U8, m, k // 2)
    if scales is not None:
        _flat("scales", scales, _scale_types(), sbytes)
    _here(h, ("x", x), ("q", q), ("scales", scales))
    if q is None:
        q = empty((m, k // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = empty((sbytes,) if swizzled else (m, k // 32), dtype=torch.uint8, device=x.device)
    yt = empty((m, k), dtype=torch.bfloat16, device=x.device) if y else None
    _check(load_library().mx_quantize_rows_fp4(h.ptr, m, k, x.data_ptr(), x.stride(0), code, q.data_ptr(),
                                               scales.data_ptr(), int(swizzled), _ptr(yt), _stream_of(h, stream)),
           "mx_quantize_rows_fp4")
    return q, scales, yt


def _fp4_activations(a, m: int, k: int):
    """1 if a holds m rows of packed MXFP4, 0 if of MXFP8: told by its columns."""
    if a is None or a.dim() != 2 or a.shape[1] not in (k, k // 2):
        raise ValueError(f"a: expected [>= {m}, {k}] MXFP8 codes or [>= {m}, {k // 2}] packed MXFP4 codes")
    fp4 = a.shape[1] == k // 2
    _matrix("a", a, _U8 if fp4 else _codes_types(), m, a.shape[1])
    return int(fp4)


def mx_gemm_fp4(h: Handle, a, a_scales, w, w_scales, out=None, m: int | None = None, pdl: bool = False,
                stream=None):
    """out[M, N] bf16 = dequant(a) x dequant(w)^T with MXFP4 weights w: packed codes uint8
    [N, K/2] and swizzled scales. a: MXFP8 codes [M, K] or packed MXFP4 codes [M, K/2],
    with swizzled scales (M = a's rows unless m is given). pdl as for mx_gemm: no kernel
    still running on the stream may write w or w_scales."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if w is None or w.dim() != 2:
        raise ValueError("w: a 2-D [N, K/2] tensor is required")
    n, k = w.shape[0], 2 * w.shape[1]
    _matrix("w", w, _U8, n, k // 2)
    _flat("w_scales", w_scales, _scale_types(), _sbytes(n, k))
    m = a.shape[0] if m is None else m
    fp4 = _fp4_activations(a, m, k)
    _flat("a_scales", a_scales, _scale_types(), _sbytes(m, k))
    if out is not None:
        _matrix("out", out, _BF16, m, n)
    _here(h, ("a", a), ("a_scales", a_scales), ("w", w), ("w_scales", w_scales), ("out", out))
    if out is None:
        out = empty((m, n), dtype=torch.bfloat16, device=w.device)
    _check(load_library().mx_gemm_fp4(h.ptr, m, n, k, a.data_ptr(), a_scales.data_ptr(), fp4, w.data_ptr(),
                                      w_scales.data_ptr(), out.data_ptr(), MX_FLAG_PDL if pdl else 0,
                                      _stream_of(h, stream)), "mx_gemm_fp4")
    return out


def mx_gemm_fp4_grouped(h: Handle, a, a_scales, w, w_scales, offsets, tokens=None, gated: bool = False,
                        out=None, stream=None):
    """The experts' products: out[r] = dequant(a[tokens[r]]) x dequant(w[e])^T for rows
    offsets[e] <= r < offsets[e + 1] (tokens None: row r of a). a: MXFP8 codes [rows, K] or
    packed MXFP4 codes [rows, K/2] with plain [rows, K/32] scales; w: packed codes uint8
    [E, N, K/2], w_scales each expert's swizzled scales; offsets int32 [E + 1], tokens
    int32 [R]. gated: weight rows 2i, 2i + 1 are gate i, up i and out is [R, N/2],
    silu(gate) * up. Rows that no expert has are left as they are."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if w is None or w.dim() != 3:
        raise ValueError("w: a 3-D [E, N, K/2] tensor is required")
    e, n, k = w.shape[0], w.shape[1], 2 * w.shape[2]
    _flat("w", w, _U8, e * n * k // 2)
    if n % 128:
        raise ValueError(f"w: {n} rows per expert, a multiple of 128 is required")
    _flat("w_scales", w_scales, _scale_types(), e * _sbytes(n, k))
    fp4 = _fp4_activations(a, 1, k)
    rows = a.shape[0]
    _flat("a_scales", a_scales, _scale_types(), rows * (k // 32))
    _flat("offsets", offsets, _I32, e + 1)
    if tokens is not None:
        _flat("tokens", tokens, _I32, 1)
    r = rows if tokens is None else tokens.numel()
    cols = n // 2 if gated else n
    if out is not None:
        _matrix("out", out, _BF16, r, cols)
    _here(h, ("a", a), ("a_scales", a_scales), ("w", w), ("w_scales", w_scales), ("offsets", offsets),
          ("tokens", tokens), ("out", out))
    if out is None:
        out = empty((r, cols), dtype=torch.bfloat16, device=w.device)
    _check(load_library().mx_gemm_fp4_grouped(h.ptr, e, r, n, k, a.data_ptr(), rows, a_scales.data_ptr(), fp4,
                                              w.data_ptr(), w_scales.data_ptr(), offsets.data_ptr(), _ptr(tokens),
                                              int(gated), out.data_ptr(), _stream_of(h, stream)),
           "mx_gemm_fp4_grouped")
    return out


def mx_route(h: Handle, logits, top_k: int, bias=None, scoring: str = "softmax", n_groups: int = 1,
             topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, weights=None, experts=None,
             offsets=None, tokens=None, slots=None, stream=None) -> dict:
    """Routes tokens to experts: logits fp32 or bf16 [T, E] (row stride logits.stride(0)),
    bias fp32 [E] for the selection only, scoring "softmax" or "sigmoid". Returns weights
    fp32 and experts int32 [T, top_k], and the rows in expert order: offsets int32 [E + 1],
    tokens int32 [T * top_k] (the token of each row), slots int32 [T, top_k] (the row of
    each choice)."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if logits.dim() != 2:
        raise ValueError("logits: a 2-D [T, E] tensor is required")
    t, e = logits.shape
    code = _type_code("logits", logits, (MX_TYPE_BF16, MX_TYPE_F32))
    _matrix("logits", logits, (logits.dtype,), t, e, row_stride=True)
    if scoring not in ("softmax", "sigmoid"):
        raise ValueError(f"scoring: {scoring!r}, expected 'softmax' or 'sigmoid'")
    top_k = int(top_k)
    if top_k < 1:
        raise ValueError(f"top_k: {top_k}, at least 1 is required")
    if bias is not None:
        _flat("bias", bias, _F32, e)
    if weights is not None:
        _flat("weights", weights, _F32, t * top_k)
    for name, x, count in (("experts", experts, t * top_k), ("offsets", offsets, e + 1),
                           ("tokens", tokens, t * top_k), ("slots", slots, t * top_k)):
        if x is not None:
            _flat(name, x, _I32, count)
    _here(h, ("logits", logits), ("bias", bias), ("weights", weights), ("experts", experts), ("offsets", offsets),
          ("tokens", tokens), ("slots", slots))
    dev, i32 = logits.device, torch.int32
    if weights is None:
        weights = empty((t, top_k), dtype=torch.float32, device=dev)
    if experts is None:
        experts = empty((t, top_k), dtype=i32, device=dev)
    if offsets is None:
        offsets = empty((e + 1,), dtype=i32, device=dev)
    if tokens is None:
        tokens = empty((t * top_k,), dtype=i32, device=dev)
    if slots is None:
        slots = empty((t, top_k), dtype=i32, device=dev)
    _check(load_library().mx_route(h.ptr, t, e, top_k, logits.data_ptr(), logits.stride(0), code, _ptr(bias),
                                   MX_SCORE_SIGMOID if scoring == "sigmoid" else MX_SCORE_SOFTMAX, n_groups,
                                   topk_groups, int(renormalize), scale, weights.data_ptr(), experts.data_ptr(),
                                   offsets.data_ptr(), tokens.data_ptr(), slots.data_ptr(), _stream_of(h, stream)),
           "mx_route")
    return dict(weights=weights, experts=experts, offsets=offsets, tokens=tokens, slots=slots)


def mx_combine(h: Handle, y, slots, weights, residual=None, out=None, stream=None):
    """out[t] = sum over j of weights[t, j] * y[slots[t, j]] (+ residual[t]): y bf16 [R, N]
    (row stride y.stride(0)), slots int32 and weights fp32 [T, top_k], bf16 [T, N] out."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if y.dim() != 2 or slots.dim() != 2:
        raise ValueError("y [R, N] and slots [T, top_k]: 2-D tensors are required")
    r, n = y.shape
    t, k = slots.shape
    _matrix("y", y, _BF16, r, n, row_stride=True)
    _matrix("slots", slots, _I32, t, k)
    _matrix("weights", weights, _F32, t, k)
    if residual is not None:
        _matrix("residual", residual, _BF16, t, n)
    if out is not None:
        _matrix("out", out, _BF16, t, n)
    _here(h, ("y", y), ("slots", slots), ("weights", weights), ("residual", residual), ("out", out))
    if out is None:
        out = empty((t, n), dtype=torch.bfloat16, device=y.device)
    _check(load_library().mx_combine(h.ptr, t, k, n, y.data_ptr(), r, y.stride(0), slots.data_ptr(),
                                     weights.data_ptr(), _ptr(residual), out.data_ptr(), _stream_of(h, stream)),
           "mx_combine")
    return out


class MxCache:
    """A paged cache in MXFP4: k uint8 [pages, heads, page_size, d / 2] packed codes, k_scales uint8
    [pages, heads, page_size, d / 32]; v and v_scales the same, or None where the values are the
    keys. A page is contiguous; pages may be any distance apart (k.stride(0))."""

    def __init__(self, k, k_scales, v=None, v_scales=None):
        _t()
        if (v is None) != (v_scales is None):
            raise ValueError("v, v_scales: both or neither are required")
        if k is None or k.dim() != 4:
            raise ValueError("k: a 4-D [pages, heads, page_size, d / 2] tensor is required")
        pages, heads, page_size, half = k.shape
        d = 2 * half
        if d % 32 or page_size % 16 or not (pages and heads and page_size and d):
            raise ValueError(f"k: shape {tuple(k.shape)}, at least one page and head, a multiple of 16 tokens and of 32 "
                             "dimensions are required")
        for name, t, cols in (("k", k, half), ("k_scales", k_scales, d // 32), ("v", v, half), ("v_scales", v_scales, d // 32)):
            if t is None and name[0] == "v":
                continue
            if t is None:
                raise ValueError(f"{name}: a tensor is required")
            if t.dtype not in (_scale_types() if name.endswith("scales") else _U8):
                raise TypeError(f"{name}: dtype {t.dtype} not supported")
            if tuple(t.shape) != (pages, heads, page_size, cols):
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(pages, heads, page_size, cols)}")
            size = heads * page_size * cols
            if (not t[0].is_contiguous() or t.data_ptr() % 16 or (pages > 1 and (t.stride(0) < size or t.stride(0) % 16))):
                raise ValueError(f"{name}: layout {t.stride()} not supported")
            if t.get_device() != k.get_device():
                raise ValueError(f"{name}: on {t.device}, k is on {k.device}")
        self.k, self.k_scales, self.v, self.v_scales = k, k_scales, v, v_scales
        self.pages, self.page_size, self.heads, self.d = pages, page_size, heads, d
        stride = lambda t: 0 if t is None else t.stride(0) if pages > 1 else t[0].numel()  # noqa: E731
        self.info = MxCacheInfo(_ptr(k), _ptr(k_scales), _ptr(v), _ptr(v_scales), pages, page_size, heads, d,
                                stride(k), stride(k_scales), stride(v), stride(v_scales))

    @staticmethod
    def zeros(h: Handle, pages: int, page_size: int, heads: int, d: int, shared: bool = False):
        """A new cache of zero rows on the handle's GPU."""
        torch = _t()
        t = lambda n: torch.zeros((pages, heads, page_size, n), dtype=torch.uint8,  # noqa: E731
                                  device=torch.device("cuda", h.device))
        return MxCache(t(d // 2), t(d // 32), *(() if shared else (t(d // 2), t(d // 32))))


def _heads(name: str, t, dtypes, tokens: int, heads: int, d: int, step: int):
    """A [tokens, heads, d] tensor whose last stride is 1 and whose other strides are multiples of step."""
    if t is None:
        raise ValueError(f"{name}: a tensor is required")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != 3 or tuple(t.shape) != (tokens, heads, d):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(tokens, heads, d)}")
    st = t.stride()
    # the stride of a dimension of one element says nothing
    if (st[2] != 1 or (tokens > 1 and (st[0] < 0 or st[0] % step)) or (heads > 1 and (st[1] < d or st[1] % step))):
        raise ValueError(f"{name}: layout {st} not supported")
    return (st[0] if tokens > 1 else heads * d), (st[1] if heads > 1 else d)


def _output(name: str, t, tokens: int, heads: int, d: int):
    """Rows of an output lie apart."""
    st = t.stride()
    if tokens > 1 and st[0] < d or (tokens > 1 and heads > 1 and
                                    max(st[0], st[1]) < min(st[0], st[1]) * ((tokens if st[0] <= st[1] else heads) - 1) + d):
        raise ValueError(f"{name}: layout {st} not supported, rows lie over one another")


def mx_rope_table(h: Handle, max_pos: int, d_rope: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  original: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, magnitude: float = 1.0, out=None,
                  stream=None):
    """float32 [max_pos, d_rope]: cosines, then sines, of every position, times magnitude. scaling: "none",
    "linear" (all frequencies / factor) or "yarn" (those that turn seldom over `original` positions)."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    kinds = {"none": MX_ROPE_PLAIN, "linear": MX_ROPE_LINEAR, "yarn": MX_ROPE_YARN}
    if scaling not in kinds:
        raise ValueError(f"scaling: {scaling!r}, expected one of {tuple(kinds)}")
    if max_pos < 1 or d_rope < 2:
        raise ValueError(f"max_pos, d_rope: {max_pos}, {d_rope}, at least 1 and 2 are required")
    if out is not None:
        _matrix("out", out, _F32, max_pos, d_rope)
        _here(h, ("out", out))
    else:
        out = empty((max_pos, d_rope), dtype=torch.float32, device=torch.device("cuda", h.device))
    _check(load_library().mx_rope_table(h.ptr, max_pos, d_rope, base, kinds[scaling], factor, original, beta_fast,
                                        beta_slow, magnitude, out.data_ptr(), _stream_of(h, stream)), "mx_rope_table")
    return out


def mx_rope(h: Handle, x, positions, cos_sin, first: int | None = None, interleaved: bool = True, inverse: bool = False,
            out=None, stream=None):
    """x [T, heads, d] (bf16, fp16 or fp32, any strides of tokens and heads) with dimensions
    first .. first + d_rope - 1 (default: the last) of each head rotated by its token's position, int64 [T]; cos_sin
    [max_pos, d_rope] as from mx_rope_table. interleaved: pairs of neighbours, else of halves. inverse:
    by the negative angle. out may be x, or memory that has nothing in common with it."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if x.dim() != 3:
        raise ValueError("x: a 3-D [T, heads, d] tensor is required")
    t, heads, d = x.shape
    code = _type_code("x", x, (MX_TYPE_BF16, MX_TYPE_F16, MX_TYPE_F32))
    ldx, ldxh = _heads("x", x, (x.dtype,), t, heads, d, 1)
    _flat("positions", positions, (torch.int64,), t)
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin: a 2-D [max_pos, d_rope] tensor is required")
    max_pos, d_rope = cos_sin.shape
    _matrix("cos_sin", cos_sin, _F32, max_pos, d_rope)
    first = d - d_rope if first is None else first
    if d_rope % 2 or first < 0 or first + d_rope > d:
        raise ValueError(f"first: {first}, {d_rope} rotated dimensions do not fit in {d}")
    if out is not None:
        ldo, ldoh = _heads("out", out, (x.dtype,), t, heads, d, 1)
        _output("out", out, t, heads, d)
    _here(h, ("x", x), ("positions", positions), ("cos_sin", cos_sin), ("out", out))
    if out is None:
        out = empty((t, heads, d), dtype=x.dtype, device=x.device)
        ldo, ldoh = heads * d, d
    _check(load_library().mx_rope(h.ptr, t, heads, d, first, d_rope, x.data_ptr(), ldx, ldxh, code, positions.data_ptr(),
                                  cos_sin.data_ptr(), max_pos, int(interleaved), int(inverse), out.data_ptr(), ldo, ldoh,
                                  _stream_of(h, stream)), "mx_rope")
    return out


def mx_cache_write(h: Handle, cache: MxCache, slots, k, v=None, values: bool = False, stream=None):
    """Quantizes k (and v) [T, heads, d], bf16, fp16 or fp32, into the cache's slots, int64 [T]: page * page_size
    + place, different ones; negative: left out. Returns the values they are held as, bf16 [T, heads, d],
    when asked, else None, None."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if k.dim() != 3:
        raise ValueError("k: a 3-D [T, heads, d] tensor is required")
    t = k.shape[0]
    code = _type_code("k", k, (MX_TYPE_BF16, MX_TYPE_F16, MX_TYPE_F32))
    ldk, ldkh = _heads("k", k, (k.dtype,), t, cache.heads, cache.d, 8)
    if (v is None) != (cache.v is None):
        raise ValueError("v: the cache has " + ("no values apart" if cache.v is None else "values, they are required"))
    ldv = ldvh = 0
    if v is not None:
        ldv, ldvh = _heads("v", v, (k.dtype,), t, cache.heads, cache.d, 8)
    _flat("slots", slots, (torch.int64,), t)
    _here(h, ("cache", cache.k), ("k", k), ("v", v), ("slots", slots))
    kv = empty((t, cache.heads, cache.d), dtype=torch.bfloat16, device=k.device) if values else None
    vv = empty((t, cache.heads, cache.d), dtype=torch.bfloat16, device=k.device) if values and v is not None else None
    _check(load_library().mx_cache_write(h.ptr, cache.info, t, slots.data_ptr(), k.data_ptr(), ldk, ldkh, _ptr(v), ldv, ldvh,
                                         code, _ptr(kv), _ptr(vv), _stream_of(h, stream)), "mx_cache_write")
    return kv, vv


def mx_cache_read(h: Handle, cache: MxCache, slots, dtype=None, k=None, v=None, stream=None):
    """The values of the cache's rows at slots, int64 [R]: (k, v) [R, heads, d] of dtype (bf16 unless given;
    fp16, fp32), v None where the cache has no values apart. Rows of negative slots are left as they are."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if slots is None or slots.dim() != 1:
        raise ValueError("slots: a 1-D tensor is required")
    r = slots.shape[0]
    _flat("slots", slots, (torch.int64,), r)
    dtype = dtype or (torch.bfloat16 if k is None else k.dtype)
    if dtype not in _TYPE_CODES:
        raise TypeError(f"dtype: {dtype} not supported")
    if v is not None and cache.v is None:
        raise ValueError("v: the cache has no values apart")
    shape = (r, cache.heads, cache.d)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _flat(name, t, (dtype,), r * cache.heads * cache.d)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    _here(h, ("cache", cache.k), ("slots", slots), ("k", k), ("v", v))
    if k is None:
        k = empty(shape, dtype=dtype, device=slots.device)
    if v is None and cache.v is not None:
        v = empty(shape, dtype=dtype, device=slots.device)
    _check(load_library().mx_cache_read(h.ptr, cache.info, r, slots.data_ptr(), _TYPE_CODES[dtype], k.data_ptr(), _ptr(v),
                                        _stream_of(h, stream)), "mx_cache_read")
    return k, v


def mx_attend_bytes(h: Handle, d: int, shared: bool = False) -> int:
    return int(load_library().mx_attend_bytes(h.ptr, d, int(shared)))


def mx_attend(h: Handle, q, cache: MxCache, table, lengths, q_offsets=None, scale: float | None = None, causal: bool = True,
              window: int = 0, out=None, lse: bool = False, workspace=None, stream=None):
    """Attention of q [T, q_heads, d] (bf16 or fp16, any strides of tokens and heads) over a paged cache: table
    int32 [B, columns] pages of each sequence (row stride table.stride(0)), lengths int32 [B] cached tokens, the
    query tokens among them; q_offsets int32 [B + 1] first query token of each sequence (None: T / B each). scale:
    d^-0.5 unless given. causal: a query token sees tokens up to its own, with window only the last so many.
    Returns out [T, q_heads, d] in q's type; with lse (out, float32 [T, q_heads]). workspace: uint8 of
    mx_attend_bytes, allocated unless given."""
    torch = _t()
    empty = torch.empty if stream is None else _empty_on(stream)
    if q.dim() != 3:
        raise ValueError("q: a 3-D [T, q_heads, d] tensor is required")
    t, heads, d = q.shape
    code = _type_code("q", q, (MX_TYPE_BF16, MX_TYPE_F16))
    ldq, ldqh = _heads("q", q, (q.dtype,), t, heads, cache.d, 8)
    if not -2**31 <= window < 2**31:
        raise ValueError(f"window: {window}, at most 2^31 - 1 tokens are possible")
    if heads % cache.heads:
        raise ValueError(f"q: {heads} heads, a multiple of the cache's {cache.heads} is required")
    if table.dim() != 2 or table.dtype != torch.int32:
        raise (ValueError if table.dtype == torch.int32 else TypeError)("table: a 2-D int32 [B, columns] tensor is required")
    b, cols = table.shape
    _matrix("table", table, _I32, b, cols, row_stride=b > 1)
    _flat("lengths", lengths, _I32, b)
    if q_offsets is not None:
        _flat("q_offsets", q_offsets, _I32, b + 1)
    elif b == 0 or t % b:
        raise ValueError(f"q: {t} query tokens of {b} sequences, q_offsets is required")
    if out is not None:
        ldo, ldoh = _heads("out", out, (q.dtype,), t, heads, d, 8)
        _output("out", out, t, heads, d)
    bytes_ = mx_attend_bytes(h, d, cache.v is None)
    if workspace is not None:
        _flat("workspace", workspace, _U8, bytes_)
    _here(h, ("q", q), ("cache", cache.k), ("table", table), ("lengths", lengths), ("q_offsets", q_offsets), ("out", out),
          ("workspace", workspace))
    if out is None:
        out = empty((t, heads, d), dtype=q.dtype, device=q.device)
        ldo, ldoh = heads * d, d
    if workspace is None:
        workspace = empty((max(bytes_, 16),), dtype=torch.uint8, device=q.device)
    sums = empty((t, heads), dtype=torch.float32, device=q.device) if lse else None
    _check(load_library().mx_attend(h.ptr, cache.info, b, t, heads, q.data_ptr(), ldq, ldqh, code, _ptr(q_offsets),
                                    table.data_ptr(), cols, table.stride(0) if b > 1 else cols, lengths.data_ptr(),
                                    d ** -0.5 if scale is None else scale, int(causal), window, out.data_ptr(), ldo, ldoh,
                                    _ptr(sums), workspace.data_ptr(), bytes_, _stream_of(h, stream)), "mx_attend")
    return (out, sums) if lse else out


def mx_warmup(h: Handle, weights, rows, stream=None) -> list:
    """Ready the GEMM of every distinct weight shape at each row count (plans,
    tensor maps, one launch on a zero MXFP8 activation). weights: (w, w_scales)
    pairs; returns the runs' bf16 outputs ([rows, n], all zero for finite
    weights) in run order: shapes in increasing (n, k), then rows as given."""
    import torch
    empty = torch.empty if stream is None else _empty_on(stream)
    if not weights or not rows:
        raise ValueError("mx_warmup needs at least one weight and one row count")
    ws = (MxWeight * len(weights))(*[MxWeight(_ptr(w), _ptr(s), w.shape[0], w.shape[1])
                                     for w, s in weights])
    rr = (_i * len(rows))(*[int(r) for r in rows])
    lib = load_library()
    nbytes = int(lib.mx_warmup_bytes(ws, len(weights), rr, len(rows)))
    if nbytes == 0:
        raise MxError(MX_ERR_INVALID_ARG, "mx_warmup_bytes")
    dev = weights[0][0].device
    scratch = empty(nbytes + 256, dtype=torch.uint8, device=dev)
    off0 = (-scratch.data_ptr()) % 256
    buf = scratch[off0:off0 + nbytes]
    _check(lib.mx_warmup(h.ptr, ws, len(weights), rr, len(rows), _ptr(buf), nbytes, _stream(stream)),
           "mx_warmup")
    shapes = sorted({(w.shape[0], w.shape[1]) for w, _ in weights})
    r256 = lambda v: (v + 255) // 256 * 256
    off = r256(max(r * k for _, k in shapes for r in rows)) + \
        r256(max(mx_scale_bytes(r, k) for _, k in shapes for r in rows))
    outs = []
    for n, k in shapes:
        for r in rows:
            outs.append(buf[off:off + r * n * 2].view(torch.bfloat16).view(r, n))
            off += r256(r * n * 2)
    return outs


def mx_plan_gemm(m: int, n: int, k: int, sm_count: int = 152, fused: bool = False, norm: bool = False,
                 push: int = MX_PUSH_FULL) -> dict:
    """The launch plan mx_gemm (fused: mx_gemm_bf16; norm: the chain-norm's
    G2) makes for [m, k] x [n, k]^T on a device with sm_count SMs. Host only."""
    info = MxPlanInfo()
    _check(load_library().mx_plan_gemm(m, n, k, sm_count, int(fused), int(norm), push, ctypes.byref(info)),
           "mx_plan_gemm")
    return {f: getattr(info, f) for f, _ in MxPlanInfo._fields_}


def mx_plan_gemm_fp4(m: int, n: int, k: int, experts: int = 0, fp4_activations: bool = False, pdl: bool = False,
                     sm_count: int = 152, clusters=(76, 46, 36, 28, 23, 15, 15)) -> dict:
    """The plan of mx_gemm_fp4 for m rows, or (experts > 0) of mx_gemm_fp4_grouped, on a device
    with sm_count SMs that holds so many clusters of 2..8 CTAs at once. Host only."""
    info = MxPlanFp4Info()
    _check(load_library().mx_plan_gemm_fp4(experts, m, n, k, int(fp4_activations), MX_FLAG_PDL if pdl else 0, sm_count,
                                           (_i * 7)(*clusters), ctypes.byref(info)), "mx_plan_gemm_fp4")
    return {f: getattr(info, f) for f, _ in MxPlanFp4Info._fields_}


def mx_plan_chain_push(m: int, shapes, norm: bool = False, sm_count: int = 152, smem_per_sm: int = 233472,
                       smem_reserved: int = 1024) -> list:
    """The push receive area (MX_PUSH_*) of each projection of mx_gemm_chain
    (norm: mx_gemm_chain_norm) at m rows; shapes = [(n, k)] * 3. Host only."""
    ws = (MxWeight * 3)(*[MxWeight(None, None, n, k) for n, k in shapes])
    modes = (_i * 3)()
    _check(load_library().mx_plan_chain_push(m, ws, int(norm), sm_count, smem_per_sm, smem_reserved, modes),
           "mx_plan_chain_push")
    return list(modes)


def mx_device_status(h: Handle) -> int:
    """MX_OK, or the error a kernel recorded since the last call (synchronizes)."""
    v = _i(0)
    _check(load_library().mx_device_status(h.ptr, ctypes.byref(v)), "mx_device_status")
    return v.value


def mx_wait_selftest(h: Handle, stream=None) -> None:
    """Launch the bounded-wait diagnostic: about one second later the kernel gives
    up on a barrier nothing completes, and the next mx_device_status reports
    MX_ERR_TIMEOUT."""
    _check(load_library().mx_wait_selftest(h.ptr, _stream(stream)), "mx_wait_selftest")

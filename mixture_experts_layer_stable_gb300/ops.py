"""ctypes binding of the operators of include/moe_ops.h in libmoe.so: layer
norm, rows sorted by expert and back, and the experts' product in microscaled
4-bit floating point (MXFP4).

Argument marshalling only, as in binding.py: tensors are torch CUDA tensors
whose sizes, strides and types are passed on; every step runs in the library's
CUDA kernels, on the current stream unless `stream` is given.  The functions
keep the C names.  Each raises MoeError when the library returns a status other
than MOE_OK, or when tensors do not fit together.
"""

import ctypes

import torch

from .binding import MOE_ERR_INVALID_ARG, MoeError, _check, _stream as _given_stream, lib as _base_lib

MOE_DT_F32 = 0
MOE_DT_BF16 = 1
MOE_DT_F16 = 2
MOE_ACT_NONE = 0
MOE_ACT_SWIGLU = 1

_DT = {torch.float32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}

_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_PROTOTYPES = {
    "moe_layernorm_forward": (_i32, _i32, _i64, _i32, _vp, _i64, _vp, _vp, _f32, _vp, _i64, _vp, _vp, _vp),
    "moe_layernorm_workspace_bytes": (_i64, _i32),
    "moe_layernorm_backward": (_i32, _i32, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _i64,
                               _vp, _vp, _vp, _sz, _vp),
    "moe_sort_workspace_bytes": (_i64, _i32),
    "moe_sort_rows": (_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp),
    "moe_permute": (_i32, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp),
    "moe_unpermute": (_i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp),
    "moe_unpermute_backward": (_i32, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp),
    "moe_mxfp4_weight_scale_bytes": (_i64, _i32, _i32),
    "moe_mxfp4_row_scale_bytes": (_i64, _i32, _i32),
    "moe_quantize_mxfp4": (_i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp),
    "moe_dequantize_mxfp4": (_i32, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp),
    "moe_quantize_mxfp4_rows": (_i32, _i64, _i32, _vp, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _vp),
    "moe_dequantize_mxfp4_rows": (_i32, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i64, _vp),
    "moe_mxfp4_product_workspace_bytes": (_i64, _i32, _i32, _i32),
    "moe_mxfp4_product": (_i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i64, _vp, _sz, _vp),
}
EXPORTED = list(_PROTOTYPES)

_lib = None


def lib():
    """libmoe.so with the operators' prototypes (raises if it was not built)."""
    global _lib
    if _lib is None:
        L = _base_lib()
        for name, args in _PROTOTYPES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = _sz if name.endswith("_bytes") else ctypes.c_int
        _lib = L
    return _lib


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, t):
    """`stream`, or the current stream of t's device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return stream if type(stream) is int else _given_stream(stream)


def _need(ok, where):
    if not ok:
        raise MoeError(MOE_ERR_INVALID_ARG, where)


def _dt(t, where):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise MoeError(MOE_ERR_INVALID_ARG, where) from None


def _rows(t, n, d, dtype, where):
    """Row stride of a [n, d] tensor with contiguous rows."""
    ld, one = t.stride()
    if t.dtype != dtype or t.shape != (n, d) or (one != 1 and d != 1):
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return ld if n > 1 else max(d, ld)


def _flat(t, n, dtype, where):
    """Pointer of a contiguous tensor of n elements; None stays None."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return t.data_ptr()


_u8 = torch.uint8


def _bytes(t, n, where):
    if t.dtype != _u8 or t.numel() < n or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return t.data_ptr()


def _tiles(K):
    """Bytes of a run of scale tiles along K."""
    return (K + 127) // 128 * 512


# ---------------------------------------------------------------- layer norm
def moe_layernorm_workspace_bytes(rows, d):
    return int(lib().moe_layernorm_workspace_bytes(rows, d))


def moe_layernorm_forward(x, weight, bias, eps, y, mean=None, rstd=None, stream=None):
    """y = layer norm of the rows of x; mean and rstd ([rows] fp32) for the backward."""
    w = "moe_layernorm_forward"
    n, d = x.shape
    dt, wt = _dt(x, w), weight if weight is not None else bias
    wdtype = x.dtype if wt is None else wt.dtype
    _check((_lib or lib()).moe_layernorm_forward(
        dt, dt if wt is None else _dt(wt, w), n, d, x.data_ptr(), _rows(x, n, d, x.dtype, w),
        _flat(weight, d, wdtype, w), _flat(bias, d, wdtype, w), eps, y.data_ptr(), _rows(y, n, d, x.dtype, w),
        _flat(mean, n, torch.float32, w), _flat(rstd, n, torch.float32, w), _stream(stream, x)), w)


def moe_layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, ws, dadd=None, stream=None):
    """dx (+ dadd), dweight and dbias (each of the two may be None; ws is needed for either)."""
    w = "moe_layernorm_backward"
    n, d = x.shape
    dt = _dt(x, w)
    wt = next((t for t in (weight, dweight, dbias) if t is not None), x)
    _check((_lib or lib()).moe_layernorm_backward(
        dt, _dt(wt, w), n, d, dy.data_ptr(), _rows(dy, n, d, x.dtype, w), x.data_ptr(), _rows(x, n, d, x.dtype, w),
        _flat(weight, d, wt.dtype, w), _flat(mean, n, torch.float32, w), _flat(rstd, n, torch.float32, w),
        None if dadd is None else dadd.data_ptr(), 0 if dadd is None else _rows(dadd, n, d, x.dtype, w),
        dx.data_ptr(), _rows(dx, n, d, x.dtype, w), _flat(dweight, d, wt.dtype, w), _flat(dbias, d, wt.dtype, w),
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes,
        _stream(stream, x)), w)


# ---------------------------------------------------------------- rows by expert
def moe_sort_workspace_bytes(R, E):
    return int(lib().moe_sort_workspace_bytes(R, E))


def moe_sort_rows(ids, counts, offsets, perm, inv, ws, stream=None):
    """counts [E], offsets [E+1], perm and inv [R] of the expert ids [R] (int32)."""
    w = "moe_sort_rows"
    R, E = ids.numel(), counts.numel()
    i32 = torch.int32
    _check((_lib or lib()).moe_sort_rows(_flat(ids, R, i32, w), R, E, _flat(counts, E, i32, w), _flat(offsets, E + 1, i32, w),
                               _flat(perm, R, i32, w), _flat(inv, R, i32, w), ws.data_ptr(),
                               ws.nbytes, _stream(stream, ids)), w)


def moe_permute(x, k, inv, offsets, xp, stream=None):
    """xp[inv[t*k+j]] = x[t]; dropped rows are zeros."""
    w = "moe_permute"
    E, off = _segments(offsets, w)
    T, d = x.shape
    _check((_lib or lib()).moe_permute(_dt(x, w), T, d, k, E, x.data_ptr(), _rows(x, T, d, x.dtype, w),
                             _flat(inv, T * k, torch.int32, w), off,
                             _flat(xp, T * k * d, x.dtype, w), _stream(stream, x)), w)


def moe_unpermute(y, weights, k, inv, offsets, out, base=None, stream=None):
    """out[t] = base[t] + sum_j weights[t*k+j] * y[inv[t*k+j]]; weights None: all 1 (the backward of moe_permute)."""
    w = "moe_unpermute"
    E, off = _segments(offsets, w)
    T, d = out.shape
    _check((_lib or lib()).moe_unpermute(_dt(out, w), T, d, k, E, _flat(y, T * k * d, out.dtype, w),
                               _flat(weights, T * k, torch.float32, w), _flat(inv, T * k, torch.int32, w),
                               off,
                               None if base is None else base.data_ptr(),
                               0 if base is None else _rows(base, T, d, out.dtype, w), out.data_ptr(),
                               _rows(out, T, d, out.dtype, w), _stream(stream, out)), w)


def moe_unpermute_backward(dout, y, weights, k, inv, offsets, dy, dw, stream=None):
    """dy and dw of moe_unpermute (dw, and y with it, may be None)."""
    w = "moe_unpermute_backward"
    E, off = _segments(offsets, w)
    T, d = dout.shape
    _check((_lib or lib()).moe_unpermute_backward(
        _dt(dout, w), T, d, k, E, dout.data_ptr(), _rows(dout, T, d, dout.dtype, w),
        _flat(y, T * k * d, dout.dtype, w), _flat(weights, T * k, torch.float32, w),
        _flat(inv, T * k, torch.int32, w), off,
        _flat(dy, T * k * d, dout.dtype, w), _flat(dw, T * k, torch.float32, w), _stream(stream, dout)), w)


# ---------------------------------------------------------------- MXFP4
def moe_mxfp4_weight_scale_bytes(batch, K, N):
    return int(lib().moe_mxfp4_weight_scale_bytes(batch, K, N))


def moe_mxfp4_row_scale_bytes(rows, K, G=1):
    return int(lib().moe_mxfp4_row_scale_bytes(rows, K, G))


def moe_mxfp4_product_workspace_bytes(rows, N, K, G=1):
    return int(lib().moe_mxfp4_product_workspace_bytes(rows, N, K, G))


def moe_quantize_mxfp4(weights, q, scales, paired=False, stream=None):
    """weights [batch, K, N] -> codes q [batch, N, K/2] and scale tiles."""
    w = "moe_quantize_mxfp4"
    b, K, N = weights.shape
    _check((_lib or lib()).moe_quantize_mxfp4(_dt(weights, w), _flat(weights, b * K * N, weights.dtype, w), b, K, N, int(paired),
                                    _bytes(q, b * N * (K // 2), w),
                                    _bytes(scales, b * ((N + 127) // 128) * _tiles(K), w), _stream(stream, weights)), w)


def moe_dequantize_mxfp4(q, scales, weights, paired=False, stream=None):
    """The values of quantised weights, into weights [batch, K, N]."""
    w = "moe_dequantize_mxfp4"
    b, K, N = weights.shape
    _check((_lib or lib()).moe_dequantize_mxfp4(_dt(weights, w), _bytes(q, b * N * (K // 2), w),
                                      _bytes(scales, b * ((N + 127) // 128) * _tiles(K), w), b, K, N, int(paired),
                                      _flat(weights, b * K * N, weights.dtype, w), _stream(stream, weights)), w)


def _segments(offsets, where):
    """(G, pointer) of the experts' segments; offsets None: one segment."""
    if offsets is None:
        return 1, None
    n = offsets.numel()
    return n - 1, _flat(offsets, n, torch.int32, where)


def moe_quantize_mxfp4_rows(x, q, scales, offsets=None, perm=None, k=1, stream=None):
    """Rows x -> codes q [rows, K/2] and scale tiles, in expert order.  With perm [rows] row p is x[perm[p] // k]."""
    w = "moe_quantize_mxfp4_rows"
    G, off = _segments(offsets, w)
    n, K = x.shape
    rows = n if perm is None else perm.numel()
    _need(perm is None or rows <= n * k, w)
    _check((_lib or lib()).moe_quantize_mxfp4_rows(_dt(x, w), rows, K, x.data_ptr(), _rows(x, n, K, x.dtype, w), G, off,
                                         _flat(perm, rows, torch.int32, w), k, _bytes(q, rows * (K // 2), w),
                                         _bytes(scales, (rows // 128 + G) * _tiles(K), w), _stream(stream, x)), w)


def moe_dequantize_mxfp4_rows(q, scales, y, offsets=None, stream=None):
    """The values of quantised rows, into y [rows, K]."""
    w = "moe_dequantize_mxfp4_rows"
    G, off = _segments(offsets, w)
    rows, K = y.shape
    _check((_lib or lib()).moe_dequantize_mxfp4_rows(_dt(y, w), rows, K, _bytes(q, rows * (K // 2), w),
                                           _bytes(scales, (rows // 128 + G) * _tiles(K), w), G, off,
                                           y.data_ptr(), _rows(y, rows, K, y.dtype, w), _stream(stream, y)), w)


def moe_mxfp4_product(q, scales, offsets, wq, wscales, act, out, ws, stream=None):
    """out[p] = row p times its expert's weights wq [G, N, K/2] (act MOE_ACT_SWIGLU: silu(gate) * up of paired ones)."""
    w = "moe_mxfp4_product"
    G, off = _segments(offsets, w)
    rows, n_out = out.shape
    experts, N, half = wq.shape
    K = 2 * half
    if experts != G or n_out != (N // 2 if act == MOE_ACT_SWIGLU else N):
        raise MoeError(MOE_ERR_INVALID_ARG, w)
    _check((_lib or lib()).moe_mxfp4_product(_dt(out, w), rows, N, K, G, off, _bytes(q, rows * (K // 2), w),
                                   _bytes(scales, (rows // 128 + G) * _tiles(K), w),
                                   _bytes(wq, G * N * (K // 2), w),
                                   _bytes(wscales, G * ((N + 127) // 128) * _tiles(K), w), act, out.data_ptr(),
                                   _rows(out, rows, n_out, out.dtype, w), ws.data_ptr(),
                                   ws.nbytes, _stream(stream, out)), w)

"""ctypes binding of the operators of include/moe_ops.h in libmoe.so: layer
norm, rows sorted by expert and back, the experts' products with their
gradients, SwiGLU and activation checkpoints in 8 bits (MXINT8), and the
experts' product in microscaled 4-bit floating point (MXFP4).

Argument marshalling only, as in binding.py: tensors are torch CUDA tensors
whose sizes, strides and types are passed on; every step runs in the library's
CUDA kernels, on the current stream unless `stream` is given.  The functions
keep the C names.  Each raises MoeError when the library returns a status other
than MOE_OK, or when tensors do not fit together or are not all on the current GPU.
"""

import ctypes

import torch

from .binding import MOE_ERR_INVALID_ARG, MoeError, _stream as _given_stream, lib as _base_lib

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
    "moe_grouped_product_workspace_bytes": (_i64, _i32, _i32, _i32),
    "moe_grouped_product": (_i32, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _vp, _i32, _vp, _i64, _vp, _sz, _vp),
    "moe_grouped_product_dw": (_i32, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _vp, _sz,
                               _vp),
    "moe_mxint8_scale_bytes": (_i64, _i32),
    "moe_quantize_mxint8_rows": (_i32, _i64, _i32, _vp, _i64, _vp, _vp, _vp),
    "moe_dequantize_mxint8_rows": (_i32, _i64, _i32, _vp, _vp, _vp, _i64, _vp),
    "moe_swiglu_forward": (_i32, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp),
    "moe_swiglu_backward": (_i32, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp),
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


_f32t, _i32t, _u8, _i8 = torch.float32, torch.int32, torch.uint8, torch.int8
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                   (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _gpu(t, where):
    """The GPU of t, which has to be the current one: a launch goes there.  (The checks of
    the others compare with it.)"""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return dev


def _handle(stream):
    return stream if type(stream) is int else _given_stream(stream)


def _dt(dtype, where):
    try:
        return _DT[dtype]
    except KeyError:
        raise MoeError(MOE_ERR_INVALID_ARG, where) from None


def _ld(t, n, d, where):
    """Row stride of a tensor of shape [n, d] with contiguous rows."""
    ld, one = t.stride()
    if one != 1 and d != 1:
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return ld if n > 1 else max(d, ld)


def _rows(t, n, d, dtype, dev, where):
    """Row stride of a tensor that has to be [n, d] with contiguous rows."""
    if t.dtype is not dtype or t.shape != (n, d) or t.get_device() != dev:
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return _ld(t, n, d, where)


def _flat(t, n, dtype, dev, where):
    """Pointer of a contiguous tensor of n elements; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return t.data_ptr()


def _bytes(t, n, dev, where):
    if t.dtype is not _u8 or t.numel() < n or t.get_device() != dev or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return t.data_ptr()


def _ws(t, dev, where):
    """Pointer of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    return t.data_ptr()


def _segments(offsets, dev, where):
    """(G, pointer) of the experts' segments; offsets None: one segment."""
    if offsets is None:
        return 1, None
    n = offsets.numel()
    return n - 1, _flat(offsets, n, _i32t, dev, where)


def _tiles(K):
    """Bytes of a run of scale tiles along K."""
    return (K + 127) // 128 * 512


# ---------------------------------------------------------------- layer norm
def moe_layernorm_workspace_bytes(rows, d):
    return int(lib().moe_layernorm_workspace_bytes(rows, d))


def moe_layernorm_forward(x, weight, bias, eps, y, mean=None, rstd=None, stream=None):
    """y = layer norm of the rows of x; mean and rstd ([rows] fp32) for the backward."""
    w = "moe_layernorm_forward"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    n, d = x.shape
    xt, wt = x.dtype, weight if weight is not None else bias
    wt = xt if wt is None else wt.dtype
    rc = (_lib or lib()).moe_layernorm_forward(
        _dt(xt, w), _dt(wt, w), n, d, x.data_ptr(), _ld(x, n, d, w), _flat(weight, d, wt, dev, w),
        _flat(bias, d, wt, dev, w), eps, y.data_ptr(), _rows(y, n, d, xt, dev, w), _flat(mean, n, _f32t, dev, w),
        _flat(rstd, n, _f32t, dev, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_layernorm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, ws, dadd=None, stream=None):
    """dx (+ dadd), dweight and dbias (each of the two may be None; ws is needed for either)."""
    w = "moe_layernorm_backward"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    n, d = x.shape
    xt = x.dtype
    wt = next((t for t in (weight, dweight, dbias) if t is not None), x).dtype
    rc = (_lib or lib()).moe_layernorm_backward(
        _dt(xt, w), _dt(wt, w), n, d, dy.data_ptr(), _rows(dy, n, d, xt, dev, w), x.data_ptr(), _ld(x, n, d, w),
        _flat(weight, d, wt, dev, w), _flat(mean, n, _f32t, dev, w), _flat(rstd, n, _f32t, dev, w),
        None if dadd is None else dadd.data_ptr(), 0 if dadd is None else _rows(dadd, n, d, xt, dev, w),
        dx.data_ptr(), _rows(dx, n, d, xt, dev, w), _flat(dweight, d, wt, dev, w), _flat(dbias, d, wt, dev, w),
        None if ws is None else _ws(ws, dev, w), 0 if ws is None else ws.nbytes, st)
    if rc:
        raise MoeError(rc, w)


# ---------------------------------------------------------------- rows by expert
def moe_sort_workspace_bytes(R, E):
    return int(lib().moe_sort_workspace_bytes(R, E))


def moe_sort_rows(ids, counts, offsets, perm, inv, ws, stream=None):
    """counts [E], offsets [E+1], perm and inv [R] of the expert ids [R] (int32)."""
    w = "moe_sort_rows"
    dev = _gpu(ids, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    R, E = ids.numel(), counts.numel()
    rc = (_lib or lib()).moe_sort_rows(
        _flat(ids, R, _i32t, dev, w), R, E, _flat(counts, E, _i32t, dev, w), _flat(offsets, E + 1, _i32t, dev, w),
        _flat(perm, R, _i32t, dev, w), _flat(inv, R, _i32t, dev, w), _ws(ws, dev, w), ws.nbytes, st)
    if rc:
        raise MoeError(rc, w)


def moe_permute(x, k, inv, offsets, xp, stream=None):
    """xp[inv[t*k+j]] = x[t]; dropped rows are zeros."""
    w = "moe_permute"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    E, off = _segments(offsets, dev, w)
    T, d = x.shape
    rc = (_lib or lib()).moe_permute(
        _dt(x.dtype, w), T, d, k, E, x.data_ptr(), _ld(x, T, d, w), _flat(inv, T * k, _i32t, dev, w), off,
        _flat(xp, T * k * d, x.dtype, dev, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_unpermute(y, weights, k, inv, offsets, out, base=None, stream=None):
    """out[t] = base[t] + sum_j weights[t*k+j] * y[inv[t*k+j]]; weights None: all 1 (the backward of moe_permute)."""
    w = "moe_unpermute"
    dev = _gpu(out, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    E, off = _segments(offsets, dev, w)
    T, d = out.shape
    ot = out.dtype
    rc = (_lib or lib()).moe_unpermute(
        _dt(ot, w), T, d, k, E, _flat(y, T * k * d, ot, dev, w), _flat(weights, T * k, _f32t, dev, w),
        _flat(inv, T * k, _i32t, dev, w), off, None if base is None else base.data_ptr(),
        0 if base is None else _rows(base, T, d, ot, dev, w), out.data_ptr(), _ld(out, T, d, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_unpermute_backward(dout, y, weights, k, inv, offsets, dy, dw, stream=None):
    """dy and dw of moe_unpermute (dw, and y with it, may be None)."""
    w = "moe_unpermute_backward"
    dev = _gpu(dout, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    E, off = _segments(offsets, dev, w)
    T, d = dout.shape
    gt = dout.dtype
    rc = (_lib or lib()).moe_unpermute_backward(
        _dt(gt, w), T, d, k, E, dout.data_ptr(), _ld(dout, T, d, w), _flat(y, T * k * d, gt, dev, w),
        _flat(weights, T * k, _f32t, dev, w), _flat(inv, T * k, _i32t, dev, w), off,
        _flat(dy, T * k * d, gt, dev, w), _flat(dw, T * k, _f32t, dev, w), st)
    if rc:
        raise MoeError(rc, w)


# ---------------------------------------------------------------- products by expert
def moe_grouped_product_workspace_bytes(rows, K, N, G=1):
    """Bytes for the products and gradients of up to `rows` rows."""
    return int(lib().moe_grouped_product_workspace_bytes(rows, K, N, G))


def moe_grouped_product(x, weights, offsets, out, ws, transposed=False, stream=None):
    """out[p] = x[p] times its expert's weights [G, K, N]; transposed: [G, N, K] and their transpose, the gradient of
    x for out = dx and x = dy with the forward's weights."""
    w = "moe_grouped_product"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    G, off = _segments(offsets, dev, w)
    rows, K = x.shape
    n, N = out.shape
    xt, ot = x.dtype, out.dtype
    ldx, x1 = x.stride()
    ldo, o1 = out.stride()
    # (one condition: a call of a few rows waits for its checks)
    if (n != rows or weights.shape != ((G, N, K) if transposed else (G, K, N)) or weights.dtype is not xt or
            not weights.is_contiguous() or weights.get_device() != dev or out.get_device() != dev or
            ws.get_device() != dev or not ws.is_contiguous() or (x1 != 1 and K != 1) or (o1 != 1 and N != 1)):
        raise MoeError(MOE_ERR_INVALID_ARG, w)
    if rows <= 1:
        ldx, ldo = max(ldx, K), max(ldo, N)
    rc = (_lib or lib()).moe_grouped_product(_dt(xt, w), _dt(ot, w), rows, K, N, G, off, x.data_ptr(), ldx,
                                             weights.data_ptr(), 1 if transposed else 0, out.data_ptr(), ldo,
                                             ws.data_ptr(), ws.nbytes, st)
    if rc:
        raise MoeError(rc, w)


def moe_grouped_product_dw(x, dy, offsets, dweights, ws, accumulate=False, stream=None):
    """dweights[g] = x^T dy over expert g's rows (accumulate: added to what is there)."""
    w = "moe_grouped_product_dw"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    G, off = _segments(offsets, dev, w)
    rows, K = x.shape
    n, N = dy.shape
    xt = x.dtype
    ldx, x1 = x.stride()
    lddy, y1 = dy.stride()
    if (n != rows or dweights.shape != (G, K, N) or dy.dtype is not xt or not dweights.is_contiguous() or
            dweights.get_device() != dev or dy.get_device() != dev or ws.get_device() != dev or not ws.is_contiguous() or
            (x1 != 1 and K != 1) or (y1 != 1 and N != 1)):
        raise MoeError(MOE_ERR_INVALID_ARG, w)
    if rows <= 1:
        ldx, lddy = max(ldx, K), max(lddy, N)
    rc = (_lib or lib()).moe_grouped_product_dw(_dt(xt, w), _dt(dweights.dtype, w), rows, K, N, G, off, x.data_ptr(), ldx,
                                                dy.data_ptr(), lddy, dweights.data_ptr(), 1 if accumulate else 0,
                                                ws.data_ptr(), ws.nbytes, st)
    if rc:
        raise MoeError(rc, w)


# ---------------------------------------------------------------- MXINT8 and SwiGLU
def moe_mxint8_scale_bytes(rows, n):
    return int(lib().moe_mxint8_scale_bytes(rows, n))


def _kept(q, scales, rows, n, dev, where):
    """Pointers of a checkpoint: codes of rows * n elements and their scales; None stay None."""
    if (q is None) != (scales is None):
        raise MoeError(MOE_ERR_INVALID_ARG, where)
    if q is None:
        return None, None
    return _flat(q, rows * n, _i8, dev, where), _bytes(scales, rows * ((n + 31) // 32), dev, where)


def moe_quantize_mxint8_rows(x, q, scales, stream=None):
    """Rows x [rows, n] -> codes q [rows, n] (int8) and scale bytes [rows, ceil(n / 32)]."""
    w = "moe_quantize_mxint8_rows"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    rows, n = x.shape
    qp, sp = _kept(q, scales, rows, n, dev, w)
    rc = (_lib or lib()).moe_quantize_mxint8_rows(
        _dt(x.dtype, w), rows, n, x.data_ptr(), _ld(x, rows, n, w), qp, sp, st)
    if rc:
        raise MoeError(rc, w)


def moe_dequantize_mxint8_rows(q, scales, y, stream=None):
    """The values of rows in 8 bits, into y [rows, n]."""
    w = "moe_dequantize_mxint8_rows"
    dev = _gpu(y, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    rows, n = y.shape
    qp, sp = _kept(q, scales, rows, n, dev, w)
    rc = (_lib or lib()).moe_dequantize_mxint8_rows(
        _dt(y.dtype, w), rows, n, qp, sp, y.data_ptr(), _ld(y, rows, n, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_swiglu_forward(h, a, q=None, scales=None, stream=None):
    """a = silu(g) * u of the rows h = [g | u]; q [rows, 2f] and scales: h in 8 bits, kept for the backward."""
    w = "moe_swiglu_forward"
    dev = _gpu(a, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    rows, f = a.shape
    at = a.dtype
    qp, sp = _kept(q, scales, 2 * rows, f, dev, w)
    rc = (_lib or lib()).moe_swiglu_forward(
        _dt(at, w), rows, f, h.data_ptr(), _rows(h, rows, 2 * f, at, dev, w), a.data_ptr(), _ld(a, rows, f, w), qp, sp,
        st)
    if rc:
        raise MoeError(rc, w)


def moe_swiglu_backward(da, h, dh, a=None, q=None, scales=None, stream=None):
    """dh [rows, 2f], and a again, from h or (h None) its checkpoint q, scales."""
    w = "moe_swiglu_backward"
    dev = _gpu(da, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    rows, f = da.shape
    at = da.dtype
    qp, sp = _kept(q, scales, 2 * rows, f, dev, w)
    rc = (_lib or lib()).moe_swiglu_backward(
        _dt(at, w), rows, f, da.data_ptr(), _ld(da, rows, f, w), None if h is None else h.data_ptr(),
        0 if h is None else _rows(h, rows, 2 * f, at, dev, w), qp, sp, dh.data_ptr(),
        _rows(dh, rows, 2 * f, at, dev, w), None if a is None else a.data_ptr(),
        0 if a is None else _rows(a, rows, f, at, dev, w), st)
    if rc:
        raise MoeError(rc, w)


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
    dev = _gpu(weights, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    b, K, N = weights.shape
    rc = (_lib or lib()).moe_quantize_mxfp4(
        _dt(weights.dtype, w), _flat(weights, b * K * N, weights.dtype, dev, w), b, K, N, int(paired),
        _bytes(q, b * N * (K // 2), dev, w), _bytes(scales, b * ((N + 127) // 128) * _tiles(K), dev, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_dequantize_mxfp4(q, scales, weights, paired=False, stream=None):
    """The values of quantised weights, into weights [batch, K, N]."""
    w = "moe_dequantize_mxfp4"
    dev = _gpu(weights, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    b, K, N = weights.shape
    rc = (_lib or lib()).moe_dequantize_mxfp4(
        _dt(weights.dtype, w), _bytes(q, b * N * (K // 2), dev, w),
        _bytes(scales, b * ((N + 127) // 128) * _tiles(K), dev, w), b, K, N, int(paired),
        _flat(weights, b * K * N, weights.dtype, dev, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_quantize_mxfp4_rows(x, q, scales, offsets=None, perm=None, k=1, stream=None):
    """Rows x -> codes q [rows, K/2] and scale tiles, in expert order.  With perm [rows] row p is x[perm[p] // k]."""
    w = "moe_quantize_mxfp4_rows"
    dev = _gpu(x, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    G, off = _segments(offsets, dev, w)
    n, K = x.shape
    rows = n if perm is None else perm.numel()
    if perm is not None and rows > n * k:
        raise MoeError(MOE_ERR_INVALID_ARG, w)
    rc = (_lib or lib()).moe_quantize_mxfp4_rows(
        _dt(x.dtype, w), rows, K, x.data_ptr(), _ld(x, n, K, w), G, off, _flat(perm, rows, _i32t, dev, w), k,
        _bytes(q, rows * (K // 2), dev, w), _bytes(scales, (rows // 128 + G) * _tiles(K), dev, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_dequantize_mxfp4_rows(q, scales, y, offsets=None, stream=None):
    """The values of quantised rows, into y [rows, K]."""
    w = "moe_dequantize_mxfp4_rows"
    dev = _gpu(y, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    G, off = _segments(offsets, dev, w)
    rows, K = y.shape
    rc = (_lib or lib()).moe_dequantize_mxfp4_rows(
        _dt(y.dtype, w), rows, K, _bytes(q, rows * (K // 2), dev, w),
        _bytes(scales, (rows // 128 + G) * _tiles(K), dev, w), G, off, y.data_ptr(), _ld(y, rows, K, w), st)
    if rc:
        raise MoeError(rc, w)


def moe_mxfp4_product(q, scales, offsets, wq, wscales, act, out, ws, stream=None):
    """out[p] = row p times its expert's weights wq [G, N, K/2] (act MOE_ACT_SWIGLU: silu(gate) * up of paired ones)."""
    w = "moe_mxfp4_product"
    dev = _gpu(out, w)
    st = _current_stream(dev) if stream is None else _handle(stream)
    G, off = _segments(offsets, dev, w)
    rows, n_out = out.shape
    experts, N, half = wq.shape
    K = 2 * half
    if experts != G or n_out != (N // 2 if act == MOE_ACT_SWIGLU else N):
        raise MoeError(MOE_ERR_INVALID_ARG, w)
    tiles = _tiles(K)
    rc = (_lib or lib()).moe_mxfp4_product(
        _dt(out.dtype, w), rows, N, K, G, off, _bytes(q, rows * half, dev, w),
        _bytes(scales, (rows // 128 + G) * tiles, dev, w), _bytes(wq, G * N * half, dev, w),
        _bytes(wscales, G * ((N + 127) // 128) * tiles, dev, w), act, out.data_ptr(), _ld(out, rows, n_out, w),
        _ws(ws, dev, w), ws.nbytes, st)
    if rc:
        raise MoeError(rc, w)

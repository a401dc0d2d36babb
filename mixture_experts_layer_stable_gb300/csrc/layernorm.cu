// layernorm.cu -- layer norm of token rows, forward and backward
// (include/moe_ops.h, moe_layernorm_*).
//
//   y  = (x - mean) * rstd * w + b
//   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dadd,  g = dy * w, xh = (x - mean) * rstd
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
#include "ops_common.cuh"

namespace moe {

namespace {

constexpr int kLnThreads = 256;
constexpr int kLnRows = 256;  // rows of one partial sum of dw and db

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_sum(v);
  __syncthreads();
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < nw; ++i) s += sh[i];
  return s;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_forward_kernel(
    const T* __restrict__ x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, float eps,
    T* __restrict__ y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int d) {
  __shared__ float sh[kLnThreads / 32];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* xr = x + r * ldx;
    float s = 0.f;
    for (int i = threadIdx.x; i < d; i += blockDim.x) s += to_f32(xr[i]);
    const float mu = block_sum(s, sh) / d;
    s = 0.f;
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float c = to_f32(xr[i]) - mu;
      s += c * c;
    }
    const float rs = 1.0f / sqrtf(block_sum(s, sh) / d + eps);
    if (threadIdx.x == 0 && mean != nullptr) {
      mean[r] = mu;
      rstd[r] = rs;
    }
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float xh = (to_f32(xr[i]) - mu) * rs;
      y[r * ldy + i] = from_f32<T>(xh * (w ? to_f32(w[i]) : 1.f) + (b ? to_f32(b[i]) : 0.f));
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLnThreads) ln_backward_kernel(
    const T* dy, int64_t lddy, const T* x, int64_t ldx, const W* w, const float* mean, const float* rstd,
    const T* dadd, int64_t ldadd, T* dx, int64_t lddx, int64_t rows, int d) {
  __shared__ float sh[kLnThreads / 32];
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float g = to_f32(dy[r * lddy + i]) * (w ? to_f32(w[i]) : 1.f);
      s1 += g;
      s2 += g * ((to_f32(x[r * ldx + i]) - mu) * rs);
    }
    const float m1 = block_sum(s1, sh) / d;
    const float m2 = block_sum(s2, sh) / d;
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float g = to_f32(dy[r * lddy + i]) * (w ? to_f32(w[i]) : 1.f);
      const float xh = (to_f32(x[r * ldx + i]) - mu) * rs;
      float v = rs * (g - m1 - xh * m2);
      if (dadd) v += to_f32(dadd[r * ldadd + i]);
      dx[r * lddx + i] = from_f32<T>(v);
    }
  }
}

// part[c][0 / 1][i]: dw and db summed over rows [c kLnRows, (c + 1) kLnRows).
template <typename T>
__global__ void __launch_bounds__(kLnThreads) ln_partial_kernel(
    const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
    const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ part, int64_t rows,
    int d) {
  const int i = blockIdx.x * kLnThreads + threadIdx.x;
  const int64_t r0 = (int64_t)blockIdx.y * kLnRows, r1 = min(rows, r0 + kLnRows);
  if (i >= d) return;
  float a = 0.f, s = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float g = to_f32(dy[r * lddy + i]);
    a += g * ((to_f32(x[r * ldx + i]) - mean[r]) * rstd[r]);
    s += g;
  }
  part[(size_t)blockIdx.y * 2 * d + i] = a;
  part[(size_t)blockIdx.y * 2 * d + d + i] = s;
}

template <typename W>
__global__ void __launch_bounds__(kLnThreads) ln_reduce_kernel(const float* __restrict__ part, int np,
                                                               W* __restrict__ dw, W* __restrict__ db, int d) {
  const int i = blockIdx.x * kLnThreads + threadIdx.x;
  if (i >= d) return;
  float a = 0.f, s = 0.f;
  for (int p = 0; p < np; ++p) {
    a += part[(size_t)p * 2 * d + i];
    s += part[(size_t)p * 2 * d + d + i];
  }
  if (dw) dw[i] = from_f32<W>(a);
  if (db) db[i] = from_f32<W>(s);
}

bool ln_args(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d) {
  return dtype_valid(dtype) && (wdtype == dtype || wdtype == MOE_DT_F32) && rows >= 0 &&
         rows <= ((int64_t)1 << 40) && d >= 1 && d <= 65536;
}

int64_t ln_parts(int64_t rows) { return (rows + kLnRows - 1) / kLnRows; }

// f(T{}, W{}) for the element types of the rows and of the weights.
template <typename F>
cudaError_t ln_types(int dtype, int wdtype, F f) {
  return with_dtype(dtype, [&](auto t) {
    if (wdtype == MOE_DT_F32) return f(t, float());
    return f(t, t);
  });
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layernorm_forward(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d, const void* x,
                                 int64_t ldx, const void* weight, const void* bias, float eps, void* y,
                                 int64_t ldy, float* mean, float* rstd, moe_stream_t stream) {
  if (!ln_args(dtype, wdtype, rows, d) || ldx < d || ldy < d || !(eps >= 0.f) || !isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype), ws = dtype_bytes(wdtype);
  if (!elem_ok_or_null(weight, ws) || !elem_ok_or_null(bias, ws) || (mean == nullptr) != (rstd == nullptr) ||
      !elem_ok_or_null(mean, 4) || !elem_ok_or_null(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!elem_ok(x, es) || !elem_ok(y, es)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(ln_types(dtype, wdtype, [&](auto t, auto wt) {
    using T = decltype(t);
    using W = decltype(wt);
    const int grid = (int)(rows < 65535 ? rows : 65535);
    TraceScope ts("layernorm_forward", st);
    ln_forward_kernel<T, W><<<grid, kLnThreads, 0, st>>>(
        static_cast<const T*>(x), ldx, static_cast<const W*>(weight), static_cast<const W*>(bias), eps,
        static_cast<T*>(y), ldy, mean, rstd, rows, d);
    return cudaGetLastError();
  }));
}

size_t moe_layernorm_workspace_bytes(int64_t rows, int32_t d) {
  if (!ln_args(MOE_DT_F32, MOE_DT_F32, rows, d)) return 0;
  return ((size_t)(ln_parts(rows) + 1) * 2 * d * sizeof(float) + 127) / 128 * 128;
}

moe_status moe_layernorm_backward(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d, const void* dy,
                                  int64_t lddy, const void* x, int64_t ldx, const void* weight,
                                  const float* mean, const float* rstd, const void* dadd, int64_t ldadd,
                                  void* dx, int64_t lddx, void* dweight, void* dbias, void* ws,
                                  size_t ws_bytes, moe_stream_t stream) {
  if (!ln_args(dtype, wdtype, rows, d) || lddy < d || ldx < d || lddx < d || (dadd != nullptr && ldadd < d))
    return MOE_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype), wb = dtype_bytes(wdtype);
  if (!elem_ok_or_null(weight, wb) || !elem_ok_or_null(dadd, es) || !elem_ok_or_null(dweight, wb) ||
      !elem_ok_or_null(dbias, wb))
    return MOE_ERR_INVALID_ARG;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (sums && (ws == nullptr || !aligned_to(ws, 128))) return MOE_ERR_INVALID_ARG;
  if (sums && ws_bytes < moe_layernorm_workspace_bytes(rows, d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (rows > 0 && (!elem_ok(dy, es) || !elem_ok(x, es) || !elem_ok(dx, es) || !elem_ok(mean, 4) || !elem_ok(rstd, 4)))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0 && !sums) return MOE_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(ln_types(dtype, wdtype, [&](auto t, auto wt) {
    using T = decltype(t);
    using W = decltype(wt);
    float* part = static_cast<float*>(ws);
    const int np = (int)ln_parts(rows), nc = (d + kLnThreads - 1) / kLnThreads;
    cudaError_t e = cudaSuccess;
    if (sums && rows > 0) {
      TraceScope ts("layernorm_partial", st);
      for (int p = 0; p < np && e == cudaSuccess; p += 65535) {
        const int n = np - p < 65535 ? np - p : 65535;
        ln_partial_kernel<T><<<dim3(nc, n), kLnThreads, 0, st>>>(
            static_cast<const T*>(dy) + (size_t)p * kLnRows * lddy, lddy,
            static_cast<const T*>(x) + (size_t)p * kLnRows * ldx, ldx, mean + (size_t)p * kLnRows,
            rstd + (size_t)p * kLnRows, part + (size_t)p * 2 * d, rows - (int64_t)p * kLnRows, d);
        e = cudaGetLastError();
      }
    }
    if (e == cudaSuccess && sums) {
      TraceScope ts("layernorm_reduce", st);
      ln_reduce_kernel<W><<<nc, kLnThreads, 0, st>>>(part, np, static_cast<W*>(dweight), static_cast<W*>(dbias), d);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess && rows > 0) {
      TraceScope ts("layernorm_backward", st);
      ln_backward_kernel<T, W><<<(int)(rows < 65535 ? rows : 65535), kLnThreads, 0, st>>>(
          static_cast<const T*>(dy), lddy, static_cast<const T*>(x), ldx, static_cast<const W*>(weight), mean,
          rstd, static_cast<const T*>(dadd), ldadd, static_cast<T*>(dx), lddx, rows, d);
      e = cudaGetLastError();
    }
    return e;
  }));
}

}  // extern "C"

// mxfp4.cu -- microscaled 4-bit floating point (include/moe_ops.h): the
// quantisers, their inverses and the experts' product.
//
// Block format: 32 elements along K share a UE8M0 scale 2^s, elements E2M1.
// s is the smallest exponent with max |v| <= 6 * 2^s, so no element saturates:
// with max |v| = m * 2^q, m in [0.5, 1), 6 * 2^s = 0.75 * 2^(s+3) gives
// s = q - 3 for m <= 0.75 and q - 2 otherwise.
#include <cuda_fp4.h>

#include "gemm_common.cuh"
#include "mx.cuh"
#include "ops_common.cuh"

namespace moe {

namespace {

constexpr int kTok = MOE_FP4_TOKENS;

// Scale exponent of a block with max |v| = amax (finite).
__device__ __forceinline__ int fp4_scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int eb = (int)(b >> 23) & 0xFF;
  if (eb == 0) return -127;  // zero or below 2^-126
  const int s = (eb - 126) - ((b & 0x7FFFFFu) <= 0x400000u ? 3 : 2);
  return max(-127, s);       // at most 126: the largest finite value is below 6 * 2^126
}
// 2^-s for s in [-127, 126], exact.
__device__ __forceinline__ float fp4_inv_scale(int s) { return __uint_as_float((uint32_t)(127 - s) << 23); }
// 2^s of a scale byte; 255 is NaN.
__device__ __forceinline__ float fp4_scale_of(uint32_t byte) {
  return byte == 255 ? __uint_as_float(0x7FFFFFFFu) : byte == 0 ? __uint_as_float(0x400000u)
                                                               : __uint_as_float(byte << 23);
}
// Two values as a byte of codes (lower index in the low bits), to nearest, ties to even.
__device__ __forceinline__ uint32_t fp4_pack2(float lo, float hi) {
  return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
// Value of a 4-bit code: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.
__device__ __forceinline__ float fp4_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float v = m < 2 ? 0.5f * m : (m & 1u ? 1.5f : 1.0f) * (float)(1u << ((m >> 1) - 1));
  return (c & 8u) ? -v : v;
}

// Offset of the scale of row i of expert g (whose rows start at off), block kb.
__host__ __device__ inline size_t fp4_row_scale_at(int64_t off, int g, int64_t i, int kb, int KT) {
  const int64_t blk = off / kTok + g + i / kTok;
  const int r = (int)(i % kTok);
  return ((size_t)(blk * 2 + (r >> 7)) * KT + (kb >> 2)) * 512u + 16 * (r & 31) + 4 * ((r & 127) >> 5) + (kb & 3);
}
__host__ __device__ inline size_t fp4_weight_scale_at(int64_t e, int n, int kb, int N, int KT) {
  return ((size_t)(e * ((N + 127) / 128) + (n >> 7)) * KT + (kb >> 2)) * 512u + 16 * (n & 31) +
         4 * ((n & 127) >> 5) + (kb & 3);
}

// Largest g in [0, G) with off[g] / div + g <= key (off NULL: 0).
__device__ __forceinline__ int find_group_block(const int* off, int G, int key, int div) {
  if (off == nullptr) return 0;
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(off + mid) / div + mid <= key) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// Expert of row p < off[G]: the largest g with off[g] <= p.
__device__ __forceinline__ int find_group(const int* off, int G, int p) {
  return off == nullptr ? 0 : find_expert(off, G, p);
}

// One block of 32 values: 16 bytes of codes and the scale byte.
__device__ __forceinline__ uint32_t fp4_quant_block(const float* v, uint8_t* q) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  if (m >= 0x7F800000u) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = 0;
    return 255u;
  }
  const int s = fp4_scale_exp(__uint_as_float(m));
  const float f = fp4_inv_scale(s);
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = (uint8_t)fp4_pack2(v[2 * i] * f, v[2 * i + 1] * f);
  return (uint32_t)(s + 127);
}

// One thread per block of a row, the padding blocks (scale 1) included.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows, int K,
                                                         int G, const int* __restrict__ off,
                                                         const int* __restrict__ perm, int k,
                                                         uint8_t* __restrict__ q, uint8_t* __restrict__ sc) {
  const int KT = (K + 127) / 128, nb = KT * 4;
  const int64_t n = (off ? off[G] : rows) * (int64_t)nb;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t p = i / nb;
    const int kb = (int)(i % nb);
    const int g = find_group(off, G, (int)p);
    const int64_t o = off ? off[g] : 0;
    uint32_t s = 127;
    if (kb * 32 < K) {
      const T* src = x + (perm ? (int64_t)(perm[p] / k) : p) * ldx + kb * 32;
      float v[32];
      for (int j = 0; j < 32; ++j) v[j] = to_f32(src[j]);
      s = fp4_quant_block(v, q + p * (K / 2) + kb * 16);
    }
    sc[fp4_row_scale_at(o, g, p - o, kb, KT)] = (uint8_t)s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dequant_rows_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ sc, int64_t rows, int K,
                                                           int G, const int* __restrict__ off, T* __restrict__ y,
                                                           int64_t ldy) {
  const int KT = (K + 127) / 128, h = K / 2;
  const int64_t n = (off ? off[G] : rows) * (int64_t)h;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t p = i / h;
    const int c = (int)(i % h);
    const int g = find_group(off, G, (int)p);
    const int64_t o = off ? off[g] : 0;
    const float s = fp4_scale_of(sc[fp4_row_scale_at(o, g, p - o, c / 16, KT)]);
    const uint32_t b = q[i];
    y[p * ldy + 2 * c] = from_f32<T>(fp4_value(b & 15u) * s);
    y[p * ldy + 2 * c + 1] = from_f32<T>(fp4_value(b >> 4) * s);
  }
}

// Column of w that row n of the codes holds.
__device__ __forceinline__ int fp4_column(int n, int N, bool paired) {
  return paired ? (n & 1) * (N / 2) + (n >> 1) : n;
}

template <typename T>
__global__ void __launch_bounds__(256) quant_weights_kernel(const T* __restrict__ w, int64_t batch, int K, int N,
                                                            bool paired, uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ sc) {
  const int KT = (K + 127) / 128, nb = KT * 4;
  const int64_t n_all = batch * nb * (int64_t)N;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n_all; i += (int64_t)gridDim.x * blockDim.x) {
    const int n = (int)(i % N), kb = (int)(i / N % nb);
    const int64_t e = i / N / nb;
    uint32_t s = 127;
    if (kb * 32 < K) {
      const T* src = w + (e * K + kb * 32) * (int64_t)N + fp4_column(n, N, paired);
      float v[32];
      for (int j = 0; j < 32; ++j) v[j] = to_f32(src[(int64_t)j * N]);
      s = fp4_quant_block(v, q + (e * N + n) * (int64_t)(K / 2) + kb * 16);
    }
    sc[fp4_weight_scale_at(e, n, kb, N, KT)] = (uint8_t)s;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) dequant_weights_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ sc, int64_t batch, int K,
                                                              int N, bool paired, T* __restrict__ w) {
  const int KT = (K + 127) / 128;
  const int64_t n_all = batch * (int64_t)(K / 2) * N;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n_all; i += (int64_t)gridDim.x * blockDim.x) {
    const int n = (int)(i % N), c = (int)(i / N % (K / 2));
    const int64_t e = i / N / (K / 2);
    const float s = fp4_scale_of(sc[fp4_weight_scale_at(e, n, c / 16, N, KT)]);
    const uint32_t b = q[(e * N + n) * (int64_t)(K / 2) + c];
    T* dst = w + (e * K + 2 * c) * (int64_t)N + fp4_column(n, N, paired);
    dst[0] = from_f32<T>(fp4_value(b & 15u) * s);
    dst[N] = from_f32<T>(fp4_value(b >> 4) * s);
  }
}

// The product on the CUDA cores: tiles of 64 rows x 64 features, a block of K
// at a time decoded into shared memory, 4 x 4 sums a thread.
template <typename T>
__global__ void __launch_bounds__(256) product_simt_kernel(const uint8_t* __restrict__ xq,
                                                           const uint8_t* __restrict__ xs,
                                                           const uint8_t* __restrict__ wq,
                                                           const uint8_t* __restrict__ ws, int64_t rows, int N, int K,
                                                           int G, const int* __restrict__ off, bool swiglu,
                                                           T* __restrict__ out, int64_t ldo,
                                                           int* __restrict__ status) {
  __shared__ float A[64][33], B[64][33];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 2) status[threadIdx.x] = 0;
  const int KT = (K + 127) / 128;
  const int g = find_group_block(off, G, blockIdx.x, 64);
  const int64_t o = off ? off[g] : 0, cnt = (off ? off[g + 1] : rows) - o;
  const int64_t i0 = (blockIdx.x - (o / 64 + g)) * (int64_t)64;
  if (i0 >= cnt) return;
  const int n0 = blockIdx.y * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int kb = 0; kb < K / 32; ++kb) {
    __syncthreads();
    for (int j = threadIdx.x; j < 64 * 16; j += 256) {
      const int r = j / 16, c = j % 16;
      float s = 0.f;
      uint32_t b = 0;
      if (i0 + r < cnt) {
        s = fp4_scale_of(xs[fp4_row_scale_at(o, g, i0 + r, kb, KT)]);
        b = xq[(o + i0 + r) * (K / 2) + kb * 16 + c];
      }
      A[r][2 * c] = fp4_value(b & 15u) * s;
      A[r][2 * c + 1] = fp4_value(b >> 4) * s;
      s = 0.f;
      b = 0;
      if (n0 + r < N) {
        s = fp4_scale_of(ws[fp4_weight_scale_at(g, n0 + r, kb, N, KT)]);
        b = wq[((int64_t)g * N + n0 + r) * (K / 2) + kb * 16 + c];
      }
      B[r][2 * c] = fp4_value(b & 15u) * s;
      B[r][2 * c + 1] = fp4_value(b >> 4) * s;
    }
    __syncthreads();
    for (int c = 0; c < 32; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(A[ty * 4 + i][c], B[tx * 4 + j][c], acc[i][j]);
  }
  for (int i = 0; i < 4; ++i) {
    if (i0 + ty * 4 + i >= cnt) break;
    T* dst = out + (o + i0 + ty * 4 + i) * ldo;
    const int n = n0 + tx * 4;
    if (swiglu) {
      for (int j = 0; j < 4; j += 2)
        if (n + j < N) dst[(n + j) / 2] = from_f32<T>(silu_f(acc[i][j]) * acc[i][j + 1]);
    } else {
      for (int j = 0; j < 4; ++j)
        if (n + j < N) dst[n + j] = from_f32<T>(acc[i][j]);
    }
  }
}

int grid_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (int)(b < 1 ? 1 : b < (1 << 20) ? b : (1 << 20));
}
bool fp4_k(int32_t K) { return K >= 32 && K % 32 == 0 && K <= (1 << 24); }
bool fp4_weights(int64_t batch, int32_t K, int32_t N) {
  return batch >= 0 && batch <= (1 << 20) && fp4_k(K) && N >= 1 && N <= (1 << 22);
}
bool fp4_rows(int64_t rows, int32_t K, int32_t G) {
  return rows >= 0 && rows <= ((int64_t)1 << 28) && fp4_k(K) && G >= 1 && G <= kMaxE;
}
bool aligned128(const void* p) { return p != nullptr && aligned_to(p, 128); }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mxfp4_weight_scale_bytes(int64_t batch, int32_t K, int32_t N) {
  if (!fp4_weights(batch, K, N)) return 0;
  return (size_t)batch * ((N + 127) / 128) * ((K + 127) / 128) * 512;
}

size_t moe_mxfp4_row_scale_bytes(int64_t rows, int32_t K, int32_t G) {
  if (!fp4_rows(rows, K, G)) return 0;
  return (size_t)(rows / kTok + G) * 2 * ((K + 127) / 128) * 512;
}

moe_status moe_quantize_mxfp4(int32_t dtype, const void* w, int64_t batch, int32_t K, int32_t N, int32_t paired,
                              uint8_t* q, uint8_t* scales, moe_stream_t stream) {
  if (!dtype_valid(dtype) || !fp4_weights(batch, K, N) || (paired && N % 2)) return MOE_ERR_INVALID_ARG;
  if (batch == 0) return MOE_OK;
  if (!elem_ok(w, dtype_bytes(dtype)) || !aligned128(q) || !aligned128(scales)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    TraceScope ts("quantize_mxfp4_weights", st);
    quant_weights_kernel<T><<<grid_for(batch * ((K + 127) / 128) * 4 * N), 256, 0, st>>>(
        static_cast<const T*>(w), batch, K, N, paired != 0, q, scales);
    return cudaGetLastError();
  }));
}

moe_status moe_dequantize_mxfp4(int32_t dtype, const uint8_t* q, const uint8_t* scales, int64_t batch, int32_t K,
                                int32_t N, int32_t paired, void* w, moe_stream_t stream) {
  if (!dtype_valid(dtype) || !fp4_weights(batch, K, N) || (paired && N % 2)) return MOE_ERR_INVALID_ARG;
  if (batch == 0) return MOE_OK;
  if (!elem_ok(w, dtype_bytes(dtype)) || !aligned128(q) || !aligned128(scales)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    TraceScope ts("dequantize_mxfp4_weights", st);
    dequant_weights_kernel<T><<<grid_for(batch * (K / 2) * N), 256, 0, st>>>(q, scales, batch, K, N, paired != 0,
                                                                              static_cast<T*>(w));
    return cudaGetLastError();
  }));
}

moe_status moe_quantize_mxfp4_rows(int32_t dtype, int64_t rows, int32_t K, const void* x, int64_t ldx, int32_t G,
                                   const int32_t* offsets, const int32_t* perm, int32_t k, uint8_t* q,
                                   uint8_t* scales, moe_stream_t stream) {
  if (!dtype_valid(dtype) || !fp4_rows(rows, K, G) || ldx < K || k < 1 || (offsets == nullptr && G != 1))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!elem_ok(x, dtype_bytes(dtype)) || !aligned128(q) || !aligned128(scales) || !elem_ok_or_null(offsets, 4) ||
      !elem_ok_or_null(perm, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    TraceScope ts("quantize_mxfp4_rows", st);
    quant_rows_kernel<T><<<grid_for(rows * ((K + 127) / 128) * 4), 256, 0, st>>>(
        static_cast<const T*>(x), ldx, rows, K, G, offsets, perm, k, q, scales);
    return cudaGetLastError();
  }));
}

moe_status moe_dequantize_mxfp4_rows(int32_t dtype, int64_t rows, int32_t K, const uint8_t* q, const uint8_t* scales,
                                     int32_t G, const int32_t* offsets, void* y, int64_t ldy, moe_stream_t stream) {
  if (!dtype_valid(dtype) || !fp4_rows(rows, K, G) || ldy < K || (offsets == nullptr && G != 1))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!elem_ok(y, dtype_bytes(dtype)) || !aligned128(q) || !aligned128(scales) || !elem_ok_or_null(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    TraceScope ts("dequantize_mxfp4_rows", st);
    dequant_rows_kernel<T><<<grid_for(rows * (K / 2)), 256, 0, st>>>(q, scales, rows, K, G, offsets,
                                                                      static_cast<T*>(y), ldy);
    return cudaGetLastError();
  }));
}

size_t moe_mxfp4_product_workspace_bytes(int64_t rows, int32_t N, int32_t K, int32_t G) {
  if (!fp4_rows(rows, K, G) || !fp4_weights(G, K, N)) return 0;
  return 128;
}

moe_status moe_mxfp4_product(int32_t dtype, int64_t rows, int32_t N, int32_t K, int32_t G, const int32_t* offsets,
                             const uint8_t* xq, const uint8_t* xscales, const uint8_t* wq, const uint8_t* wscales,
                             int32_t act, void* out, int64_t ldo, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_valid(dtype) || !fp4_rows(rows, K, G) || !fp4_weights(G, K, N) || (offsets == nullptr && G != 1) ||
      (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU) || (act == MOE_ACT_SWIGLU && N % 2) ||
      ldo < (act == MOE_ACT_SWIGLU ? N / 2 : N) || !aligned128(ws))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_mxfp4_product_workspace_bytes(rows, N, K, G)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (rows == 0) return MOE_OK;
  if (!aligned128(xq) || !aligned128(xscales) || !aligned128(wq) || !aligned128(wscales) ||
      !elem_ok(out, dtype_bytes(dtype)) || !elem_ok_or_null(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    TraceScope ts("mxfp4_product", st);
    product_simt_kernel<T><<<dim3((unsigned)(rows / 64 + G), (N + 63) / 64), 256, 0, st>>>(
        xq, xscales, wq, wscales, rows, N, K, G, offsets, act == MOE_ACT_SWIGLU, static_cast<T*>(out), ldo,
        static_cast<int*>(ws));
    return cudaGetLastError();
  }));
}

}  // extern "C"

// permute.cu -- rows sorted by expert and back (include/moe_ops.h:
// moe_sort_rows, moe_permute, moe_unpermute, moe_unpermute_backward).
#include "ops_common.cuh"

namespace moe {

namespace {

constexpr int kPmThreads = 256;
constexpr int kSortChunk = 1024;  // routed rows of one histogram / scatter block
constexpr int kSortWarps = kPmThreads / 32;

// Expert of a row, or E for one without an expert.
__device__ __forceinline__ int bucket(int id, int E) { return (unsigned)id < (unsigned)E ? id : E; }

// hist[b][e]: rows of chunk b in bucket e (e = E: dropped rows).
__global__ void __launch_bounds__(kPmThreads) sort_hist_kernel(const int* __restrict__ ids, int64_t R, int E,
                                                               int* __restrict__ hist) {
  __shared__ int sh[kMaxE + 1];
  for (int e = threadIdx.x; e <= E; e += blockDim.x) sh[e] = 0;
  __syncthreads();
  const int64_t r0 = (int64_t)blockIdx.x * kSortChunk, r1 = min(R, r0 + kSortChunk);
  for (int64_t r = r0 + threadIdx.x; r < r1; r += blockDim.x) atomicAdd(&sh[bucket(ids[r], E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) hist[(size_t)blockIdx.x * (E + 1) + e] = sh[e];
}

// One block: hist[b][e] becomes the position of chunk b's first row of bucket e.
__global__ void __launch_bounds__(1024) sort_scan_kernel(int* __restrict__ hist, int nb, int E,
                                                         int* __restrict__ counts, int* __restrict__ offsets) {
  __shared__ int sh[kMaxE + 1];
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    int run = 0;
    for (int b = 0; b < nb; ++b) {
      const int c = hist[(size_t)b * (E + 1) + e];
      hist[(size_t)b * (E + 1) + e] = run;
      run += c;
    }
    sh[e] = run;
    if (e < E) counts[e] = run;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int run = 0;
    for (int e = 0; e <= E; ++e) {
      const int c = sh[e];
      sh[e] = run;
      offsets[e] = run;  // offsets[E]: the rows kept
      run += c;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x)
    for (int b = 0; b < nb; ++b) hist[(size_t)b * (E + 1) + e] += sh[e];
}

// Stable positions of a chunk's rows: each warp counts its rows by bucket,
// prefixes over the warps, then every row ranks among the equal ones before it.
__global__ void __launch_bounds__(kPmThreads) sort_scatter_kernel(const int* __restrict__ ids, int64_t R, int E,
                                                                  const int* __restrict__ hist,
                                                                  int* __restrict__ perm, int* __restrict__ inv) {
  __shared__ int wcnt[kSortWarps][kMaxE + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kSortWarps * (E + 1); i += blockDim.x) wcnt[i / (E + 1)][i % (E + 1)] = 0;
  __syncthreads();
  constexpr int kPerWarp = kSortChunk / kSortWarps;
  const int64_t w0 = (int64_t)blockIdx.x * kSortChunk + warp * kPerWarp;
  const int64_t w1 = min(R, w0 + kPerWarp);
  for (int64_t base = w0; base < w1; base += 32) {
    const int64_t r = base + lane;
    const int e = r < w1 ? bucket(ids[r], E) : -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(peers) - 1) wcnt[warp][e] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e <= E; e += blockDim.x) {
    int run = hist[(size_t)blockIdx.x * (E + 1) + e];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = wcnt[w][e];
      wcnt[w][e] = run;
      run += c;
    }
  }
  __syncthreads();
  for (int64_t base = w0; base < w1; base += 32) {
    const int64_t r = base + lane;
    const int e = r < w1 ? bucket(ids[r], E) : -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    int p = 0;
    if (e >= 0) p = wcnt[warp][e] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) wcnt[warp][e] += __popc(peers);
    __syncwarp();
    if (e >= 0) {
      perm[p] = (int)r;
      inv[r] = p;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kPmThreads) permute_kernel(const T* __restrict__ x, int64_t ldx,
                                                             const int* __restrict__ inv,
                                                             const int* __restrict__ kept_p, int k, int d,
                                                             int64_t T_, T* __restrict__ xp) {
  const int kept = *kept_p;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x)
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const T v = x[t * ldx + i];
      for (int j = 0; j < k; ++j) {
        const int p = inv[t * k + j];
        xp[(int64_t)p * d + i] = p < kept ? v : from_f32<T>(0.f);
      }
    }
}

template <typename T>
__global__ void __launch_bounds__(kPmThreads) unpermute_kernel(const T* __restrict__ y,
                                                               const float* __restrict__ w,
                                                               const int* __restrict__ inv,
                                                               const int* __restrict__ kept_p, int k, int d,
                                                               int64_t T_, const T* base, int64_t ldbase, T* out,
                                                               int64_t ldout) {
  const int kept = *kept_p;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x)
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      float s = base ? to_f32(base[t * ldbase + i]) : 0.f;
      for (int j = 0; j < k; ++j) {
        const int p = inv[t * k + j];
        if (p < kept) s = fmaf(w ? w[t * k + j] : 1.f, to_f32(y[(int64_t)p * d + i]), s);
      }
      out[t * ldout + i] = from_f32<T>(s);
    }
}

template <typename T>
__global__ void __launch_bounds__(kPmThreads) unpermute_backward_kernel(
    const T* __restrict__ dout, int64_t lddout, const T* __restrict__ y, const float* __restrict__ w,
    const int* __restrict__ inv, const int* __restrict__ kept_p, int k, int d, int64_t R, T* __restrict__ dy,
    float* __restrict__ dw) {
  __shared__ float sh[kPmThreads / 32];
  const int kept = *kept_p;
  for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
    const int64_t t = r / k;
    const int p = inv[r];
    const bool live = p < kept;
    const float wr = live ? (w ? w[r] : 1.f) : 0.f;
    float s = 0.f;
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float g = to_f32(dout[t * lddout + i]);
      if (dw && live) s = fmaf(g, to_f32(y[(int64_t)p * d + i]), s);
      dy[(int64_t)p * d + i] = from_f32<T>(live ? wr * g : 0.f);
    }
    if (dw) {
      s = warp_sum(s);
      __syncthreads();
      if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
      __syncthreads();
      if (threadIdx.x == 0) {
        float v = 0.f;
        for (int i = 0; i < kPmThreads / 32; ++i) v += sh[i];
        dw[r] = v;
      }
    }
  }
}

int grid_rows(int64_t n) { return (int)(n < (1 << 30) ? n : (1 << 30)); }

bool pm_args(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E) {
  return dtype_valid(dtype) && T >= 0 && d >= 1 && d <= (1 << 24) && k >= 1 && k <= kMaxK && E >= 1 && E <= kMaxE &&
         T <= (((int64_t)1 << 28) / k);
}

bool sort_args(int64_t R, int32_t E) { return R >= 0 && R <= ((int64_t)1 << 28) && E >= 1 && E <= kMaxE; }

int64_t sort_chunks(int64_t R) { return (R + kSortChunk - 1) / kSortChunk; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_sort_workspace_bytes(int64_t R, int32_t E) {
  if (!sort_args(R, E)) return 0;
  return ((size_t)(sort_chunks(R) + 1) * (E + 1) * sizeof(int) + 127) / 128 * 128;
}

moe_status moe_sort_rows(const int32_t* ids, int64_t R, int32_t E, int32_t* counts, int32_t* offsets,
                         int32_t* perm, int32_t* inv, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!sort_args(R, E) || !elem_ok(counts, 4) || !elem_ok(offsets, 4) || ws == nullptr || !aligned_to(ws, 128))
    return MOE_ERR_INVALID_ARG;
  if (R > 0 && (!elem_ok(ids, 4) || !elem_ok(perm, 4) || !elem_ok(inv, 4))) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_sort_workspace_bytes(R, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int* hist = static_cast<int*>(ws);
  const int nb = (int)sort_chunks(R);
  if (nb > 0) {
    TraceScope ts("sort_hist", st);
    sort_hist_kernel<<<nb, kPmThreads, 0, st>>>(ids, R, E, hist);
  }
  {
    TraceScope ts("sort_scan", st);
    sort_scan_kernel<<<1, 1024, 0, st>>>(hist, nb, E, counts, offsets);
  }
  if (nb > 0) {
    TraceScope ts("sort_scatter", st);
    sort_scatter_kernel<<<nb, kPmThreads, 0, st>>>(ids, R, E, hist, perm, inv);
  }
  return ops_status(cudaGetLastError());
}

moe_status moe_permute(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E, const void* x, int64_t ldx,
                       const int32_t* inv, const int32_t* offsets, void* xp, moe_stream_t stream) {
  if (!pm_args(dtype, T, d, k, E) || ldx < d) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(x, es) || !elem_ok(xp, es) || !elem_ok(inv, 4) || !elem_ok(offsets, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using U = decltype(t);
    TraceScope ts("permute", st);
    permute_kernel<U><<<grid_rows(T), kPmThreads, 0, st>>>(static_cast<const U*>(x), ldx, inv, offsets + E, k, d, T,
                                                           static_cast<U*>(xp));
    return cudaGetLastError();
  }));
}

moe_status moe_unpermute(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E, const void* y, const float* w,
                         const int32_t* inv, const int32_t* offsets, const void* base, int64_t ldbase, void* out,
                         int64_t ldout, moe_stream_t stream) {
  if (!pm_args(dtype, T, d, k, E) || ldout < d || (base != nullptr && ldbase < d)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(y, es) || !elem_ok(out, es) || !elem_ok_or_null(base, es) || !elem_ok_or_null(w, 4) ||
      !elem_ok(inv, 4) || !elem_ok(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using U = decltype(t);
    TraceScope ts("unpermute", st);
    unpermute_kernel<U><<<grid_rows(T), kPmThreads, 0, st>>>(static_cast<const U*>(y), w, inv, offsets + E, k, d, T,
                                                             static_cast<const U*>(base), ldbase,
                                                             static_cast<U*>(out), ldout);
    return cudaGetLastError();
  }));
}

moe_status moe_unpermute_backward(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E, const void* dout,
                                  int64_t lddout, const void* y, const float* w, const int32_t* inv,
                                  const int32_t* offsets, void* dy, float* dw, moe_stream_t stream) {
  if (!pm_args(dtype, T, d, k, E) || lddout < d) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(dout, es) || !elem_ok(dy, es) || !elem_ok_or_null(w, 4) || !elem_ok(inv, 4) || !elem_ok(offsets, 4) ||
      !elem_ok_or_null(dw, 4) || (dw != nullptr && !elem_ok(y, es)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(with_dtype(dtype, [&](auto t) {
    using U = decltype(t);
    TraceScope ts("unpermute_backward", st);
    unpermute_backward_kernel<U><<<grid_rows(T * k), kPmThreads, 0, st>>>(
        static_cast<const U*>(dout), lddout, static_cast<const U*>(y), w, inv, offsets + E, k, d, T * k,
        static_cast<U*>(dy), dw);
    return cudaGetLastError();
  }));
}

}  // extern "C"

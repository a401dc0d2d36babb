// ops_common.cuh -- shared by the operators of include/moe_ops.h: element
// types, vectors of a row, block reductions and argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/moe_ops.h"
#include "moe_internal.h"

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements of a row, loaded and stored as one access.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& v) {
  *reinterpret_cast<Vec<T, V>*>(p) = v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ host side
inline size_t dtype_bytes(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }
inline bool dtype_valid(int dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// a pointer that must be there, aligned to its element
inline bool elem_ok(const void* p, size_t es) { return p != nullptr && aligned_to(p, es); }
inline bool elem_ok_or_null(const void* p, size_t es) { return p == nullptr || aligned_to(p, es); }
inline moe_status ops_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// f(T{}) for the element type of dt.
template <typename F>
cudaError_t with_dtype(int dt, F f) {
  switch (dt) {
    case MOE_DT_F32: return f(float());
    case MOE_DT_BF16: return f(__nv_bfloat16());
    default: return f(__half());
  }
}

}  // namespace moe

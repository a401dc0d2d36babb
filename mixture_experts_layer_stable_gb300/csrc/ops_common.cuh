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

// Two fp32 values in a register pair: one instruction does both (each rounded
// as its scalar form).
struct F2 {
  unsigned long long v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
  __device__ __forceinline__ float2 get() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  const float2 f = a.get();
  return f.x + f.y;
}
// Elements 2k and 2k + 1 of an array of T as fp32, and back.
__device__ __forceinline__ F2 pair_f32(const float* p) { return F2(p[0], p[1]); }
__device__ __forceinline__ F2 pair_f32(const __nv_bfloat16* p) {
  const uint32_t u = (uint32_t)__bfloat16_as_ushort(p[0]) | ((uint32_t)__bfloat16_as_ushort(p[1]) << 16);
  return F2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ F2 pair_f32(const __half* p) {
  const float2 f = __half22float2(__halves2half2(p[0], p[1]));
  return F2(f.x, f.y);
}
__device__ __forceinline__ void pair_to(float* p, F2 v) {
  const float2 f = v.get();
  p[0] = f.x;
  p[1] = f.y;
}
__device__ __forceinline__ void pair_to(__nv_bfloat16* p, F2 v) {
  const float2 f = v.get();
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  p[0] = h.x;
  p[1] = h.y;
}
__device__ __forceinline__ void pair_to(__half* p, F2 v) {
  const float2 f = v.get();
  const __half2 h = __floats2half2_rn(f.x, f.y);
  p[0] = __low2half(h);
  p[1] = __high2half(h);
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

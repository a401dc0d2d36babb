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
#include "smem_limit.h"

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

// Loads of global memory that stay where they are written.  The kernels start before
// the one that writes their inputs has ended and wait for it (ops_wait), so none of
// their inputs is read-only for the whole kernel: a load that the compiler takes for
// one (__ldg, const __restrict__ pointers) might be moved before the wait.
__device__ __forceinline__ uint4 gload(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t gload(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t gload(const uint16_t* p) {
  uint16_t v;
  asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t gload(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int gload(const int* p) { return (int)gload(reinterpret_cast<const uint32_t*>(p)); }
__device__ __forceinline__ float gload(const float* p) {
  return __uint_as_float(gload(reinterpret_cast<const uint32_t*>(p)));
}
__device__ __forceinline__ float gload_f32(const float* p) { return gload(p); }
__device__ __forceinline__ float gload_f32(const __nv_bfloat16* p) {
  return __uint_as_float(gload(reinterpret_cast<const uint16_t*>(p)) << 16);
}
__device__ __forceinline__ float gload_f32(const __half* p) {
  return __half2float(__ushort_as_half((uint16_t)gload(reinterpret_cast<const uint16_t*>(p))));
}

// Two 16-bit elements at p, each only where a / b says that it exists (else 0), to be
// joined as lo | hi << 16 at their use.  Without a branch: a value loaded behind one is
// waited for where it joins.  (A third load, of both as a word into lo where p allows
// it, costs more than it saves: it waits for the other that has the same target.)
__device__ __forceinline__ void gload_pair(const void* p, bool a, bool b, uint32_t& lo, uint32_t& hi) {
  asm volatile(
      "{\n\t.reg .pred l, h;\n\t"
      "setp.ne.b32 l, %3, 0;\n\t"
      "setp.ne.b32 h, %4, 0;\n\t"
      "mov.b32 %0, 0;\n\t"
      "mov.b32 %1, 0;\n\t"
      "@l ld.global.u16 %0, [%2];\n\t"
      "@h ld.global.u16 %1, [%2+2];\n\t}"
      : "=&r"(lo), "=&r"(hi)
      : "l"(p), "r"((int)a), "r"((int)b));
}

// V consecutive elements of a row, stored as one access.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};
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
// Two elements of T, as the 32-bit words they lie in (one word of two, or two of
// one), to fp32 and back.  (Arrays of 16-bit values would be taken apart and put
// together again around every use.)
template <typename T>
__device__ __forceinline__ F2 pair_f32(const uint32_t* w);
template <>
__device__ __forceinline__ F2 pair_f32<float>(const uint32_t* w) {
  return F2(__uint_as_float(w[0]), __uint_as_float(w[1]));
}
template <>
__device__ __forceinline__ F2 pair_f32<__nv_bfloat16>(const uint32_t* w) {
  return F2(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ F2 pair_f32<__half>(const uint32_t* w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(w));
  return F2(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ void pair_to(uint32_t* w, F2 v);
template <>
__device__ __forceinline__ void pair_to<float>(uint32_t* w, F2 v) {
  const float2 f = v.get();
  w[0] = __float_as_uint(f.x);
  w[1] = __float_as_uint(f.y);
}
template <>
__device__ __forceinline__ void pair_to<__nv_bfloat16>(uint32_t* w, F2 v) {
  const float2 f = v.get();
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(f.y), "f"(f.x));
}
template <>
__device__ __forceinline__ void pair_to<__half>(uint32_t* w, F2 v) {
  const float2 f = v.get();
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[0]) : "f"(f.y), "f"(f.x));
}

// E elements of T in registers, moved V at a time (V * sizeof(T) is 16, 4 or the
// element's size): vector i of them from or to memory at p.
template <typename T, int E>
struct Words {
  static constexpr int kWords = E * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ F2 pair(int k) const { return pair_f32<T>(w + k * (int)sizeof(T) / 2); }
  __device__ __forceinline__ void set(int k, F2 v) { pair_to<T>(w + k * (int)sizeof(T) / 2, v); }
  template <int V>
  __device__ __forceinline__ void load(int i, const T* p) {  // from global memory
    if constexpr (V * sizeof(T) == 16) {
      const uint4 u = gload(reinterpret_cast<const uint4*>(p));
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    } else if constexpr (V * sizeof(T) == 4) {
      w[i] = gload(reinterpret_cast<const uint32_t*>(p));
    } else {  // one 16-bit element
      const uint32_t u = gload(reinterpret_cast<const uint16_t*>(p));
      w[i / 2] = i % 2 ? w[i / 2] | (u << 16) : u;
    }
  }
  __device__ __forceinline__ void load16_shared(int i, const T* p) {  // 16 bytes of shared memory
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[4 * i] = u.x;
    w[4 * i + 1] = u.y;
    w[4 * i + 2] = u.z;
    w[4 * i + 3] = u.w;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  template <int V>
  __device__ __forceinline__ void zero(int i) {
    if constexpr (V * sizeof(T) == 16) w[4 * i] = w[4 * i + 1] = w[4 * i + 2] = w[4 * i + 3] = 0;
    else if constexpr (V * sizeof(T) == 4) w[i] = 0;
    else if (i % 2 == 0) w[i / 2] = 0;
  }
  template <int V>
  __device__ __forceinline__ void store(int i, T* p) const {
    if constexpr (V * sizeof(T) == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    else if constexpr (V * sizeof(T) == 4) *reinterpret_cast<uint32_t*>(p) = w[i];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
  }
};

// Programmatic dependent launch: a kernel launched by launch_ops may start while the
// kernel before it in the stream still runs, as soon as every block of that one has
// started and called ops_begin (or has ended).  ops_begin lets the next kernel in
// and waits until everything before this one has completed and is visible; it comes
// before a kernel's first access to global memory.  In a chain of small operators
// this hides the launch latency of each.  (A kernel that fills shared memory calls
// the two parts apart: blocks let in at its start would begin on an SM with next to
// no L1 cache: with that a quantiser and a 4-bit product took 803 us, not 751.)
__device__ __forceinline__ void ops_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void ops_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void ops_begin() {
  ops_let_next();
  ops_wait();
}

// ------------------------------------------------------------------ host side
template <typename... P, typename... A>
cudaError_t launch_ops(const char* name, void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TraceScope ts(name, st);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

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

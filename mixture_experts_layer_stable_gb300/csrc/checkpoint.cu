// checkpoint.cu -- activations kept in 8 bits between a forward and its backward
// (include/moe_ops.h, moe_*_mxint8_rows), and SwiGLU, whose backward works from them
// (moe_swiglu_*).
//
//   block of 32: 2^s the smallest with max |v| <= 127 * 2^s, codes rint(v * 2^-s)
//   a  = g * sg * u,  sg = 1 / (1 + exp(-g))
//   dg = da * u * sg * (1 + g * (1 - sg)),  du = da * g * sg
//
// Scales are powers of two, so v * 2^-s is exact, codes do not depend on the order or
// precision of any arithmetic, and a code times its scale is exact in fp32.
//
// Every call is bound by HBM.  A thread holds V elements of a block (16 bytes of a row;
// one element of rows that are not 16-byte aligned), the 32 / V threads of a block are
// neighbours in a warp and take its maximum by shuffles, and everything a thread reads
// is loaded before anything is computed.
#include "gemm_common.cuh"
#include "ops_common.cuh"

namespace moe {

namespace {

constexpr int kThreadsCk = 256;

// Which part of which row a thread has: rpb rows a block, or several blocks (y) a row.
struct CkLay {
  int per_row;     // threads of a row
  int rpb;         // rows of a block
  uint32_t magic;  // 2^32 / per_row rounded up: thread / per_row by multiplication
  int nq;          // blocks of 32 that one pass over a row's threads covers
};

// Scale exponent of a block with max |v| = amax (finite): amax = m * 2^q, m in [1, 2), is
// at most 127 * 2^s = 1.984375 * 2^(s + 6) from s = q - 6 or q - 5 on.
__device__ __forceinline__ int int8_scale_exp(uint32_t amax_bits) {
  const int eb = (int)(amax_bits >> 23);
  if (eb == 0) return -127;  // zero or below 2^-126
  return max(-127, eb - 127 - ((amax_bits & 0x7FFFFFu) <= 0x7E0000u ? 6 : 5));
}

// Four whole numbers, each the low byte of a float that 1.5 * 2^23 was added to.
__device__ __forceinline__ uint32_t pack_bytes(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// V elements of a row in fp32 as pairs (V = 1: one element, the pair's first).
template <typename T, int V>
struct Piece {
  Words<T, V == 1 ? 2 : V> w;
  float one;
  __device__ __forceinline__ void load(const T* p, bool there) {
    if constexpr (V == 1) {
      one = there ? gload_f32(p) : 0.f;
    } else {
      if (there) w.template load<V>(0, p);
      else w.clear();
    }
  }
  __device__ __forceinline__ F2 pair(int k) const {
    if constexpr (V == 1) return F2(one, 0.f);
    else return w.pair(k);
  }
};
template <typename T, int V>
__device__ __forceinline__ void store_pairs(T* p, const F2 (&v)[(V + 1) / 2]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(v[0].get().x);
  } else {
    Words<T, V> w;
#pragma unroll
    for (int k = 0; k < V / 2; ++k) w.set(k, v[k]);
    w.template store<V>(0, p);
  }
}

// The block's codes and scale from its threads' elements; the warp calls it together.
// there: whether this thread's elements exist (else they are zeros), sub: its place in
// the block.
template <int V>
__device__ __forceinline__ void int8_store(const F2 (&v)[(V + 1) / 2], int8_t* codes, uint8_t* scale, bool there,
                                           int sub) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < (V + 1) / 2; ++k) {
    const float2 f = v[k].get();
    m = max(m, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
  }
#pragma unroll
  for (int o = 16 / V; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool finite = m < 0x7F800000u;
  const int s = finite ? int8_scale_exp(m) : 0;
  const float inv = finite ? ue8m0_inverse(s) : 0.f;
  if (!there) return;
  if (sub == 0) *scale = finite ? (uint8_t)(s + 127) : (uint8_t)255;
  const float lim = s >= 122 ? 63.f : 127.f;  // 64 * 2^122 is past fp32's range
  float r[2 * ((V + 1) / 2)];
#pragma unroll
  for (int k = 0; k < (V + 1) / 2; ++k) {
    const float2 f = v[k].get();
    // one rounding, to a whole number: the sum is in [2^23, 2^24)
    r[2 * k] = finite ? fmaf(f.x, inv, 12582912.f) : 0.f;
    r[2 * k + 1] = finite ? fmaf(f.y, inv, 12582912.f) : 0.f;
    if (s >= 122) {
      r[2 * k] = fminf(fmaxf(r[2 * k], 12582912.f - lim), 12582912.f + lim);
      r[2 * k + 1] = fminf(fmaxf(r[2 * k + 1], 12582912.f - lim), 12582912.f + lim);
    }
  }
  if constexpr (V == 1) {
    *codes = (int8_t)__float_as_uint(r[0]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(codes) = pack_bytes(r[0], r[1], r[2], r[3]);
  } else {
    uint2 w;
    w.x = pack_bytes(r[0], r[1], r[2], r[3]);
    w.y = pack_bytes(r[4], r[5], r[6], r[7]);
    *reinterpret_cast<uint2*>(codes) = w;
  }
}

// V codes and their scale byte, as loaded, and their values.
template <int V>
struct Kept {
  uint32_t w[(V + 3) / 4], byte;
  __device__ __forceinline__ void load(const int8_t* codes, const uint8_t* scale, bool there) {
    byte = 127;
#pragma unroll
    for (int i = 0; i < (V + 3) / 4; ++i) w[i] = 0;
    if (there) {
      byte = gload(scale);
      if constexpr (V == 1) {
        w[0] = gload(reinterpret_cast<const uint8_t*>(codes));
      } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) w[i] = 0;
        if constexpr (V == 8) {
          asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(codes));
        } else {
          w[0] = gload(reinterpret_cast<const uint32_t*>(codes));
        }
      }
    }
  }
  __device__ __forceinline__ void values(F2 (&v)[(V + 1) / 2]) const {
    const float s = ue8m0_value(byte);
    if constexpr (V == 1) {
      v[0] = F2((float)(int8_t)w[0] * s, 0.f);
    } else {
      // code + 128 as the low byte of 2^23, from which 2^23 + 128 is taken
      const F2 s2(s, s), off(-8388736.f, -8388736.f);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const uint32_t u = w[k / 2] ^ 0x80808080u;
        const F2 f(__uint_as_float(__byte_perm(u, 0x4B000000u, k % 2 ? 0x7542 : 0x7540)),
                   __uint_as_float(__byte_perm(u, 0x4B000000u, k % 2 ? 0x7543 : 0x7541)));
        v[k] = mul2(add2(f, off), s2);
      }
    }
  }
};

// The thread's row and its place t among the row's threads.
struct CkAt {
  int64_t row;
  int t;
  bool there;
};
__device__ __forceinline__ CkAt ck_at(const CkLay& l, int64_t rows) {
  CkAt a;
  const int r = l.rpb > 1 ? (int)__umulhi(threadIdx.x, l.magic) : 0;
  a.t = l.rpb > 1 ? (int)threadIdx.x - r * l.per_row : (int)(blockIdx.y * blockDim.x + threadIdx.x);
  a.row = (int64_t)blockIdx.x * l.rpb + r;
  a.there = r < l.rpb && a.row < rows && a.t < l.per_row;
  return a;
}

// fp16 cannot hold a code of 64 times 2^10: values past its range become its largest.
template <typename T>
__device__ __forceinline__ F2 in_range(F2 v) {
  if constexpr (sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value) {
    float2 f = v.get();
    f.x = f.x > 65504.f ? 65504.f : f.x < -65504.f ? -65504.f : f.x;  // (NaN stays)
    f.y = f.y > 65504.f ? 65504.f : f.y < -65504.f ? -65504.f : f.y;
    return F2(f.x, f.y);
  } else {
    return v;
  }
}

template <typename T, int V, int U>
__global__ void __launch_bounds__(kThreadsCk)
    int8_quantize_kernel(const T* x, int64_t ldx, int64_t rows, int n, CkLay l, int8_t* q, uint8_t* scales) {
  ops_begin();
  constexpr int L = 32 / V;
  const CkAt at = ck_at(l, rows);
  const int nb = (n + 31) / 32, sub = at.t % L;
  Piece<T, V> p[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    p[i].load(x + at.row * ldx + c, at.there && c < n);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    F2 v[(V + 1) / 2];
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) v[k] = p[i].pair(k);
    int8_store<V>(v, q + at.row * n + c, scales + at.row * nb + b, at.there && c < n, sub);
  }
}

template <typename T, int V, int U>
__global__ void __launch_bounds__(kThreadsCk)
    int8_dequantize_kernel(const int8_t* q, const uint8_t* scales, int64_t rows, int n, CkLay l, T* y, int64_t ldy) {
  ops_begin();
  constexpr int L = 32 / V;
  const CkAt at = ck_at(l, rows);
  const int nb = (n + 31) / 32, sub = at.t % L;
  Kept<V> p[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    p[i].load(q + at.row * n + c, scales + at.row * nb + b, at.there && c < n);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    if (!(at.there && c < n)) continue;
    F2 v[(V + 1) / 2];
    p[i].values(v);
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) v[k] = in_range<T>(v[k]);
    store_pairs<T, V>(y + at.row * ldy + c, v);
  }
}

// sigmoid(g) and 1 - sigmoid(g).  For 16-bit results from the hardware exponential and
// reciprocal, as the layer's (2^-18, and 0 below -87); for fp32 ones from exp(-|g|), which
// cannot overflow.
template <typename T>
__device__ __forceinline__ void sigmoids(float g, float& s, float& c) {
  if constexpr (sizeof(T) == 4) {
    const float t = expf(-fabsf(g)), r = 1.0f / (1.0f + t), q = t * r;
    s = g < 0.f ? q : r;
    c = g < 0.f ? r : q;
  } else {
    s = sigmoid_f(g);
    c = 1.0f - s;
  }
}

template <typename T, int V, int U, bool KEEP>
__global__ void __launch_bounds__(kThreadsCk)
    swiglu_forward_kernel(const T* h, int64_t ldh, int64_t rows, int f, CkLay l, T* a, int64_t lda, int8_t* q,
                          uint8_t* scales) {
  ops_begin();
  constexpr int L = 32 / V, P = (V + 1) / 2;
  const CkAt at = ck_at(l, rows);
  const int nb = (f + 31) / 32, sub = at.t % L;
  Piece<T, V> pg[U], pu[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    pg[i].load(h + at.row * ldh + c, at.there && c < f);
    pu[i].load(h + at.row * ldh + f + c, at.there && c < f);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    const bool there = at.there && c < f;
    F2 g[P], u[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      g[k] = pg[i].pair(k);
      u[k] = pu[i].pair(k);
    }
    if constexpr (KEEP) {
      int8_store<V>(g, q + at.row * 2 * f + c, scales + at.row * 2 * nb + b, there, sub);
      int8_store<V>(u, q + at.row * 2 * f + f + c, scales + at.row * 2 * nb + nb + b, there, sub);
    }
    if (!there) continue;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const float2 gf = g[k].get();
      float s0, s1, c0;
      sigmoids<T>(gf.x, s0, c0);
      sigmoids<T>(gf.y, s1, c0);
      g[k] = mul2(mul2(g[k], F2(s0, s1)), u[k]);
    }
    store_pairs<T, V>(a + at.row * lda + c, g);
  }
}

template <typename T, int V, int U, bool KEPT>
__global__ void __launch_bounds__(kThreadsCk)
    swiglu_backward_kernel(const T* da, int64_t ldda, const T* h, int64_t ldh, const int8_t* q, const uint8_t* scales,
                           int64_t rows, int f, CkLay l, T* dh, int64_t lddh, T* a, int64_t lda) {
  ops_begin();
  constexpr int L = 32 / V, P = (V + 1) / 2;
  const CkAt at = ck_at(l, rows);
  const int nb = (f + 31) / 32, sub = at.t % L;
  Piece<T, V> pd[U], pg[U], pu[U];
  Kept<V> kg[U], ku[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    const bool there = at.there && c < f;
    if constexpr (KEPT) {
      kg[i].load(q + at.row * 2 * f + c, scales + at.row * 2 * nb + b, there);
      ku[i].load(q + at.row * 2 * f + f + c, scales + at.row * 2 * nb + nb + b, there);
    } else {
      pg[i].load(h + at.row * ldh + c, there);
      pu[i].load(h + at.row * ldh + f + c, there);
    }
    pd[i].load(da + at.row * ldda + c, there);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    if (!(at.there && c < f)) continue;
    F2 g[P], u[P], d[P], again[P];
    if constexpr (KEPT) {
      kg[i].values(g);
      ku[i].values(u);
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (!KEPT) {
        g[k] = pg[i].pair(k);
        u[k] = pu[i].pair(k);
      }
      d[k] = pd[i].pair(k);
      const float2 gf = g[k].get();
      float s0, s1, c0, c1;
      sigmoids<T>(gf.x, s0, c0);
      sigmoids<T>(gf.y, s1, c1);
      const F2 s(s0, s1), gs = mul2(g[k], s);
      again[k] = mul2(gs, u[k]);
      // sg * (1 + g * (1 - sg)) = sg + (g sg)(1 - sg)
      const F2 slope = fma2(gs, F2(c0, c1), s);
      g[k] = mul2(mul2(d[k], u[k]), slope);
      u[k] = mul2(d[k], gs);
    }
    store_pairs<T, V>(dh + at.row * lddh + c, g);
    store_pairs<T, V>(dh + at.row * lddh + f + c, u);
    if (a != nullptr) store_pairs<T, V>(a + at.row * lda + c, again);
  }
}

// ------------------------------------------------------------------ host side
bool ck_args(int32_t dtype, int64_t rows, int32_t n) {
  return dtype_valid(dtype) && rows >= 0 && rows <= ((int64_t)1 << 30) && n >= 1 && n <= (1 << 22);
}
uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// Whether rows of n elements move as 16-byte vectors: `a` the or of the rows' addresses
// and strides in bytes; the codes of a vector (es * 8 bytes' worth) lie aligned too.
bool ck_vec(size_t es, int n, uintptr_t a, const void* q) {
  return ((a | (uintptr_t)n * es) & 15) == 0 && (bits(q) & (16 / es - 1)) == 0;
}

struct CkLaunch {
  CkLay lay;
  dim3 grid, block;
};
CkLaunch ck_lay(int64_t rows, int n, int V, int U) {
  CkLaunch l;
  const int nb = (n + 31) / 32;
  l.lay.nq = (nb + U - 1) / U;
  l.lay.per_row = l.lay.nq * (32 / V);
  l.lay.rpb = l.lay.per_row < kThreadsCk ? kThreadsCk / l.lay.per_row : 1;
  if (l.lay.rpb > rows) l.lay.rpb = (int)rows;
  l.lay.magic = l.lay.per_row > 1 ? (uint32_t)((((uint64_t)1 << 32) + l.lay.per_row - 1) / l.lay.per_row) : 0;
  const int used = l.lay.per_row * l.lay.rpb;
  l.block = dim3(used >= kThreadsCk ? kThreadsCk : (used + 31) / 32 * 32);
  l.grid = dim3((unsigned)((rows + l.lay.rpb - 1) / l.lay.rpb),
                l.lay.per_row > kThreadsCk ? (l.lay.per_row + kThreadsCk - 1) / kThreadsCk : 1);
  return l;
}

// Blocks of 32 that a thread of loose rows takes part in.
constexpr int kLooseU = 4;

// f(T{}, V, U) for the element type and the way rows move.
template <typename F>
cudaError_t ck_pick(int dtype, bool vec, F f) {
  return with_dtype(dtype, [&](auto t) {
    constexpr int V = 16 / (int)sizeof(t);
    return vec ? f(t, std::integral_constant<int, V>(), std::integral_constant<int, 1>())
               : f(t, std::integral_constant<int, 1>(), std::integral_constant<int, kLooseU>());
  });
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mxint8_scale_bytes(int64_t rows, int32_t n) {
  if (rows > ((int64_t)1 << 31) || !ck_args(MOE_DT_F32, rows / 2, n)) return 0;
  return (size_t)rows * ((n + 31) / 32);
}

moe_status moe_quantize_mxint8_rows(int32_t dtype, int64_t rows, int32_t n, const void* x, int64_t ldx, int8_t* q,
                                    uint8_t* scales, moe_stream_t stream) {
  if (!ck_args(dtype, rows, n) || ldx < n) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(x, es) || q == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(ck_pick(dtype, ck_vec(es, n, bits(x) | (uintptr_t)(ldx * es), q), [&](auto t, auto v, auto u) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value, U = decltype(u)::value;
    const CkLaunch l = ck_lay(rows, n, V, U);
    return launch_ops("quantize_mxint8_rows", int8_quantize_kernel<T, V, U>, l.grid, l.block, 0, st,
                      static_cast<const T*>(x), ldx, rows, n, l.lay, q, scales);
  }));
}

moe_status moe_dequantize_mxint8_rows(int32_t dtype, int64_t rows, int32_t n, const int8_t* q, const uint8_t* scales,
                                      void* y, int64_t ldy, moe_stream_t stream) {
  if (!ck_args(dtype, rows, n) || ldy < n) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(y, es) || q == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(ck_pick(dtype, ck_vec(es, n, bits(y) | (uintptr_t)(ldy * es), q), [&](auto t, auto v, auto u) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value, U = decltype(u)::value;
    const CkLaunch l = ck_lay(rows, n, V, U);
    return launch_ops("dequantize_mxint8_rows", int8_dequantize_kernel<T, V, U>, l.grid, l.block, 0, st, q, scales,
                      rows, n, l.lay, static_cast<T*>(y), ldy);
  }));
}

moe_status moe_swiglu_forward(int32_t dtype, int64_t rows, int32_t f, const void* h, int64_t ldh, void* a, int64_t lda,
                              int8_t* q, uint8_t* scales, moe_stream_t stream) {
  if (!ck_args(dtype, rows, f) || ldh < 2 * (int64_t)f || lda < f || (q == nullptr) != (scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(h, es) || !elem_ok(a, es)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = ck_vec(es, f, bits(h) | bits(a) | (uintptr_t)(ldh * es) | (uintptr_t)(lda * es), q);
  return ops_status(ck_pick(dtype, vec, [&](auto t, auto v, auto u) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value, U = decltype(u)::value;
    const CkLaunch l = ck_lay(rows, f, V, U);
    auto kern = q ? swiglu_forward_kernel<T, V, U, true> : swiglu_forward_kernel<T, V, U, false>;
    return launch_ops("swiglu_forward", kern, l.grid, l.block, 0, st, static_cast<const T*>(h), ldh, rows, f, l.lay,
                      static_cast<T*>(a), lda, q, scales);
  }));
}

moe_status moe_swiglu_backward(int32_t dtype, int64_t rows, int32_t f, const void* da, int64_t ldda, const void* h,
                               int64_t ldh, const int8_t* q, const uint8_t* scales, void* dh, int64_t lddh, void* a,
                               int64_t lda, moe_stream_t stream) {
  if (!ck_args(dtype, rows, f) || ldda < f || lddh < 2 * (int64_t)f || (h != nullptr && ldh < 2 * (int64_t)f) ||
      (a != nullptr && lda < f) || (q == nullptr) != (scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(da, es) || !elem_ok(dh, es) || !elem_ok_or_null(h, es) || !elem_ok_or_null(a, es) ||
      (h == nullptr && q == nullptr))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const uintptr_t rows_at = bits(da) | bits(dh) | bits(a) | bits(h) | (uintptr_t)(ldda * es) | (uintptr_t)(lddh * es) |
                            (uintptr_t)((a ? lda : 0) * es) | (uintptr_t)((h ? ldh : 0) * es);
  return ops_status(ck_pick(dtype, ck_vec(es, f, rows_at, h ? nullptr : q), [&](auto t, auto v, auto u) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value, U = decltype(u)::value;
    const CkLaunch l = ck_lay(rows, f, V, U);
    auto kern = h ? swiglu_backward_kernel<T, V, U, false> : swiglu_backward_kernel<T, V, U, true>;
    return launch_ops("swiglu_backward", kern, l.grid, l.block, 0, st, static_cast<const T*>(da), ldda,
                      static_cast<const T*>(h), ldh, q, scales, rows, f, l.lay, static_cast<T*>(dh), lddh,
                      static_cast<T*>(a), lda);
  }));
}

}  // extern "C"

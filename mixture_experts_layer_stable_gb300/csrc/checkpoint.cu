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
// Every call is bound by HBM.  A thread holds V elements of a block: 16 bytes of a row as
// one access, 8 where rows allow no more, eight elements in four words, or four elements
// one by one in rows that start anywhere.  The 32 / V threads of a block are neighbours in
// a warp and take its maximum by shuffles, and everything a thread reads is loaded before
// anything is computed.
#include "gemm_common.cuh"
#include "ops_common.cuh"

namespace moe {

namespace {

constexpr int kThreadsCk = 256;
// Pieces of a thread: 32768 rows of 4096 bf16 to 8 bits 80 us with one, 68 with two, 66 with
// four, back 76, 64, 66.
constexpr int kPieces = 2;

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

// One element where it exists, else 0, without a branch (behind one it would be waited for).
__device__ __forceinline__ uint32_t gload_if(const uint32_t* p, bool there) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}"
               : "=&r"(v) : "l"(p), "r"((int)there));
  return v;
}
__device__ __forceinline__ uint32_t gload_if(const uint16_t* p, bool there) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
               : "=&r"(v) : "l"(p), "r"((int)there));
  return v;
}
__device__ __forceinline__ uint32_t gload_if(const uint8_t* p, bool there) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.u8 %0, [%1];\n\t}"
               : "=&r"(v) : "l"(p), "r"((int)there));
  return v;
}

// V elements of a row, of which n exist (the others are zeros), as one access (all of them or
// none exist).  LOOSE 1: one by one; 2: 16-bit elements two by two (n is even).
template <typename T, int V, int LOOSE>
struct Piece {
  Words<T, V> w;
  uint32_t one[LOOSE == 1 ? V : 1];
  // the elements, before their first use
  __device__ __forceinline__ void join() {
    if constexpr (LOOSE == 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (sizeof(T) == 4) w.w[j] = one[j];
        else w.w[j / 2] = j % 2 ? w.w[j / 2] | one[j] << 16 : one[j];
      }
    }
  }
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (LOOSE == 2) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) w.w[j] = gload_if(reinterpret_cast<const uint32_t*>(p + 2 * j), 2 * j < n);
    } else if constexpr (LOOSE == 1) {
      using E = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
#pragma unroll
      for (int j = 0; j < V; ++j) one[j] = gload_if(reinterpret_cast<const E*>(p + j), j < n);
    } else if (n <= 0) {
      w.clear();
    } else if constexpr (V * sizeof(T) == 8) {
      asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w.w[0]), "=r"(w.w[1]) : "l"(p));
    } else {
      w.template load<V>(0, p);
    }
  }
  __device__ __forceinline__ void store(T* p, int n) const {
    if constexpr (LOOSE == 2) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j)
        if (2 * j < n) *reinterpret_cast<uint32_t*>(p + 2 * j) = w.w[j];
    } else if constexpr (LOOSE == 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (sizeof(T) == 4) {
          if (j < n) *reinterpret_cast<uint32_t*>(p + j) = w.w[j];
        } else {
          if (j < n) *reinterpret_cast<uint16_t*>(p + j) = (uint16_t)(w.w[j / 2] >> (16 * (j % 2)));
        }
      }
    } else if (n > 0) {
      if constexpr (V * sizeof(T) == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w.w[0], w.w[1]);
      else w.template store<V>(0, p);
    }
  }
  // the bits of max |v| in fp32
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) m = max(m, w.w[j] & 0x7FFFFFFFu);
      return m;
    } else {  // two at a time: magnitudes are ordered as their bits are
      uint32_t m = w.w[0] & 0x7FFF7FFFu;
#pragma unroll
      for (int j = 1; j < V / 2; ++j) m = __vmaxu2(m, w.w[j] & 0x7FFF7FFFu);
      const uint32_t one = max(m >> 16, m & 0xFFFFu);
      if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((uint16_t)one)));
      else return one << 16;
    }
  }
};

// The block's codes and scale from its threads' elements (n of V exist here, this thread's
// place in the block is sub); the warp calls it together.
template <typename T, int V, int LOOSE>
__device__ __forceinline__ void int8_store(const Piece<T, V, LOOSE>& x, int8_t* codes, uint8_t* scale, int n, int sub) {
  uint32_t m = x.top();
#pragma unroll
  for (int o = 16 / V; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool finite = m < 0x7F800000u;
  const int s = finite ? int8_scale_exp(m) : 0;
  const float inv = ue8m0_inverse(s);
  if (n <= 0) return;
  if (sub == 0) *scale = finite ? (uint8_t)(s + 127) : (uint8_t)255;
  const F2 inv2(inv, inv), magic(12582912.f, 12582912.f);
  float r[V];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    // one rounding, to a whole number: the sum is in [2^23, 2^24)
    const float2 f = fma2(x.w.pair(k), inv2, magic).get();
    r[2 * k] = f.x;
    r[2 * k + 1] = f.y;
  }
  if (finite && s >= 122) {  // 64 * 2^122 is past fp32's range
#pragma unroll
    for (int k = 0; k < V; ++k) r[k] = fminf(fmaxf(r[k], 12582912.f - 63.f), 12582912.f + 63.f);
  }
  uint32_t w[V / 4];
#pragma unroll
  for (int k = 0; k < V / 4; ++k)
    w[k] = finite ? pack_bytes(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]) : 0u;
  if constexpr (LOOSE == 2) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
      if (2 * j < n) *reinterpret_cast<uint16_t*>(codes + 2 * j) = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
  } else if constexpr (LOOSE == 1) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) codes[j] = (int8_t)(w[j / 4] >> (8 * (j % 4)));
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint32_t*>(codes) = w[0];
  } else {
    *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
  }
}

// V codes and their scale byte, as loaded, and their values.
template <int V, int LOOSE>
struct Kept {
  uint32_t w[V / 4], byte, one[LOOSE == 1 ? V : LOOSE == 2 ? V / 2 : 1];
  __device__ __forceinline__ void load(const int8_t* codes, const uint8_t* scale, int n) {
    byte = gload_if(scale, n > 0);
    if constexpr (LOOSE == 2) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) one[j] = gload_if(reinterpret_cast<const uint16_t*>(codes + 2 * j), 2 * j < n);
    } else if constexpr (LOOSE == 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) one[j] = gload_if(reinterpret_cast<const uint8_t*>(codes + j), j < n);
    } else if (n > 0) {
      if constexpr (V == 8) asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(codes));
      else w[0] = gload(reinterpret_cast<const uint32_t*>(codes));
    }
  }
  __device__ __forceinline__ void values(F2 (&v)[V / 2]) {
    if constexpr (LOOSE == 2) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) w[i] = one[2 * i] | one[2 * i + 1] << 16;
    } else if constexpr (LOOSE == 1) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) w[i] = one[4 * i] | one[4 * i + 1] << 8 | one[4 * i + 2] << 16 | one[4 * i + 3] << 24;
    }
    // code + 128 as the low byte of 2^23, from which 2^23 + 128 is taken
    const float s = ue8m0_value(byte);
    const F2 s2(s, s), off(-8388736.f, -8388736.f);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const uint32_t u = w[k / 2] ^ 0x80808080u;
      const F2 f(__uint_as_float(__byte_perm(u, 0x4B000000u, k % 2 ? 0x7542 : 0x7540)),
                 __uint_as_float(__byte_perm(u, 0x4B000000u, k % 2 ? 0x7543 : 0x7541)));
      v[k] = mul2(add2(f, off), s2);
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

template <typename T, int V, int LOOSE>
__global__ void __launch_bounds__(kThreadsCk)
    int8_quantize_kernel(const T* x, int64_t ldx, int64_t rows, int n, CkLay l, int8_t* q, uint8_t* scales) {
  ops_begin();
  constexpr int L = 32 / V;
  const CkAt at = ck_at(l, rows);
  const int nb = (n + 31) / 32, sub = at.t % L;
  Piece<T, V, LOOSE> p[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    p[i].load(x + at.row * ldx + c, at.there ? n - c : 0);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    p[i].join();
    int8_store(p[i], q + at.row * n + c, scales + at.row * nb + b, at.there ? n - c : 0, sub);
  }
}

template <typename T, int V, int LOOSE>
__global__ void __launch_bounds__(kThreadsCk)
    int8_dequantize_kernel(const int8_t* q, const uint8_t* scales, int64_t rows, int n, CkLay l, T* y, int64_t ldy) {
  ops_begin();
  constexpr int L = 32 / V;
  const CkAt at = ck_at(l, rows);
  const int nb = (n + 31) / 32, sub = at.t % L;
  Kept<V, LOOSE> p[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    p[i].load(q + at.row * n + c, scales + at.row * nb + b, at.there ? n - c : 0);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    if (!(at.there && c < n)) continue;
    F2 v[V / 2];
    Piece<T, V, LOOSE> o;
    p[i].values(v);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) o.w.set(k, in_range<T>(v[k]));
    o.store(y + at.row * ldy + c, n - c);
  }
}

// sigmoid(g) and 1 - sigmoid(g).  For 16-bit results from the hardware exponential and
// reciprocal, as the layer's (2^-18 from -20 on, where the exponential's 2 + 1.173 |g| ulp
// begin to count 2^-16, and 0 below -87); for fp32 ones from exp(-|g|), which
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

template <typename T, int V, int LOOSE, bool KEEP>
__global__ void __launch_bounds__(kThreadsCk)
    swiglu_forward_kernel(const T* h, int64_t ldh, int64_t rows, int f, CkLay l, T* a, int64_t lda, int8_t* q,
                          uint8_t* scales) {
  ops_begin();
  constexpr int L = 32 / V, P = V / 2;
  const CkAt at = ck_at(l, rows);
  const int nb = (f + 31) / 32, sub = at.t % L;
  Piece<T, V, LOOSE> pg[kPieces], pu[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    const int n = at.there ? f - c : 0;
    pg[i].load(h + at.row * ldh + c, n);
    pu[i].load(h + at.row * ldh + f + c, n);
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    const int n = at.there ? f - c : 0;
    pg[i].join();
    pu[i].join();
    if constexpr (KEEP) {
      int8_store(pg[i], q + at.row * 2 * f + c, scales + at.row * 2 * nb + b, n, sub);
      int8_store(pu[i], q + at.row * 2 * f + f + c, scales + at.row * 2 * nb + nb + b, n, sub);
    }
    if (n <= 0) continue;
    Piece<T, V, LOOSE> o;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const F2 g = pg[i].w.pair(k);
      const float2 gf = g.get();
      float s0, s1, c0;
      sigmoids<T>(gf.x, s0, c0);
      sigmoids<T>(gf.y, s1, c0);
      o.w.set(k, mul2(mul2(g, F2(s0, s1)), pu[i].w.pair(k)));
    }
    o.store(a + at.row * lda + c, n);
  }
}

template <typename T, int V, int LOOSE, bool KEPT>
__global__ void __launch_bounds__(kThreadsCk)
    swiglu_backward_kernel(const T* da, int64_t ldda, const T* h, int64_t ldh, const int8_t* q, const uint8_t* scales,
                           int64_t rows, int f, CkLay l, T* dh, int64_t lddh, T* a, int64_t lda) {
  ops_begin();
  constexpr int L = 32 / V, P = V / 2;
  const CkAt at = ck_at(l, rows);
  const int nb = (f + 31) / 32, sub = at.t % L;
  Piece<T, V, LOOSE> pd[kPieces], pg[kPieces], pu[kPieces];
  Kept<V, LOOSE> kg[kPieces], ku[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    const int n = at.there ? f - c : 0;
    if constexpr (KEPT) {
      kg[i].load(q + at.row * 2 * f + c, scales + at.row * 2 * nb + b, n);
      ku[i].load(q + at.row * 2 * f + f + c, scales + at.row * 2 * nb + nb + b, n);
    } else {
      pg[i].load(h + at.row * ldh + c, n);
      pu[i].load(h + at.row * ldh + f + c, n);
    }
    pd[i].load(da + at.row * ldda + c, n);
  }
  // dh may be h and a may be da, and du needs no u, a no da: no store moves up over the loads
  // (which the compiler does not know to read memory)
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int b = at.t / L + i * l.nq, c = b * 32 + sub * V;
    if (!(at.there && c < f)) continue;
    F2 g[P], u[P];
    Piece<T, V, LOOSE> og, ou, oa;
    pd[i].join();
    if constexpr (KEPT) {
      kg[i].values(g);
      ku[i].values(u);
    } else {
      pg[i].join();
      pu[i].join();
    }
#pragma unroll
    for (int k = 0; k < P; ++k) {
      if constexpr (!KEPT) {
        g[k] = pg[i].w.pair(k);
        u[k] = pu[i].w.pair(k);
      }
      const F2 d = pd[i].w.pair(k);
      const float2 gf = g[k].get();
      float s0, s1, c0, c1;
      sigmoids<T>(gf.x, s0, c0);
      sigmoids<T>(gf.y, s1, c1);
      const F2 s(s0, s1), gs = mul2(g[k], s);
      oa.w.set(k, mul2(gs, u[k]));
      // sg * (1 + g * (1 - sg)) = sg + (g sg)(1 - sg)
      const F2 slope = fma2(gs, F2(c0, c1), s);
      og.w.set(k, mul2(mul2(d, u[k]), slope));
      ou.w.set(k, mul2(d, gs));
    }
    og.store(dh + at.row * lddh + c, f - c);
    ou.store(dh + at.row * lddh + f + c, f - c);
    if (a != nullptr) oa.store(a + at.row * lda + c, f - c);
  }
}

// ------------------------------------------------------------------ host side
bool ck_args(int32_t dtype, int64_t rows, int32_t n) {
  return dtype_valid(dtype) && rows >= 0 && rows <= ((int64_t)1 << 30) && n >= 1 && n <= (1 << 22);
}
uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// Bytes that a thread moves at once of rows of n elements: 16, 8 or 4 (of 16-bit types)
// where every row allows it, else 0, one by one.  (12793 rows of 2 x 4690 bf16, in words:
// forward with its checkpoint 119 us, backward 131, one by one 367 together; 71 and 89 for
// the bytes.  5331 rows of 2 x 1333 fp16, one by one: 25 and 31; 8 and 10 for the bytes.)  `a`: the or of the rows' addresses and
// strides in bytes; the codes of a vector lie aligned too.
int ck_bytes(size_t es, int n, uintptr_t a, const void* q) {
  a |= (uintptr_t)n * es;
  if (((a & 15) | (bits(q) & (16 / es - 1))) == 0) return 16;
  if (es == 2 && ((a & 7) | (bits(q) & 3)) == 0) return 8;
  return es == 2 && ((a & 3) | (bits(q) & 1)) == 0 ? 4 : 0;
}

struct CkLaunch {
  CkLay lay;
  dim3 grid, block;
};
CkLaunch ck_lay(int64_t rows, int n, int V) {
  CkLaunch l;
  const int nb = (n + 31) / 32;
  l.lay.nq = (nb + kPieces - 1) / kPieces;
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

template <typename T_, int V_, int LOOSE_>
struct CkTag {
  using T = T_;
  static constexpr int V = V_;
  static constexpr int LOOSE = LOOSE_;
};
// f(tag) for the element type and the way rows move.
template <typename F>
cudaError_t ck_pick(int dtype, int bytes, F f) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (bytes == 16) return f(CkTag<T, 16 / (int)sizeof(T), 0>());
    if constexpr (sizeof(T) == 2) {
      if (bytes == 8) return f(CkTag<T, 4, 0>());
      if (bytes == 4) return f(CkTag<T, 8, 2>());
    }
    return f(CkTag<T, 4, 1>());
  });
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mxint8_scale_bytes(int64_t rows, int32_t n) {
  if (rows < 0 || rows > ((int64_t)1 << 31) || !ck_args(MOE_DT_F32, 0, n)) return 0;  // (two a row of SwiGLU's)
  return (size_t)rows * ((n + 31) / 32);
}

moe_status moe_quantize_mxint8_rows(int32_t dtype, int64_t rows, int32_t n, const void* x, int64_t ldx, int8_t* q,
                                    uint8_t* scales, moe_stream_t stream) {
  if (!ck_args(dtype, rows, n) || ldx < n) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(x, es) || q == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return ops_status(ck_pick(dtype, ck_bytes(es, n, bits(x) | (uintptr_t)(ldx * es), q), [&](auto tag) {
    using K = decltype(tag);
    using T = typename K::T;
    const CkLaunch l = ck_lay(rows, n, K::V);
    return launch_ops("quantize_mxint8_rows", int8_quantize_kernel<T, K::V, K::LOOSE>, l.grid, l.block, 0, st,
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
  return ops_status(ck_pick(dtype, ck_bytes(es, n, bits(y) | (uintptr_t)(ldy * es), q), [&](auto tag) {
    using K = decltype(tag);
    using T = typename K::T;
    const CkLaunch l = ck_lay(rows, n, K::V);
    return launch_ops("dequantize_mxint8_rows", int8_dequantize_kernel<T, K::V, K::LOOSE>, l.grid, l.block, 0, st, q, scales,
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
  const int bytes = ck_bytes(es, f, bits(h) | bits(a) | (uintptr_t)(ldh * es) | (uintptr_t)(lda * es), q);
  return ops_status(ck_pick(dtype, bytes, [&](auto tag) {
    using K = decltype(tag);
    using T = typename K::T;
    const CkLaunch l = ck_lay(rows, f, K::V);
    auto kern = q ? swiglu_forward_kernel<T, K::V, K::LOOSE, true> : swiglu_forward_kernel<T, K::V, K::LOOSE, false>;
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
  return ops_status(ck_pick(dtype, ck_bytes(es, f, rows_at, h ? nullptr : q), [&](auto tag) {
    using K = decltype(tag);
    using T = typename K::T;
    const CkLaunch l = ck_lay(rows, f, K::V);
    auto kern = h ? swiglu_backward_kernel<T, K::V, K::LOOSE, false> : swiglu_backward_kernel<T, K::V, K::LOOSE, true>;
    return launch_ops("swiglu_backward", kern, l.grid, l.block, 0, st, static_cast<const T*>(da), ldda,
                      static_cast<const T*>(h), ldh, q, scales, rows, f, l.lay, static_cast<T*>(dh), lddh,
                      static_cast<T*>(a), lda);
  }));
}

}  // extern "C"

// mxfp4.cu -- microscaled 4-bit floating point (include/moe_ops.h): the
// quantisers, their inverses and the experts' product.
//
// Block format: 32 elements along K share a UE8M0 scale 2^s, elements E2M1.
// s is the smallest exponent with max |v| <= 6 * 2^s, so no element saturates:
// with max |v| = m * 2^q, m in [0.5, 1), 6 * 2^s = 0.75 * 2^(s+3) gives
// s = q - 3 for m <= 0.75 and q - 2 otherwise.
#include "gemm_common.cuh"
#include "ops_common.cuh"
#include "row_tiles.h"

namespace moe {

namespace {

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
// Eight values as 4-bit codes (lowest index in the lowest bits), to nearest, ties to even.
__device__ __forceinline__ uint32_t fp4_pack8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Value of a 4-bit code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives): codes
// 2..7 are a two-bit exponent and one mantissa bit, 1 is 0.5.
__device__ __forceinline__ float fp4_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const uint32_t b = m >= 2 ? (m << 22) + 0x3F000000u : m * 0x3F000000u;
  return __uint_as_float(b | ((c & 8u) << 28));
}

// Offset of the scale of row i of expert g (whose rows start at off), block kb:
// off / 128 + g leaves every expert room for its rows rounded up to 128.
__device__ __forceinline__ size_t fp4_row_scale_at(uint32_t off, uint32_t g, uint32_t i, uint32_t kb, uint32_t KT) {
  const uint32_t run = off / 128 + g + i / 128, r = i % 128;
  return ((size_t)run * KT + (kb >> 2)) * 512u + 16 * (r & 31) + 4 * (r >> 5) + (kb & 3);
}
__host__ __device__ inline size_t fp4_weight_scale_at(int64_t e, int n, int kb, int N, int KT) {
  return ((size_t)(e * ((N + 127) / 128) + (n >> 7)) * KT + (kb >> 2)) * 512u + 16 * (n & 31) +
         4 * ((n & 127) >> 5) + (kb & 3);
}

// One block of 32 values: 16 bytes of codes and the scale byte.
__device__ __forceinline__ uint32_t fp4_quant_block(float* v, uint8_t* q) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  uint4 code = make_uint4(0, 0, 0, 0);
  uint32_t byte = 255;
  if (m < 0x7F800000u) {
    const int s = fp4_scale_exp(__uint_as_float(m));
    const float f = fp4_inv_scale(s);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= f;
    code = make_uint4(fp4_pack8(v), fp4_pack8(v + 8), fp4_pack8(v + 16), fp4_pack8(v + 24));
    byte = (uint32_t)(s + 127);
  }
  *reinterpret_cast<uint4*>(q) = code;
  return byte;
}

// ------------------------------------------------------------------ rows
// Expert of row p, the same in every lane: each compares 1/32 of the offsets, twice.
__device__ __forceinline__ int warp_find_group(const int* __restrict__ off, int G, int p, int lane) {
  if (off == nullptr) return 0;
  const int stride = (G + 31) >> 5;
  const int i = lane * stride;
  const uint32_t b = __ballot_sync(0xffffffffu, i < G && gload(off + i) <= p);
  const int lo = (31 - __clz(b | 1u)) * stride;
  const bool in = lane < stride && lo + lane < G && gload(off + lo + lane) <= p;
  return lo + 31 - __clz(__ballot_sync(0xffffffffu, in) | 1u);
}

// The same for a row of each lane's own.
__device__ __forceinline__ int lane_find_group(const int* off, int G, int p) {
  if (off == nullptr) return 0;
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gload(off + mid) <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A block of 32 elements as loaded: 16 bytes at a time when V, else one by one.
template <typename T, bool V>
struct Block32 {
  static constexpr int W = V ? 16 / sizeof(T) : 1;
  Words<T, 32> e;
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 32 / W; ++i) e.template load<W>(i, p + i * W);
  }
  // Bits of the largest magnitude as fp32 (of a NaN or infinity: 0x7F800000 or more).
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 2) {
      // magnitudes order as their bits do: 16-bit integer maxima, two at a time
#pragma unroll
      for (int i = 0; i < 16; ++i) m = __vmaxu2(m, e.w[i] & 0x7FFF7FFFu);
      const uint16_t h = (uint16_t)max(m & 0xFFFFu, m >> 16);
      return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&h)));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, e.w[i] & 0x7FFFFFFFu);
      return m;
    }
  }
};

// One lane a block (the blocks that pad a row's last scale tile included, scale 1):
// the block's maximum needs no exchange, its codes leave as 16 bytes, and four lanes
// join their scale bytes into a word of the tile.  A block of threads takes one row
// (or 256 blocks of a wider one), or `rpb` short ones: it is bound by instruction
// issue, and finding places by dividing a flat index cost a tenth of its time
// (32768 x 7168: 104 us, now 95, 5.9 TB/s).
template <typename T, bool V>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T* x, int64_t ldx, int rows, int K, int G,
                                                         const int* off, const int* perm, int k, int rpb, uint8_t* q,
                                                         uint8_t* sc) {
  ops_begin();
  const int lane = threadIdx.x & 31, KT = (K + 127) / 128, nb = KT * 4;
  const int sub = rpb > 1 ? (int)threadIdx.x / nb : 0;
  const int p_raw = (int)blockIdx.x * rpb + sub, p = min(p_raw, rows - 1);
  const int kb = rpb > 1 ? (int)threadIdx.x - sub * nb : (int)(blockIdx.y * 256 + threadIdx.x);
  const bool mine = p_raw < rows && sub < rpb && kb < nb, in = mine && kb * 32 < K;
  Block32<T, V> v;
  if (in) v.load(x + (int64_t)(perm ? gload(perm + p) / k : p) * ldx + kb * 32);
  const int g = rpb > 1 ? lane_find_group(off, G, p) : warp_find_group(off, G, p, lane);
  const int o = off ? gload(off + g) : 0;
  // (rows before the first segment are none's: their places would lie before the scales)
  const bool live = mine && (off == nullptr || (p >= o && o >= 0 && p < gload(off + G)));
  uint32_t byte = 127;
  if (in && live) {
    const uint32_t m = v.max_bits();
    const int s = m < 0x7F800000u ? fp4_scale_exp(__uint_as_float(m)) : 0;
    const float f = fp4_inv_scale(s);
    byte = m < 0x7F800000u ? (uint32_t)(s + 127) : 255u;
    uint32_t c[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 t = mul2(v.e.pair(w * 4 + j), F2(f, f)).get();
        y[2 * j] = t.x;
        y[2 * j + 1] = t.y;
      }
      c[w] = byte != 255u ? fp4_pack8(y) : 0u;
    }
    *reinterpret_cast<uint4*>(q + (int64_t)p * (K / 2) + kb * 16) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  byte <<= 8 * (lane & 3);
  byte |= __shfl_xor_sync(0xffffffffu, byte, 1);
  byte |= __shfl_xor_sync(0xffffffffu, byte, 2);
  if ((lane & 3) == 0 && live) *reinterpret_cast<uint32_t*>(sc + fp4_row_scale_at(o, g, p - o, kb, KT)) = byte;
}

// Two values of a byte of codes.
__device__ __forceinline__ float2 fp4_values2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A warp takes up to kSegPasses passes of 256 elements of one row, a lane 8
// elements a pass (four lanes a block), so that stores are whole lines.
constexpr int kSegPasses = 7;

template <typename T, bool V>
__global__ void __launch_bounds__(256) dequant_rows_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ sc, int64_t rows, int K,
                                                           int G, const int* __restrict__ off, int segs, int per,
                                                           T* __restrict__ y, int64_t ldy) {
  ops_begin();
  const int lane = threadIdx.x & 31, KT = (K + 127) / 128;
  const int64_t w = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5;
  const int64_t p = w / segs;
  const int pass0 = (int)(w % segs) * per;
  if (p >= rows || (off != nullptr && p >= gload(off + G))) return;
  uint32_t code[kSegPasses];
#pragma unroll
  for (int i = 0; i < kSegPasses; ++i) {
    const int c = (pass0 + i) * 256 + lane * 8;
    code[i] = i < per && c < K ? gload(reinterpret_cast<const uint32_t*>(q + p * (K / 2) + c / 2)) : 0u;
  }
  const int g = warp_find_group(off, G, (int)p, lane);
  const int64_t o = off ? gload(off + g) : 0;
  if (p < o || o < 0) return;  // a row before the first segment
  uint32_t sb[kSegPasses];
#pragma unroll
  for (int i = 0; i < kSegPasses; ++i) {
    const int c = (pass0 + i) * 256 + lane * 8;
    sb[i] = i < per && c < K ? gload(sc + fp4_row_scale_at((uint32_t)o, g, (uint32_t)(p - o), c / 32, KT)) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kSegPasses; ++i) {
    const int c = (pass0 + i) * 256 + lane * 8;
    if (i >= per || c >= K) break;
    const float s = fp4_scale_of(sb[i]);
    constexpr int W = V ? 16 / sizeof(T) : 1;
    Vec<T, W> o8[8 / W];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = fp4_values2(code[i] >> (8 * j));
      o8[2 * j / W].e[2 * j % W] = from_f32<T>(f.x * s);
      o8[(2 * j + 1) / W].e[(2 * j + 1) % W] = from_f32<T>(f.y * s);
    }
#pragma unroll
    for (int j = 0; j < 8 / W; ++j) store_vec<T, W>(y + p * ldy + c + j * W, o8[j]);
  }
}

// Segments of a row, and passes of each.
struct Segs {
  int n, per;
};
Segs row_segs(int K) {
  const int passes = (K + 255) / 256;
  Segs s;
  s.n = (passes + kSegPasses - 1) / kSegPasses;
  s.per = (passes + s.n - 1) / s.n;
  return s;
}
// Rows whose 8-element groups are 16-byte aligned.
bool rows16(const void* p, int64_t ld, int dt) {
  return aligned_to(p, 16) && ld * (int64_t)dtype_bytes(dt) % 16 == 0;
}

// Column of w that row n of the codes holds.
__device__ __forceinline__ int fp4_column(int n, int N, bool paired) {
  return paired ? (n & 1) * (N / 2) + (n >> 1) : n;
}

// Weights, once when they are frozen: a lane a block of a column, neighbouring lanes
// neighbouring columns (16 x 7168 x 4096 in bf16: 262 us, 4.5 of HBM's 6.8 TB/s).
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

// Their values, to look at them: a lane a byte of codes, and neighbouring lanes' bytes
// lie K / 2 apart (the same weights: 1407 us, 175 for the bytes).
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

// ------------------------------------------------------------------ the product
// Warp-specialised, persistent, one CTA per SM: warp 0 issues the copies, one
// thread of warp 1 the tensor-core instructions, warps 2..9 the epilogue.
//
// The weights are the MMA's A operand (M = 128 features) and the rows its B
// (N = rows of the tile rounded up to 16, at most kMaxTok): the accumulator
// holds features on TMEM lanes and rows on TMEM columns, so an expert with a
// few rows costs its weight stream and little else.  A unit of work is (expert,
// 128 features, tile of rows); a stage of the ring holds 256 elements of K:
//   weights 128 x 128 B, rows up to 192 x 128 B (both 128-byte swizzled), their
//   scale tiles (2 x 512 B for the features and for each 128 rows).
// The stage's scale tiles are copied to TMEM (tcgen05.cp) right before its four
// MMAs of K = 64, into the stage's own columns.
// TMEM: two accumulators as wide as the largest tile of rows (at most 192
// columns), then 24 scale columns for every stage.
//
// When experts have few rows a stage is 17 KB of weights, 0.38 us of an SM's share
// of HBM, and issuing its copies and MMAs must not take longer: the copy and MMA
// warps run their loops in all lanes without branches, every copy and MMA
// predicated on one elected lane and on what the stage needs, and wait out of
// line.  The election has to stand in the role's own branch: with its result
// merged across branches (or with lane == 0 instead) every one of these
// instructions took 70 cycles or more, against 10 to 20, and a stage 850 cycles
// instead of what its bytes take.
constexpr int kEpiWarps4 = 8;          // two for each quarter of the TMEM lanes
constexpr int kThreads4 = 64 + 32 * kEpiWarps4;
constexpr int kMaxStages = 12;
constexpr int kSfCols = 24;             // TMEM columns of a stage's scales: features 2 x 4, rows 2 x 8
constexpr int kWBytes = 128 * 128;      // weights of a stage
constexpr int kTables4 = 8704;          // static shared memory: the experts' rows and units, barriers
constexpr int kSmem4 = 232448 - kTables4;  // the rest of what a block may have: ring and staging
constexpr int kStage4 = 1024;           // staging of an epilogue warp: 16 rows x 32 features of 16 bits

// Shared-memory descriptors as their low words (address in units of 16 bytes and
// the leading offset, so that adding moves the address); the high words are
// constants: 128-byte swizzle with 1024 bytes between 8-row groups, or none with 128.
constexpr uint32_t kDescSw128 = (1024 >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescPlain = (128 >> 4) | (1u << 14);
MOE_DEV uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }

// The following do nothing in lanes where `on` is 0.
// D (+)= (A * sfa) (B * sfb): E2M1 operands, a UE8M0 scale per 32 elements, K = 64.
template <bool PAIR>
MOE_DEV void tc_mma_mxf4(int on, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                         uint32_t accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %8, 0;\n\t"
        "mov.b64 a, {%1, %7};\n\t"
        "mov.b64 b, {%2, %7};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescSw128), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.ne.b32 q, %8, 0;\n\t"
        "mov.b64 a, {%1, %7};\n\t"
        "mov.b64 b, {%2, %7};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescSw128), "r"(on)
        : "memory");
  }
}
// A 512-byte scale tile into four TMEM columns (its 32 rows of 16 bytes in every lane quarter).
// Of a pair: in each CTA, from its own shared memory into its own TMEM.
template <bool PAIR>
MOE_DEV void tc_cp_scales(int on, uint32_t taddr, uint32_t lo) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b64 s;\n\t"
        "setp.ne.b32 q, %3, 0;\n\t"
        "mov.b64 s, {%1, %2};\n\t"
        "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], s;\n\t}" ::"r"(taddr), "r"(lo), "n"(kDescPlain), "r"(on)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b64 s;\n\t"
        "setp.ne.b32 q, %3, 0;\n\t"
        "mov.b64 s, {%1, %2};\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], s;\n\t}" ::"r"(taddr), "r"(lo), "n"(kDescPlain), "r"(on)
        : "memory");
}
// One arrival on the barrier (of a pair: at this place in each CTA of mask) when what
// was issued so far has completed.
template <bool PAIR>
MOE_DEV void tc_commit_on(int on, uint32_t bar, uint16_t mask = 3) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::
            "r"(bar),
        "r"(on), "h"(mask)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(on)
        : "memory");
}
MOE_DEV void expect_tx_on(int on, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(on)
      : "memory");
}
// (Of a pair: `bar` may be the other CTA's, by its shared::cluster address.)
template <bool PAIR>
MOE_DEV void tma_load_2d_on(int on, uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(on)
        : "memory");
  }
}
template <bool PAIR>
MOE_DEV void tma_load_3d_on(int on, uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(on)
        : "memory");
  }
}
MOE_DEV void bulk_load_on(int on, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "r"(on)
      : "memory");
}
MOE_DEV bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The rest of a wait whose first try failed: gives up (false) on the abort flag
// or after kWaitLimitNs, which it reports.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, int where) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        report_status(status, kStatusTimeout, where);
        return false;
      }
    }
  }
}
// Instruction descriptor: E2M1 A and B (K-major), UE8M0 scales taken from bytes
// sf, sf + 1 of a 32-bit scale column (sf 0 or 2).
MOE_DEV uint32_t idesc_mxf4(int M, int N, int sf) {
  return ((uint32_t)sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf << 29);
}

// One lane of a converged warp.
MOE_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// A value that is the same in every lane, as one the compiler knows to be: a
// warp reduction's result is warp-uniform (a shuffle's is not).
MOE_DEV int uniform(int v) { return (int)__reduce_max_sync(0xffffffffu, (unsigned)v); }

struct P4 {
  const int* off;      // [G+1] or NULL (one segment of `rows`)
  const uint8_t* xs;
  const uint8_t* ws;
  void* out;
  int64_t ldo;
  int* status;
  int rows, G, N, K, NT, KT, stages_k;
  int n_units;  // units along the features: NT, of a pair half as many
};

// SiLU in the epilogue.  For results of 16 bits the layer's own: its hardware
// exponential and reciprocal are off by less than 2^-18, a hundredth of a rounding to
// bf16 or fp16.  For fp32 results accurate to fp32, from exp(-|g|), which cannot
// overflow (exp(-g) would below -88, where the result has not vanished yet).  The
// quotient n / d, d in [1, 2], is one from the hardware reciprocal with its residual's
// added, one Newton step (64 experts' 256 rows of 2048 x 1536: 42 us, 57 with the IEEE
// division, 39 with silu_f).
template <typename T>
MOE_DEV float silu_for(float g) {
  if constexpr (sizeof(T) == 4) {
    const float t = expf(-fabsf(g)), n = g < 0.f ? g * t : g, d = 1.0f + t;
    const float r = __fdividef(1.0f, d), q = n * r;
    return fabsf(q) < INFINITY ? fmaf(fmaf(-q, d, n), r, q) : q;
  } else {
    return silu_f(g);
  }
}

struct Unit4 {
  int e, n, row0, first, nt;  // expert, feature tile, first row of the expert, first row in it, rows
};

// PAIR: two CTAs (a cluster) share each MMA of M = 256 features, 128 in each, and
// each holds half of the rows, so that an SM takes in 28 KB a stage for 128 x 192
// products instead of 40.  The even CTA's barriers count both CTAs' copies, its one
// thread issues for both, and its commits arrive in both.
// tm_x128: rows in boxes of 128; of a pair the scale tiles of the rows, and tm_ws of
// the weights, as rows of 256 bytes (a plain bulk copy cannot arrive on the other
// CTA's barrier).
template <typename T, bool SWIGLU, bool PAIR>
__global__ void __launch_bounds__(kThreads4, 1)
    product_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x128,
                   const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_ws, const P4 p) {
  extern __shared__ uint8_t smem_raw[];
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  __shared__ int s_off[kMaxE + 1];    // first row of each expert
  __shared__ int s_unit[kMaxE + 1];   // first unit of each expert
  __shared__ alignas(8) uint64_t full[kMaxStages], empty[kMaxStages], tfull[2], tempty[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_most;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], (PAIR ? 2 : 1) * kEpiWarps4);
    }
    mbar_init(&drain, 1);
    s_abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_x128);
    tma_prefetch_desc(&tm_w);
    if (PAIR) tma_prefetch_desc(&tm_ws);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(&s_tmem), 512);  // both CTAs, collectively
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(&s_tmem), 512);
      tmem_relinquish();
    }
  }
  ops_wait();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;

  // experts' rows and units
  // (offsets out of order or range give wrong rows, not accesses out of range)
  for (int i = threadIdx.x; i <= p.G; i += blockDim.x) s_off[i] = p.off ? min(max(gload(p.off + i), 0), p.rows) : (i ? p.rows : 0);
  __syncthreads();
  if (warp == 0) {
    int run = 0, most = 0;
    for (int base = 0; base < p.G; base += 32) {
      const int e = base + lane;
      const int c = e < p.G ? max(0, s_off[e + 1] - s_off[e]) : 0;
      const int tt = tok_tiles(c);
      most = max(most, tok_most(c));
      int inc = tt * p.n_units;
      const int mine = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (e < p.G) s_unit[e] = run + inc - mine;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      s_unit[p.G] = run;
      s_most = most;
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the other CTA's barriers exist before their use
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem);
  const int total = uniform(s_unit[p.G]);
  volatile int* abort_flag = &s_abort;

  // stage layout for the largest tile there is: weights, rows, scales
  const int cap = uniform((s_most + 31) & ~31);
  const uint32_t sfb_runs = cap > 128 ? 2 : 1;
  const int cap_x = PAIR ? (cap / 2 + 31) & ~31 : cap;  // rows in this CTA's shared memory
  const uint32_t stage_bytes = (uint32_t)kWBytes + (uint32_t)cap_x * 128u + 1024u + sfb_runs * 1024u;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t room = kSmem4 - kEpiWarps4 * kStage4 - (base - smem_u32(smem_raw));
  const uint32_t staging = base + room;  // (16-byte aligned: base and the sizes are)
  const int S = min(min(kMaxStages, (int)(room / stage_bytes)), (512 - 2 * cap) / kSfCols);

  const int rank = PAIR ? uniform((int)cluster_ctarank()) : 0;
  const int unit0 = PAIR ? blockIdx.x / 2 : blockIdx.x, unit_step = PAIR ? gridDim.x / 2 : gridDim.x;

  // Unit u; each role walks its units upwards and keeps its place in the experts.
  int at_e = 0;
  auto unit_at = [&](int u) {
    while (u >= uniform(s_unit[at_e + 1])) ++at_e;
    Unit4 t;
    t.e = at_e;
    t.row0 = uniform(s_off[at_e]);
    const int c = uniform(s_off[at_e + 1]) - t.row0, tt = tok_tiles(c), r = u - uniform(s_unit[at_e]);
    const int n = tt == 1 ? r : r / tt, i = r - n * tt;
    t.n = PAIR ? 2 * n + rank : n;
    t.first = tt == 1 ? 0 : tok_start(c, tt, i);
    t.nt = (i + 1 < tt ? tok_start(c, tt, i + 1) : c) - t.first;
    return t;
  };

  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
  // All lanes wait; the result is the same in each.
  auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
    if (__all_sync(0xffffffffu, try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity, abort_flag, p.status, where)) != 0;
  };
  if (warp == 0) {
    const int leader = elect_one();
    int s = 0;
    uint32_t ph = 0, used = 0, last = 0;
    for (int u = unit0; u < total; u += unit_step) {
      const Unit4 t = unit_at(u);
      const int runs = ((t.first & 127) + t.nt + 127) / 128;
      // this CTA's rows: all, or its half of the MMA's N; in boxes of 128 (one CTA), the rest of 32
      const int mine = PAIR ? ((t.nt + 31) & ~31) / 2 : t.nt;
      const int boxes = (mine + 31) / 32;
      const int row = t.row0 + t.first + (PAIR ? rank * mine : 0);
      const int big = !PAIR && leader && boxes >= 4, small0 = !PAIR && boxes >= 4 ? 4 : 0;
      const size_t wrun = (size_t)t.e * p.NT + t.n, xrun = (size_t)(t.row0 / 128 + t.e + t.first / 128);
      const uint8_t* wsp = p.ws + wrun * p.KT * 512u;
      const uint8_t* xsp = p.xs + xrun * p.KT * 512u;
      const uint8_t* xsp2 = xsp + (size_t)p.KT * 512u;
      const uint32_t bytes = (uint32_t)kWBytes + (uint32_t)boxes * 4096u;
      for (int kb = 0; kb < p.stages_k; ++kb) {
        if (!wait_all(empty0 + 8u * s, ph ^ 1u, 1000 + s)) goto produced;
        const uint32_t sa = base + (uint32_t)s * stage_bytes, sb = sa + kWBytes, sf = sb + (uint32_t)cap_x * 128u;
        if constexpr (PAIR) {
          const uint32_t fb = mapa_shared(full0 + 8u * s, 0);
          expect_tx_on(leader && rank == 0, full0 + 8u * s, 2u * (bytes + 1024u * (1u + runs)));
          tma_load_3d_on<true>(leader, sa, &tm_w, fb, kb * 128, t.n * 128, t.e);
          for (int i = 0; i < boxes; ++i) tma_load_2d_on<true>(leader, sb + i * 4096u, &tm_x, fb, kb * 128, row + i * 32);
          tma_load_2d_on<true>(leader, sf, &tm_ws, fb, 0, (int)(wrun * p.KT * 2) + kb * 4);
          tma_load_2d_on<true>(leader, sf + 1024u, &tm_x128, fb, 0, (int)(xrun * p.KT * 2) + kb * 4);
          tma_load_2d_on<true>(leader && runs > 1, sf + 2048u, &tm_x128, fb, 0, (int)((xrun + 1) * p.KT * 2) + kb * 4);
        } else {
          const uint32_t fb = full0 + 8u * s;
          const uint32_t sfn = 512u * (uint32_t)min(2, p.KT - 2 * kb);
          expect_tx_on(leader, fb, bytes + sfn * (1u + runs));
          tma_load_3d_on<false>(leader, sa, &tm_w, fb, kb * 128, t.n * 128, t.e);
          bulk_load_on(leader, sf, wsp, sfn, fb);
          tma_load_2d_on<false>(big, sb, &tm_x128, fb, kb * 128, row);
          for (int i = small0; i < boxes; ++i) tma_load_2d_on<false>(leader, sb + i * 4096u, &tm_x, fb, kb * 128, row + i * 32);
          bulk_load_on(leader, sf + 1024u, xsp, sfn, fb);
          bulk_load_on(leader && runs > 1, sf + 2048u, xsp2, sfn, fb);
          wsp += 1024;
          xsp += 1024;
          xsp2 += 1024;
        }
        used |= 1u << s;
        last = (last & ~(1u << s)) | (ph << s);
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  produced:
    // every issued copy has landed before the CTA can exit (of a pair the even CTA's
    // barriers count both CTAs'), and of a pair every commit has arrived
    for (int i = 0; i < kMaxStages; ++i) {
      if (((used >> i) & 1u) == 0) continue;
      if (rank == 0 && !mbar_wait_drain(&full[i], (last >> i) & 1u)) break;
      if (PAIR && !mbar_wait_drain(&empty[i], (last >> i) & 1u)) break;
    }
  } else if (warp == 1 && rank == 0) {
    const int leader = elect_one();
    int s = 0, acc = 0;
    uint32_t ph = 0, aph = 0;
    const uint32_t da0 = desc_lo(base), step = stage_bytes / 16u, sf0 = tmem + 2u * (uint32_t)cap;
    const uint32_t b_off = kWBytes / 16u, s_off16 = b_off + (uint32_t)cap_x * 8u;
    for (int u = unit0; u < total; u += unit_step) {
      const Unit4 t = unit_at(u);
      const int mma_n = PAIR ? (t.nt + 31) & ~31 : (t.nt + 15) & ~15;
      const int two = leader && (t.first & 127) + t.nt > 128;
      const uint32_t shift = 8u + (uint32_t)(t.first & 127) / 32u;  // scale columns of the rows: 0 or 2 in
      const uint32_t id0 = idesc_mxf4(PAIR ? 256 : 128, mma_n, 0), id2 = idesc_mxf4(PAIR ? 256 : 128, mma_n, 2);
      const uint32_t d = tmem + (uint32_t)(acc * cap);
      if (!wait_all(smem_u32(&tempty[acc]), aph ^ 1u, 1100 + acc)) goto issued;
      tc_fence_after();
      int left = p.K;  // elements of K still to come
      uint32_t more = 0;
      for (int kb = 0; kb < p.stages_k; ++kb) {
        if (!wait_all(full0 + 8u * s, ph, 1200 + s)) goto issued;
        tc_fence_after();
        // descriptors advance in units of 16 bytes
        const uint32_t da = da0 + (uint32_t)s * step, db = da + b_off, ds = da + s_off16;
        const uint32_t tsf = sf0 + (uint32_t)s * kSfCols, tsb = tsf + shift;
        const int half = leader && left > 128;
        tc_cp_scales<PAIR>(leader, tsf, ds);
        tc_cp_scales<PAIR>(leader, tsf + 8u, ds + 64u);
        tc_cp_scales<PAIR>(two, tsf + 12u, ds + 128u);
        tc_cp_scales<PAIR>(half, tsf + 4u, ds + 32u);
        tc_cp_scales<PAIR>(half, tsf + 16u, ds + 96u);
        tc_cp_scales<PAIR>(two && half, tsf + 20u, ds + 160u);
        tc_mma_mxf4<PAIR>(leader, d, da, db, id0, tsf, tsb, more);
        tc_mma_mxf4<PAIR>(leader && left > 64, d, da + 2u, db + 2u, id2, tsf, tsb, 1u);
        tc_mma_mxf4<PAIR>(half, d, da + 4u, db + 4u, id0, tsf + 4u, tsb + 8u, 1u);
        tc_mma_mxf4<PAIR>(leader && left > 192, d, da + 6u, db + 6u, id2, tsf + 4u, tsb + 8u, 1u);
        tc_commit_on<PAIR>(leader, empty0 + 8u * s);
        left -= 256;
        more = 1u;
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
      tc_commit_on<PAIR>(leader, smem_u32(&tfull[acc]));
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
  issued:
    tc_commit_on<PAIR>(leader, smem_u32(&drain), 1);
    mbar_wait_drain(&drain, 0);
  } else if (warp > 1) {
    // A warp takes every other 32 rows of its quarter's 32 features.  A lane holds one
    // feature: results of 16 bits go through the warp's staging, 16 rows at a time, and
    // leave as 16-byte stores.  Output rows that are not 16-byte aligned, features
    // past N and fp32 results are stored from the lanes (64 experts' 256 rows of 2048 x
    // 1536: 45 us, 47 with rows of an odd stride, 47 in fp32; 8 experts' 2048 rows of
    // 7168 x 4096: 150, 156, 164).
    const int q = warp & 3;  // TMEM lane quarter of this warp
    const uint32_t stg = staging + (uint32_t)(warp - 2) * kStage4;
    constexpr int kCols = SWIGLU ? 16 : 32;  // output columns of 32 features
    int acc = 0;
    uint32_t aph = 0;
    T* out = static_cast<T*>(p.out);
    const bool rows16 = sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(out) & 15) == 0 && p.ldo % 8 == 0;
    for (int u = unit0; u < total; u += unit_step) {
      const Unit4 t = unit_at(u);
      if (!wait_all(smem_u32(&tfull[acc]), aph, 1400 + acc)) break;
      tc_fence_after();
      const int n0 = t.n * 128 + q * 32, n = n0 + lane;
      T* dst = out + (int64_t)(t.row0 + t.first) * p.ldo + (SWIGLU ? n0 >> 1 : n0);
      const bool odd = lane & 1;
      for (int c0 = 32 * ((warp - 2) >> 2); c0 < t.nt; c0 += 64) {
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * cap + c0), v);
        if (SWIGLU) {
          // even lanes hold gates, odd lanes the matching up products: of each
          // pair of rows an even lane finishes the first (left in v[c]), an odd
          // lane the second (left in v[c] too).  The choice comes before silu: after
          // it both sides are computed (fp32 results: 68 us, not 42)
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float y = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
            const float up = odd ? v[c + 1] : y;
            v[c] = silu_for<T>(odd ? y : v[c]) * up;
          }
        }
        if (rows16 && n0 + 32 <= p.N) {
          if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
#pragma unroll
              for (int c = 0; c < 16; c += SWIGLU ? 2 : 1) {
                const T r = from_f32<T>(v[h + c]);
                const uint32_t at = SWIGLU ? stg + c * kCols * 2 + lane * 2 + (odd ? kCols * 2 - 2 - (lane >> 1) * 2 : -(lane >> 1) * 2)
                                           : stg + c * kCols * 2 + lane * 2;
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<const uint16_t*>(&r)) : "memory");
              }
              __syncwarp();
              constexpr int kLanes = kCols / 8;  // lanes of a row
#pragma unroll
              for (int i = 0; i < 16 * kLanes / 32; ++i) {
                const int row = i * (32 / kLanes) + lane / kLanes, col = lane % kLanes * 8;
                uint4 w;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                             : "r"(stg + (uint32_t)(row * kCols + col) * 2u));
                if (c0 + h + row < t.nt) *reinterpret_cast<uint4*>(dst + (int64_t)(c0 + h + row) * p.ldo + col) = w;
              }
              __syncwarp();
            }
          }
        } else if (n < p.N) {
#pragma unroll
          for (int c = 0; c < 32; c += SWIGLU ? 2 : 1) {
            const int row = c0 + c + (SWIGLU && odd ? 1 : 0);
            if (row < t.nt) dst[(int64_t)row * p.ldo + (SWIGLU ? lane >> 1 : lane)] = from_f32<T>(v[c]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
        else mbar_arrive(&tempty[acc]);
      }
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
  }
  ops_let_next();
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the pair's MMAs and remote arrivals are done
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

int grid_for(int64_t n) {
  const int64_t b = (n + 255) / 256;
  return (int)(b < 1 ? 1 : b < (1 << 20) ? b : (1 << 20));
}
// Clusters of two CTAs of kern that the GPU holds at once.  resident: the answer for
// each device (0: not asked yet), kept by the caller for its kernel; threads that ask
// at the same time store the same value.
template <typename K>
int pair_clusters(K kern, const cudaLaunchConfig_t& cfg, std::atomic<int> (&resident)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int n = resident[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = num_sms() / 2;
    resident[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <typename T, bool SWIGLU, bool PAIR>
cudaError_t launch_product(const CUtensorMap* tm, const P4& p, cudaStream_t st) {
  auto kern = product_kernel<T, SWIGLU, PAIR>;
  const int smem = kSmem4;
  static SmemAllowed allowed;
  const cudaError_t e = allow_smem(kern, smem, allowed);
  if (e != cudaSuccess) return e;
  // units: at most n_units for every expert with a row and every 192 rows
  const int64_t units = (int64_t)p.n_units * ((int64_t)p.rows / kMaxTok + (p.G < p.rows ? p.G : p.rows));
  if constexpr (!PAIR) {
    const int grid = units < num_sms() ? (int)units : num_sms();
    return launch_ops("mxfp4_product", kern, dim3(grid), dim3(kThreads4), smem, st, tm[0], tm[1], tm[2], tm[3], p);
  } else {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms() & ~1));
    cfg.blockDim = dim3(kThreads4);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<int> resident[64];
    const int most = pair_clusters(kern, cfg, resident);
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(2 * (unsigned)(units < most ? units : most));
    TraceScope ts("mxfp4_product", st);
    return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], p);
  }
}

// Whether the product runs on CTA pairs: where it is bound by what the SMs take in,
// that is experts with many rows, and K long enough that the pairs' hand-overs between
// units do not cost more.  us, one CTA / pairs: 2048 rows an expert (8 experts, N =
// 4096) K = 7168: 174 / 151, 4096: 109 / 97, 2048: 70 / 73; K = 7168, 512 rows (32):
// 197 / 174, 204 (80): 299 / 273, 128 (256): 641 / 643.
bool product_pairs(int64_t rows, int G, int K, int NT) { return NT > 1 && K >= 4096 && rows >= 160 * (int64_t)G; }

bool fp4_k(int32_t K) { return K >= 32 && K % 32 == 0 && K <= (1 << 24); }
bool fp4_weights(int64_t batch, int32_t K, int32_t N) {
  return batch >= 0 && batch <= (1 << 20) && fp4_k(K) && N >= 1 && N <= (1 << 22);
}
bool fp4_rows(int64_t rows, int32_t K, int32_t G) {
  return rows >= 0 && rows <= ((int64_t)1 << 28) && fp4_k(K) && G >= 1 && G <= kMaxE;
}
// The status of a call that launches no kernel.  (A ws that is not the device's memory
// -- there may be no device -- has none to clear.)
moe_status clear_status(void* ws, cudaStream_t st) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, ws) != cudaSuccess) {
    cudaGetLastError();
    return MOE_OK;
  }
  if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) return MOE_OK;
  return ops_status(cudaMemsetAsync(ws, 0, 2 * sizeof(int), st));
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
  return (size_t)(rows / 128 + G) * ((K + 127) / 128) * 512;
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
    auto kern = rows16(x, ldx, dtype) ? quant_rows_kernel<T, true> : quant_rows_kernel<T, false>;
    const int nb = (K + 127) / 128 * 4, rpb = nb < 64 ? 128 / nb : 1;
    const int threads = nb > 256 ? 256 : (nb * rpb + 31) / 32 * 32;
    return launch_ops("quantize_mxfp4_rows", kern, dim3((unsigned)((rows + rpb - 1) / rpb), (nb + 255) / 256),
                      dim3(threads), 0, st, static_cast<const T*>(x), ldx, (int)rows, K, G, offsets, perm, k, rpb, q,
                      scales);
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
    const Segs sg = row_segs(K);
    const unsigned grid = (unsigned)((rows * sg.n + 7) / 8);
    auto kern = rows16(y, ldy, dtype) ? dequant_rows_kernel<T, true> : dequant_rows_kernel<T, false>;
    return launch_ops("dequantize_mxfp4_rows", kern, dim3(grid), dim3(256), 0, st, q, scales, rows, K, G, offsets, sg.n,
                      sg.per, static_cast<T*>(y), ldy);
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
  if (rows == 0) return clear_status(ws, reinterpret_cast<cudaStream_t>(stream));
  if (!aligned128(xq) || !aligned128(xscales) || !aligned128(wq) || !aligned128(wscales) ||
      !elem_ok(out, dtype_bytes(dtype)) || !elem_ok_or_null(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int NT = (N + 127) / 128, KT = (K + 127) / 128;
  const bool pair = product_pairs(rows, G, K, NT);
  CUtensorMap tm[4];
  bool ok = map2d(&tm[0], xq, (uint64_t)K / 2, (uint64_t)rows, 128, 32, true) &&
            map3d(&tm[2], wq, (uint64_t)K / 2, (uint64_t)N, (uint64_t)G, 128, 128, true);
  if (pair) {
    ok = ok && map2d(&tm[1], xscales, 256, (uint64_t)(rows / 128 + G) * KT * 2, 256, 4, true, CU_TENSOR_MAP_SWIZZLE_NONE) &&
         map2d(&tm[3], wscales, 256, (uint64_t)G * NT * KT * 2, 256, 4, true, CU_TENSOR_MAP_SWIZZLE_NONE);
  } else {
    ok = ok && map2d(&tm[1], xq, (uint64_t)K / 2, (uint64_t)rows, 128, 128, true);
    tm[3] = tm[1];
  }
  if (!ok) return MOE_ERR_CUDA;
  P4 p;
  p.off = offsets;
  p.xs = xscales;
  p.ws = wscales;
  p.out = out;
  p.ldo = ldo;
  p.status = static_cast<int*>(ws);
  p.rows = (int)rows;
  p.G = G;
  p.N = N;
  p.K = K;
  p.NT = NT;
  p.KT = KT;
  p.n_units = pair ? (NT + 1) / 2 : NT;
  p.stages_k = (K + 255) / 256;
  return ops_status(with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (act == MOE_ACT_SWIGLU)
      return pair ? launch_product<T, true, true>(tm, p, st) : launch_product<T, true, false>(tm, p, st);
    return pair ? launch_product<T, false, true>(tm, p, st) : launch_product<T, false, false>(tm, p, st);
  }));
}

}  // extern "C"

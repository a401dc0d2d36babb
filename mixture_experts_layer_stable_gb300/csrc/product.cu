// product.cu -- products of rows with their expert's weights and the weights'
// gradients (include/moe_ops.h, moe_grouped_product, moe_grouped_product_dw).
//
//   out[p] = x[p] * w[g]      p in [offsets[g], offsets[g + 1])
//   dw[g]  = sum over g's rows p of x[p]^T * dy[p]
//
// All three forms are D = A * B per expert: A is the expert's rows (or their transpose),
// B its weights (or rows), and the work is cut into units (expert, tile of D) that each
// block numbers by itself from the offsets, so no call looks at them on the host.
#include "product.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ fp32 units
// fp32 operands of any alignment: square tiles of B by 2 B threads, 8 x B / 16 results a
// thread, 16 of the contraction at a time through shared memory, the next 16 on their way
// in registers.
constexpr int kSimtK = 16;

// A tile of C x kSimtK elements on its way to 2 C threads: C columns of D's side, MN: they
// are the contiguous ones in memory (else the contraction is).
template <int C, bool MN, bool VEC>
struct SimtTile {
  static constexpr int kSimtThreads = 2 * C;
  static constexpr int V = VEC ? 4 : 1;
  static constexpr int kVecs = C * kSimtK / V;
  static constexpr int N = (kVecs + kSimtThreads - 1) / kSimtThreads;
  Words<float, V == 1 ? 2 : V> w[V == 1 ? 1 : N];
  float f[V == 1 ? N : 1];

  // place of vector i of this thread: column c of the tile, contraction k
  __device__ __forceinline__ static void place(int i, int& c, int& k) {
    const int v = i * kSimtThreads + threadIdx.x;
    if constexpr (MN) {
      c = v % (C / V) * V;
      k = v / (C / V);
    } else {
      k = v % (kSimtK / V) * V;
      c = v / (kSimtK / V);
    }
  }
  // columns [0, cn) and contraction [0, kn) exist
  __device__ __forceinline__ void load(const float* base, int64_t ld, int cn, int kn) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int c, k;
      place(i, c, k);
      const bool there = c < cn && k < kn && (kVecs % kSimtThreads == 0 || i * kSimtThreads + (int)threadIdx.x < kVecs);
      const float* p = MN ? base + k * ld + c : base + c * ld + k;
      if constexpr (V == 1) {
        f[i] = there ? gload(p) : 0.f;
      } else {
        if (there) w[i].template load<V>(0, p);
        else w[i].clear();
      }
    }
  }
  __device__ __forceinline__ void store(float (*sh)[C + 4]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int c, k;
      place(i, c, k);
      if (kVecs % kSimtThreads != 0 && i * kSimtThreads + (int)threadIdx.x >= kVecs) continue;
      if constexpr (V == 1) {
        sh[k][c] = f[i];
      } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 e = w[i].pair(j).get();
          if constexpr (MN) {
            *reinterpret_cast<float2*>(&sh[k][c + 2 * j]) = e;
          } else {
            sh[k + 2 * j][c] = e.x;
            sh[k + 2 * j + 1][c] = e.y;
          }
        }
      }
    }
  }
};

// A_MN / B_MN: whether the columns of D's side (not the contraction) are contiguous in A /
// B.  The forward has (false, true), with transposed weights (false, false), the weights'
// gradient (true, true): there the contraction is over the expert's rows.
template <bool A_MN, bool B_MN, bool VEC, int B>
__global__ void __launch_bounds__(2 * B, B == 64 ? 5 : 2) simt_product_kernel(const ProdArgs p) {
  constexpr bool DW = A_MN;
  constexpr int C = B / 64;  // quads of D's columns that a thread has
  __shared__ int s_off[kMaxG + 1], s_unit[kMaxG + 1];
  __shared__ __align__(16) float sa[2][kSimtK][B + 4], sb[2][kSimtK][B + 4];
  ops_begin();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  const int nt = (p.N + B - 1) / B;
  const int mt_dw = (p.K + B - 1) / B;
  number_units(p, DW ? 0 : B, DW ? mt_dw * nt : nt, s_off, s_unit);
  const int total = s_unit[p.G];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const float *A = static_cast<const float*>(p.a), *W = static_cast<const float*>(p.b);
  float* out = static_cast<float*>(p.out);
  int e = 0;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    while (u >= s_unit[e + 1]) ++e;
    const int row0 = s_off[e], count = max(0, s_off[e + 1] - row0);
    const int mts = DW ? mt_dw : (count + B - 1) / B;
    const int r = u - s_unit[e], n0 = r / mts * B, m0 = (r - r / mts * mts) * B;
    const int M = DW ? p.K : count, kk = DW ? count : p.K;
    // tile bases: A[m0.., k], B[k, n0..]
    const float* a = DW ? A + (int64_t)row0 * p.lda + m0 : A + (int64_t)(row0 + m0) * p.lda;
    const float* b = DW ? W + (int64_t)row0 * p.ldb + n0
                    : W + (int64_t)e * p.K * p.N + (B_MN ? (int64_t)n0 : (int64_t)n0 * p.ldb);
    const int64_t ak = A_MN ? kSimtK * p.lda : kSimtK, bk = B_MN ? kSimtK * p.ldb : kSimtK;
    SimtTile<B, A_MN, VEC> ta;
    SimtTile<B, B_MN, VEC> tb;
    F2 acc[8][2 * C];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2 * C; ++j) acc[i][j] = F2(0.f, 0.f);
    const int steps = (kk + kSimtK - 1) / kSimtK;
    if (steps > 0) {
      ta.load(a, p.lda, M - m0, kk);
      tb.load(b, p.ldb, p.N - n0, kk);
      ta.store(sa[0]);
      tb.store(sb[0]);
    }
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
      const bool more = s + 1 < steps;
      if (more) {
        ta.load(a + (s + 1) * ak, p.lda, M - m0, kk - (s + 1) * kSimtK);
        tb.load(b + (s + 1) * bk, p.ldb, p.N - n0, kk - (s + 1) * kSimtK);
      }
      const float(*ca)[B + 4] = sa[s & 1];
      const float(*cb)[B + 4] = sb[s & 1];
#pragma unroll
      for (int k = 0; k < kSimtK; ++k) {
        float av[8];
        F2 bv[2 * C];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(&ca[k][i * (B / 2) + ty * 4]);
          av[4 * i] = v.x;
          av[4 * i + 1] = v.y;
          av[4 * i + 2] = v.z;
          av[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(&cb[k][j * 64 + tx * 4]);
          bv[2 * j] = F2(v.x, v.y);
          bv[2 * j + 1] = F2(v.z, v.w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const F2 a2(av[i], av[i]);
#pragma unroll
          for (int j = 0; j < 2 * C; ++j) acc[i][j] = fma2(a2, bv[j], acc[i][j]);
        }
      }
      if (more) {
        ta.store(sa[(s + 1) & 1]);
        tb.store(sb[(s + 1) & 1]);
      }
      __syncthreads();
    }
    float* d = DW ? out + (int64_t)e * p.K * p.N : out + (int64_t)row0 * p.ldo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = m0 + i / 4 * (B / 2) + ty * 4 + i % 4;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 2 * C; ++j) {
        const int n = n0 + j / 2 * 64 + tx * 4 + j % 2 * 2;
        float2 v = acc[i][j].get();
        float* q = d + (int64_t)m * p.ldo + n;
        if (DW && p.accumulate) {
          if (n < p.N) v.x += q[0];
          if (n + 1 < p.N) v.y += q[1];
        }
        if (n < p.N) q[0] = v.x;
        if (n + 1 < p.N) q[1] = v.y;
      }
    }
  }
}

// ------------------------------------------------------------------ host side
// (No array has more than 2^40 elements, so units are numbered in 32 bits.)
bool prod_sizes(int64_t rows, int32_t K, int32_t N, int32_t G) {
  constexpr int64_t most = (int64_t)1 << 40;
  return rows >= 0 && rows <= ((int64_t)1 << 28) && K >= 1 && K <= (1 << 22) && N >= 1 && N <= (1 << 22) && G >= 1 &&
         G <= kMaxG && (int64_t)K * N <= most / G && rows <= most / (K > N ? K : N);
}

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

template <bool A_MN, bool B_MN>
cudaError_t launch_simt(const ProdArgs& p, cudaStream_t st) {
  // vectors: every row starts on 16 bytes and is a whole number of them (a vector at the
  // end of a row would pass the array's)
  const uintptr_t es = 4, a_row = (uintptr_t)p.K * es, b_row = (uintptr_t)(B_MN ? p.N : p.K) * es;
  const bool vec = ((bits(p.a) | bits(p.b) | (uintptr_t)p.lda * es | (uintptr_t)p.ldb * es | a_row | b_row) & 15) == 0;
  // tiles of 128 where they fill the GPU twice, else of 64
  const int64_t nt = (p.N + 127) / 128, units = A_MN ? nt * ((p.K + 127) / 128) * p.G : nt * (p.rows / 128 + 1);
  const char* name = A_MN ? "grouped_product_dw" : "grouped_product";
  auto go = [&](auto size, int per_sm) {
    constexpr int B = decltype(size)::value;
    auto kern = vec ? simt_product_kernel<A_MN, B_MN, true, B> : simt_product_kernel<A_MN, B_MN, false, B>;
    return launch_ops(name, kern, dim3(per_sm * num_sms()), dim3(2 * B), 0, st, p);
  };
  if (units >= 2 * num_sms()) return go(std::integral_constant<int, 128>(), 2);
  return go(std::integral_constant<int, 64>(), 5);
}

cudaError_t launch_product(ProdForm form, int dtype, const ProdArgs& p, cudaStream_t st) {
  if (dtype != MOE_DT_F32) return launch_product_tc(form, dtype, p, st);
  switch (form) {
    case PROD_ROWS: return launch_simt<false, true>(p, st);
    case PROD_ROWS_T: return launch_simt<false, false>(p, st);
    default: return launch_simt<true, true>(p, st);
  }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_product_workspace_bytes(int64_t rows, int32_t K, int32_t N, int32_t G) {
  if (!prod_sizes(rows, K, N, G)) return 0;
  return 128;
}

moe_status moe_grouped_product(int32_t dtype, int32_t odtype, int64_t rows, int32_t K, int32_t N, int32_t G,
                               const int32_t* offsets, const void* x, int64_t ldx, const void* w, int32_t transposed,
                               void* out, int64_t ldo, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_valid(dtype) || (odtype != dtype && odtype != MOE_DT_F32) || !prod_sizes(rows, K, N, G) || ldx < K ||
      ldo < N || (offsets == nullptr && G != 1) || ws == nullptr || !aligned_to(ws, 128))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_grouped_product_workspace_bytes(rows, K, N, G)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) return clear_status(ws, st);
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(x, es) || !elem_ok(w, es) || !elem_ok(out, dtype_bytes(odtype)) || !elem_ok_or_null(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  ProdArgs p = {};
  p.off = offsets;
  p.a = x;
  p.b = w;
  p.out = out;
  p.lda = ldx;
  p.ldb = transposed ? K : N;
  p.ldo = ldo;
  p.status = static_cast<int*>(ws);
  p.rows = (int)rows;
  p.G = G;
  p.K = K;
  p.N = N;
  p.odt = odtype;
  return ops_status(launch_product(transposed ? PROD_ROWS_T : PROD_ROWS, dtype, p, st));
}

moe_status moe_grouped_product_dw(int32_t dtype, int32_t wdtype, int64_t rows, int32_t K, int32_t N, int32_t G,
                                  const int32_t* offsets, const void* x, int64_t ldx, const void* dy, int64_t lddy,
                                  void* dw, int32_t accumulate, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_valid(dtype) || (wdtype != dtype && wdtype != MOE_DT_F32) || !prod_sizes(rows, K, N, G) || ldx < K ||
      lddy < N || (offsets == nullptr && G != 1) || ws == nullptr || !aligned_to(ws, 128))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_grouped_product_workspace_bytes(rows, K, N, G)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(dw, dtype_bytes(wdtype)) ||
      (rows > 0 && (!elem_ok(x, es) || !elem_ok(dy, es) || !elem_ok_or_null(offsets, 4))))
    return MOE_ERR_INVALID_ARG;
  ProdArgs p = {};
  p.off = rows > 0 ? offsets : nullptr;
  p.a = x;
  p.b = dy;
  p.out = dw;
  p.lda = ldx;
  p.ldb = lddy;
  p.ldo = N;
  p.status = static_cast<int*>(ws);
  p.rows = (int)rows;
  p.G = G;
  p.K = K;
  p.N = N;
  p.odt = wdtype;
  p.accumulate = accumulate != 0;
  return ops_status(launch_product(PROD_DW, dtype, p, st));
}

}  // extern "C"

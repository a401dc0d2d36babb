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
// Operands of any type and alignment: tiles of BM x 128 by 256 threads, 16 of the
// contraction at a time in fp32 through shared memory, the next 16 on their way in
// registers.
constexpr int kSimtN = 128, kSimtK = 16, kSimtThreads = 256;

// A tile of C x kSimtK elements on its way: C columns of D's side, MN: they are the
// contiguous ones in memory (else the contraction is).
template <typename T, int C, bool MN, bool VEC>
struct SimtTile {
  static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
  static constexpr int kVecs = C * kSimtK / V;
  static constexpr int N = (kVecs + kSimtThreads - 1) / kSimtThreads;
  Words<T, V == 1 ? 2 : V> w[V == 1 ? 1 : N];
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
  __device__ __forceinline__ void load(const T* base, int64_t ld, int cn, int kn) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int c, k;
      place(i, c, k);
      const bool there = c < cn && k < kn && (kVecs % kSimtThreads == 0 || i * kSimtThreads + (int)threadIdx.x < kVecs);
      const T* p = MN ? base + k * ld + c : base + c * ld + k;
      if constexpr (V == 1) {
        f[i] = there ? gload_f32(p) : 0.f;
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
template <typename T, typename O, bool A_MN, bool B_MN, bool VEC, int BM>
__global__ void __launch_bounds__(kSimtThreads) simt_product_kernel(const ProdArgs p) {
  constexpr bool DW = A_MN;
  constexpr int R = BM / 64;  // quads of D's rows that a thread has
  __shared__ int s_off[kMaxG + 1], s_unit[kMaxG + 1];
  __shared__ __align__(16) float sa[2][kSimtK][BM + 4], sb[2][kSimtK][kSimtN + 4];
  ops_begin();
  if (blockIdx.x == 0 && threadIdx.x < 2) p.status[threadIdx.x] = 0;
  const int nt = (p.N + kSimtN - 1) / kSimtN;
  const int mt_dw = (p.K + BM - 1) / BM;
  number_units(p, DW ? 0 : BM, DW ? mt_dw * nt : nt, s_off, s_unit);
  const int total = s_unit[p.G];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const T *A = static_cast<const T*>(p.a), *B = static_cast<const T*>(p.b);
  O* out = static_cast<O*>(p.out);
  int e = 0;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    while (u >= s_unit[e + 1]) ++e;
    const int row0 = s_off[e], count = max(0, s_off[e + 1] - row0);
    const int mts = DW ? mt_dw : (count + BM - 1) / BM;
    const int r = u - s_unit[e], n0 = r / mts * kSimtN, m0 = (r - r / mts * mts) * BM;
    const int M = DW ? p.K : count, kk = DW ? count : p.K;
    // tile bases: A[m0.., k], B[k, n0..]
    const T* a = DW ? A + (int64_t)row0 * p.lda + m0 : A + (int64_t)(row0 + m0) * p.lda;
    const T* b = DW ? B + (int64_t)row0 * p.ldb + n0
                    : B + (int64_t)e * p.K * p.N + (B_MN ? (int64_t)n0 : (int64_t)n0 * p.ldb);
    const int64_t ak = A_MN ? kSimtK * p.lda : kSimtK, bk = B_MN ? kSimtK * p.ldb : kSimtK;
    SimtTile<T, BM, A_MN, VEC> ta;
    SimtTile<T, kSimtN, B_MN, VEC> tb;
    F2 acc[4 * R][4];
#pragma unroll
    for (int i = 0; i < 4 * R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = F2(0.f, 0.f);
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
      const float(*ca)[BM + 4] = sa[s & 1];
      const float(*cb)[kSimtN + 4] = sb[s & 1];
#pragma unroll
      for (int k = 0; k < kSimtK; ++k) {
        float av[4 * R];
        F2 bv[4];
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(&ca[k][i * 64 + ty * 4]);
          av[4 * i] = v.x;
          av[4 * i + 1] = v.y;
          av[4 * i + 2] = v.z;
          av[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(&cb[k][j * 64 + tx * 4]);
          bv[2 * j] = F2(v.x, v.y);
          bv[2 * j + 1] = F2(v.z, v.w);
        }
#pragma unroll
        for (int i = 0; i < 4 * R; ++i) {
          const F2 a2(av[i], av[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fma2(a2, bv[j], acc[i][j]);
        }
      }
      if (more) {
        ta.store(sa[(s + 1) & 1]);
        tb.store(sb[(s + 1) & 1]);
      }
      __syncthreads();
    }
    O* d = DW ? out + (int64_t)e * p.K * p.N : out + (int64_t)row0 * p.ldo;
#pragma unroll
    for (int i = 0; i < 4 * R; ++i) {
      const int m = m0 + i / 4 * 64 + ty * 4 + i % 4;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + j / 2 * 64 + tx * 4 + j % 2 * 2;
        float2 v = acc[i][j].get();
        O* q = d + (int64_t)m * p.ldo + n;
        if (DW && p.accumulate) {
          if (n < p.N) v.x += to_f32(q[0]);
          if (n + 1 < p.N) v.y += to_f32(q[1]);
        }
        if (n < p.N) q[0] = from_f32<O>(v.x);
        if (n + 1 < p.N) q[1] = from_f32<O>(v.y);
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

// f(T{}, O{}) for the operands' and the results' types.
template <typename F>
cudaError_t prod_types(int dtype, int odtype, F f) {
  return with_dtype(dtype, [&](auto t) {
    if (odtype == MOE_DT_F32) return f(t, float());
    return f(t, t);
  });
}

uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

template <typename T, typename O, bool A_MN, bool B_MN>
cudaError_t launch_simt(const ProdArgs& p, cudaStream_t st) {
  // vectors: every row starts on 16 bytes and is a whole number of them (a vector at the
  // end of a row would pass the array's)
  const uintptr_t es = sizeof(T), a_row = (uintptr_t)p.K * es, b_row = (uintptr_t)(B_MN ? p.N : p.K) * es;
  const bool vec = ((bits(p.a) | bits(p.b) | (uintptr_t)p.lda * es | (uintptr_t)p.ldb * es | a_row | b_row) & 15) == 0;
  auto kern = vec ? simt_product_kernel<T, O, A_MN, B_MN, true, 128> : simt_product_kernel<T, O, A_MN, B_MN, false, 128>;
  return launch_ops(A_MN ? "grouped_product_dw" : "grouped_product", kern, dim3(2 * num_sms()), dim3(kSimtThreads), 0, st, p);
}

cudaError_t launch_product(ProdForm form, int dtype, int odtype, const ProdArgs& p, cudaStream_t st) {
  if (dtype != MOE_DT_F32) return launch_product_tc(form, dtype, p, st);
  return prod_types(dtype, odtype, [&](auto t, auto o) {
    using T = decltype(t);
    using O = decltype(o);
    switch (form) {
      case PROD_ROWS: return launch_simt<T, O, false, true>(p, st);
      case PROD_ROWS_T: return launch_simt<T, O, false, false>(p, st);
      default: return launch_simt<T, O, true, true>(p, st);
    }
  });
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
  return ops_status(launch_product(transposed ? PROD_ROWS_T : PROD_ROWS, dtype, odtype, p, st));
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
  return ops_status(launch_product(PROD_DW, dtype, wdtype, p, st));
}

}  // extern "C"

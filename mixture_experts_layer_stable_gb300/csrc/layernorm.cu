// layernorm.cu -- layer norm of token rows, forward and backward
// (include/moe_ops.h, moe_layernorm_*).
//
//   y  = (x - mean) * rstd * w + b
//   dx = rstd * (g - mean(g) - xh * mean(g * xh)) + dadd,  g = dy * w, xh = (x - mean) * rstd
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// Every call is bound by HBM (about ten operations an element), so a row is read
// once: a group of threads (a warp or a block) holds it in registers, the mean and
// then the sum of squared distances from it are taken from there (two passes over
// registers cost little and keep the variance of rows whose mean is large).  The
// groups are persistent.  Where rows are 16-byte aligned a block copies the rows
// that follow into a ring in shared memory (cp.async, every thread its own
// elements, so the ring needs no barrier): with only the next row in flight, in
// registers, an SM has 28 KB of the backward's rows under way, half of what HBM's
// latency asks for.  The backward's groups add their rows' dw and db in registers
// and leave one partial sum a block; a second kernel adds those in block order.
#include "ops_common.cuh"

namespace moe {

namespace {

constexpr int kElems = 16;       // elements of a row that a thread holds
constexpr int kWarpRowMax = 32 * kElems;    // a warp takes a row up to this
constexpr int kBlockRowMax = 512 * kElems;  // a block up to this
constexpr int kLnWarps = 8;      // warps (rows) of a block in the warp form
constexpr int kLoopThreads = 512;

// Sums of M values over the group's threads, the same in each.  ONE: with one barrier
// instead of two -- sh is used in turns (`turn` counts the calls), and before a part is
// written again every thread has passed the barrier of the call in between.
template <bool BLOCK, bool ONE, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], float (*sh)[32][M], int& turn) {
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] = warp_sum(v[m]);
  if constexpr (BLOCK) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float(*to)[M] = ONE ? sh[turn++ & 1] : sh[0];
    if (!ONE) __syncthreads();  // the last sums' values have been read
    if (lane == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) to[warp][m] = v[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = warp_sum(lane < nw ? to[lane][m] : 0.f);
  }
}

// The part of a row that one thread holds: N vectors of V elements, vector i at
// (i * threads + thread) * V; elements past d read as zeros.  LOOSE (V = 2): rows of
// 16-bit elements that may start in the middle of a 32-bit word or end with half of
// one: elements are loaded one by one and joined by join(), before the first use, so that
// loads stay under way; they are stored as words in rows that start with one.  (Loads of
// words in those rows: a branch, 382 us against 256 in the backward of 16384 rows of
// 7167, 176 against 188 in the forward.)
template <typename T, int V, int N, bool LOOSE>
struct Part : Words<T, V * N> {
  using Base = Words<T, V * N>;
  static constexpr bool kLoose = LOOSE;
  uint32_t high[kLoose ? N : 1];
  __device__ __forceinline__ void load(const T* __restrict__ row, int d, int tid, int nt) {
    if constexpr (kLoose) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * nt + tid) * 2;
        gload_pair(p + c, c < d, c + 1 < d, Base::w[i], high[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * nt + tid) * V;
        if (c < d) Base::template load<V>(i, row + c);
        else Base::template zero<V>(i);
      }
    }
  }
  // The thread's own elements of a ring slot.
  __device__ __forceinline__ void load_ring(const T* slot, int d, int tid, int nt) {
    if constexpr (V * sizeof(T) == 16) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * nt + tid) * V;
        if (c < d) Base::load16_shared(i, slot + c);
        else Base::template zero<V>(i);
      }
    }
  }
  __device__ __forceinline__ void join() {
    if constexpr (kLoose) {
#pragma unroll
      for (int i = 0; i < N; ++i) Base::w[i] |= high[i] << 16;
    }
  }
  __device__ __forceinline__ void store(T* __restrict__ row, int d, int tid, int nt) const {
    if constexpr (kLoose) {
      uint16_t* p = reinterpret_cast<uint16_t*>(row);
      const bool half = reinterpret_cast<uintptr_t>(row) & 2;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * nt + tid) * 2;
        if (!half && c + 1 < d) {
          *reinterpret_cast<uint32_t*>(p + c) = Base::w[i];
        } else {
          if (c < d) p[c] = (uint16_t)Base::w[i];
          if (c + 1 < d) p[c + 1] = (uint16_t)(Base::w[i] >> 16);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * nt + tid) * V;
        if (c < d) Base::template store<V>(i, row + c);
      }
    }
  }
};

// The weights of the same elements (NULL: all `other`): 16 bytes at a time where rows
// are, else one by one.
template <typename W, int V, int N>
struct Weights : Words<W, V * N> {
  static constexpr int P = V <= 2 ? 1 : V * sizeof(W) > 16 ? 16 / sizeof(W) : V;
  __device__ __forceinline__ void load(const W* __restrict__ w, float other, int d, int tid, int nt) {
#pragma unroll
    for (int k = 0; k < V * N / 2; ++k) Words<W, V * N>::set(k, F2(other, other));
    if (w == nullptr) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * nt + tid) * V;
#pragma unroll
      for (int j = 0; j < V / P; ++j)
        if (c + j * P < d) Words<W, V * N>::template load<P>(i * (V / P) + j, w + c + j * P);
    }
  }
};

// s / d, rounded once for s / d exact (a row of one value has that mean), with
// inv = 1 / d: the IEEE division is a third of the forward's instructions.
__device__ __forceinline__ float mean_of(float s, float d, float inv) {
  const float q = s * inv;
  return fmaf(fmaf(-q, d, s), inv, q);
}

// Copies of one thread's vectors of a row into its places of a ring slot.
template <typename T, int V, int N>
__device__ __forceinline__ void ring_copy(T* slot, const T* __restrict__ row, int d, int tid, int nt) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * nt + tid) * V;
    if (c < d)  // (only vectors of 16 bytes have a ring)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       static_cast<uint32_t>(__cvta_generic_to_shared(slot + c))),
                   "l"(row + c)
                   : "memory");
  }
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// RING: rows that the ring in shared memory holds (block form), or 0: the next row is
// loaded into registers.  A slot is filled again during the row that follows its own,
// by the threads that read it.
template <typename T, typename W, int V, bool LOOSE, bool BLOCK, int RING>
__global__ void __launch_bounds__(BLOCK ? 512 : 32 * kLnWarps)
    ln_forward_kernel(const T* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, float eps, T* y,
                      int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int d) {
  ops_begin();
  constexpr int N = kElems / V;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float sh[2][32][2], sh1[2][32][1], sh_n[32];
  const int tid = BLOCK ? threadIdx.x : threadIdx.x & 31, nt = BLOCK ? blockDim.x : 32;
  const int64_t first = BLOCK ? blockIdx.x : blockIdx.x * (int64_t)kLnWarps + (threadIdx.x >> 5);
  const int64_t step = BLOCK ? gridDim.x : gridDim.x * (int64_t)kLnWarps;
  const float inv_d = 1.0f / (float)d;
  T* ring = reinterpret_cast<T*>(ring_mem);
  Part<T, V, N, LOOSE> cur, next;
  Weights<W, V, N> wv, bv;
  int slot = 0, turn = 0;
  auto copy_in = [&](int sl, int64_t r) {
    if (r < rows) ring_copy<T, V, N>(ring + sl * d, x + r * ldx, d, tid, nt);
    ring_commit();
  };
  if constexpr (RING > 0) {
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) copy_in(i, first + i * step);
  } else if (first < rows) {
    next.load(x + first * ldx, d, tid, nt);
  }
  // with a ring: the elements that this warp holds, and warp `lane`
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  float wn = 1.f, inv_wn = 1.f, ln = 0.f;
  if constexpr (RING > 0) {
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) mine += (float)max(0, min(V, d - (i * nt + tid) * V));
    wn = warp_sum(mine);
    inv_wn = 1.0f / wn;
    if (lane == 0) sh_n[warp] = wn;
    __syncthreads();
    ln = lane < nw ? sh_n[lane] : 0.f;
  }
  wv.load(w, 1.f, d, tid, nt);
  bv.load(b, 0.f, d, tid, nt);
  for (int64_t r = first; r < rows; r += step) {
    if constexpr (RING > 0) {
      ring_wait<RING - 2>();
      cur.load_ring(ring + slot * d, d, tid, nt);
    } else {
      cur = next;
      cur.join();
      // without a branch (past the end this row again) single elements' loads stay under
      // way (147 us, not 208, for 16384 rows of 7168 with odd strides); whole words gain
      // nothing by it (the compiler then waits for them at once: 197 us, not 117, for
      // 7166)
      if (LOOSE || sizeof(T) == 4) next.load(x + (r + step < rows ? r + step : r) * ldx, d, tid, nt);
      else if (r + step < rows) next.load(x + (r + step) * ldx, d, tid, nt);
    }
    F2 v[kElems / 2], t(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kElems / 2; ++k) {
      v[k] = cur.pair(k);
      t = add2(t, v[k]);
    }
    // With a ring: the warp's mean and its squared distances from that, and the row's
    // from the warps' (of distances only, so that a large mean costs nothing), in one
    // exchange; else the row's mean, then the distances from it, in two.
    float near;  // the mean that the distances are taken from
    if constexpr (RING > 0) {
      near = mean_of(warp_sum(sum2(t)), wn, inv_wn);
      copy_in(slot == 0 ? RING - 1 : slot - 1, r + (RING - 1) * step);
      if (++slot == RING) slot = 0;
    } else {
      float s[1] = {sum2(t)};
      group_sum<BLOCK, false>(s, sh1, turn);
      near = mean_of(s[0], (float)d, inv_d);
    }
    t = F2(0.f, 0.f);
    const F2 neg_mu(-near, -near);
#pragma unroll
    for (int k = 0; k < kElems / 2; ++k) {
      const F2 c = add2(v[k], neg_mu);
      v[k] = c;
      if (V == 1) {  // the pair's elements are of different vectors
        const float2 f = c.get();
        const float c0 = (2 * k * nt + tid) < d ? f.x : 0.f, c1 = ((2 * k + 1) * nt + tid) < d ? f.y : 0.f;
        t = fma2(F2(c0, c1), F2(c0, c1), t);
      } else if (LOOSE) {  // d may be odd
        const int e = (k * nt + tid) * 2;
        const float2 f = c.get();
        const F2 m(e < d ? f.x : 0.f, e + 1 < d ? f.y : 0.f);
        t = fma2(m, m, t);
      } else if ((2 * k / V * nt + tid) * V < d) {
        t = fma2(c, c, t);
      }
    }
    float mu = near, m2;
    if constexpr (RING > 0) {
      const float wm2 = warp_sum(sum2(t));
      float(*to)[2] = sh[turn++ & 1];  // (in turns, as in group_sum)
      if (lane == 0) {
        to[warp][0] = near;
        to[warp][1] = wm2;
      }
      __syncthreads();
      const float lmu = lane < nw ? to[lane][0] : 0.f, lm2 = lane < nw ? to[lane][1] : 0.f;
      mu = mean_of(warp_sum(ln * lmu), (float)d, inv_d);
      const float dist = lmu - mu;
      m2 = warp_sum(lane < nw ? fmaf(ln * dist, dist, lm2) : 0.f);
    } else {
      float s[1] = {sum2(t)};
      group_sum<BLOCK, false>(s, sh1, turn);
      m2 = s[0];
    }
    const float rs = rsqrtf(fmaf(m2, inv_d, eps));
    if (tid == 0 && mean != nullptr) {
      mean[r] = mu;
      rstd[r] = rs;
    }
    const F2 rs2(rs, rs);
    if constexpr (RING > 0) {
      const float shift = (near - mu) * rs;
      const F2 shift2(shift, shift);
#pragma unroll
      for (int k = 0; k < kElems / 2; ++k) cur.set(k, fma2(fma2(v[k], rs2, shift2), wv.pair(k), bv.pair(k)));
    } else {
#pragma unroll
      for (int k = 0; k < kElems / 2; ++k) cur.set(k, fma2(mul2(v[k], rs2), wv.pair(k), bv.pair(k)));
    }
    cur.store(y + r * ldy, d, tid, nt);
  }
}

// dx of the group's rows; with part, the rows' sums of dy * xh and dy to
// part[block][0 / 1][d].
template <typename T, typename W, int V, bool LOOSE, bool BLOCK, int RING>
__global__ void __launch_bounds__(BLOCK ? 512 : 32 * kLnWarps)
    ln_backward_kernel(const T* dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, const W* __restrict__ w,
                       const float* mean, const float* rstd, const T* dadd, int64_t ldadd,
                       T* dx, int64_t lddx, float* __restrict__ part, int64_t rows, int d) {
  ops_begin();
  constexpr int N = kElems / V;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float sh[2][32][2];
  const int tid = BLOCK ? threadIdx.x : threadIdx.x & 31, nt = BLOCK ? blockDim.x : 32;
  const int64_t first = BLOCK ? blockIdx.x : blockIdx.x * (int64_t)kLnWarps + (threadIdx.x >> 5);
  const int64_t step = BLOCK ? gridDim.x : gridDim.x * (int64_t)kLnWarps;
  const float inv_d = 1.0f / (float)d;
  T* ring = reinterpret_cast<T*>(ring_mem);
  F2 aw[kElems / 2], ab[kElems / 2];
#pragma unroll
  for (int k = 0; k < kElems / 2; ++k) aw[k] = ab[k] = F2(0.f, 0.f);
  Part<T, V, N, LOOSE> cx, cy, nx, ny;
  Weights<W, V, N> wv;
  float nmu = 0.f, nrs = 0.f;
  int slot = 0, turn = 0;
  auto copy_in = [&](int sl, int64_t r) {
    if (r < rows) {
      ring_copy<T, V, N>(ring + 2 * sl * d, x + r * ldx, d, tid, nt);
      ring_copy<T, V, N>(ring + (2 * sl + 1) * d, dy + r * lddy, d, tid, nt);
    }
    ring_commit();
  };
  if constexpr (RING > 0) {
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) copy_in(i, first + i * step);
  } else if (first < rows) {
    nx.load(x + first * ldx, d, tid, nt);
    ny.load(dy + first * lddy, d, tid, nt);
  }
  if (first < rows) {
    nmu = gload(mean + first);
    nrs = gload(rstd + first);
  }
  wv.load(w, 1.f, d, tid, nt);
  for (int64_t r = first; r < rows; r += step) {
    const float mu = nmu, rs = nrs;
    // the next row's loads without a branch (past the end: this row again): behind one
    // their values would be waited for where it joins (16384 rows of 7168: 30 us more
    // than the 124)
    const int64_t rn = r + step < rows ? r + step : r;
    nmu = gload(mean + rn);
    nrs = gload(rstd + rn);
    if constexpr (RING > 0) {
      ring_wait<RING - 2>();
      cx.load_ring(ring + 2 * slot * d, d, tid, nt);
      cy.load_ring(ring + (2 * slot + 1) * d, d, tid, nt);
    } else {
      cx = nx;
      cy = ny;
      cx.join();
      cy.join();
      nx.load(x + rn * ldx, d, tid, nt);
      ny.load(dy + rn * lddy, d, tid, nt);
    }
    // elements past d: dy and so g are zero
    F2 xh[kElems / 2], g[kElems / 2], s1(0.f, 0.f), s2(0.f, 0.f);
    // (x - mean first: in one fma with -mean * rstd that product's rounding would count,
    // which is large where the mean is many times the spread)
    const F2 rs2(rs, rs), neg_mu(-mu, -mu);
    // (loose rows: all of xh before the rest, 16384 rows of 7167 256 us, else 287; the
    // others lose by it: 7168 139 us, not 124)
    if constexpr (LOOSE) {
#pragma unroll
      for (int k = 0; k < kElems / 2; ++k) xh[k] = mul2(add2(cx.pair(k), neg_mu), rs2);
    }
#pragma unroll
    for (int k = 0; k < kElems / 2; ++k) {
      const F2 t = cy.pair(k);
      if constexpr (!LOOSE) xh[k] = mul2(add2(cx.pair(k), neg_mu), rs2);
      g[k] = mul2(t, wv.pair(k));
      s1 = add2(s1, g[k]);
      s2 = fma2(g[k], xh[k], s2);
      aw[k] = fma2(t, xh[k], aw[k]);
      ab[k] = add2(ab[k], t);
    }
    float s[2] = {sum2(s1), sum2(s2)};
    group_sum<BLOCK, (RING > 0)>(s, sh, turn);
    if constexpr (RING > 0) {
      copy_in(slot == 0 ? RING - 1 : slot - 1, r + (RING - 1) * step);
      if (++slot == RING) slot = 0;
    }
    // dx = rs g - rs m1 - xh rs m2
    const float m1 = -rs * (s[0] * inv_d), m2 = -rs * (s[1] * inv_d);
    const F2 m1s(m1, m1), m2s(m2, m2);
    // (loaded behind the sums: 16384 rows of 7168 take 203 us with it, 138 for the bytes,
    // and 127 without)
    if (dadd != nullptr) {
      cy.load(dadd + r * ldadd, d, tid, nt);
      cy.join();
    }
#pragma unroll
    for (int k = 0; k < kElems / 2; ++k) {
      F2 v = fma2(xh[k], m2s, fma2(g[k], rs2, m1s));
      if (dadd != nullptr) v = add2(v, cy.pair(k));
      cx.set(k, v);
    }
    cx.store(dx + r * lddx, d, tid, nt);
  }
  if (part == nullptr) return;
  float* mine = part + (size_t)blockIdx.x * 2 * d;
  float fw[kElems], fb[kElems];
#pragma unroll
  for (int k = 0; k < kElems / 2; ++k) {
    const float2 a = aw[k].get(), c = ab[k].get();
    fw[2 * k] = a.x;
    fw[2 * k + 1] = a.y;
    fb[2 * k] = c.x;
    fb[2 * k + 1] = c.y;
  }
  if constexpr (BLOCK) {
    constexpr int P = LOOSE ? 1 : V < 4 ? V : 4;  // floats at once (else d is a multiple of V)
#pragma unroll
    for (int k = 0; k < kElems; k += P) {
      const int c = (k / V * nt + tid) * V + k % V;
      if constexpr (P > 1) {
        Vec<float, P> pw, pb;
#pragma unroll
        for (int q = 0; q < P; ++q) pw.e[q] = fw[k + q], pb.e[q] = fb[k + q];
        if (c < d) {
          *reinterpret_cast<Vec<float, P>*>(mine + c) = pw;
          *reinterpret_cast<Vec<float, P>*>(mine + d + c) = pb;
        }
      } else if (c < d) {
        mine[c] = fw[k];
        mine[d + c] = fb[k];
      }
    }
  } else {
    // the warps add theirs one after the other
    __shared__ float acc[2][kWarpRowMax];
    for (int q = 0; q < kLnWarps; ++q) {
      if ((threadIdx.x >> 5) == q) {
#pragma unroll
        for (int k = 0; k < kElems; ++k) {
          const int c = (k / V * nt + tid) * V + k % V;
          if (c < d) {
            acc[0][c] = (q ? acc[0][c] : 0.f) + fw[k];
            acc[1][c] = (q ? acc[1][c] : 0.f) + fb[k];
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
      mine[c] = acc[0][c];
      mine[d + c] = acc[1][c];
    }
  }
}

// Rows too wide for a block's registers: three passes over the row (it stays in
// L1 / L2), one element at a time.  Far from HBM's rate: 4096 rows of 12288 in bf16
// take 225 us forward (30 for the bytes) and 580 backward (45), where each row also
// reads and writes the block's sums of dw and db.
template <typename T, typename W>
__global__ void __launch_bounds__(kLoopThreads)
    ln_forward_loop_kernel(const T* x, int64_t ldx, const W* __restrict__ w, const W* __restrict__ b, float eps, T* y,
                           int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd, int64_t rows, int d) {
  __shared__ float sh[2][32][1];
  int turn = 0;
  ops_begin();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const T* xr = x + r * ldx;
    float s[1] = {0.f};
    for (int i = threadIdx.x; i < d; i += blockDim.x) s[0] += gload_f32(xr + i);
    group_sum<true, false>(s, sh, turn);
    const float mu = s[0] / (float)d;
    s[0] = 0.f;
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float c = gload_f32(xr + i) - mu;
      s[0] = fmaf(c, c, s[0]);
    }
    group_sum<true, false>(s, sh, turn);
    const float rs = 1.0f / sqrtf(s[0] / (float)d + eps);
    if (threadIdx.x == 0 && mean != nullptr) {
      mean[r] = mu;
      rstd[r] = rs;
    }
    for (int i = threadIdx.x; i < d; i += blockDim.x)
      y[r * ldy + i] = from_f32<T>(fmaf((gload_f32(xr + i) - mu) * rs, w ? gload_f32(w + i) : 1.f, b ? gload_f32(b + i) : 0.f));
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kLoopThreads)
    ln_backward_loop_kernel(const T* dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, const W* __restrict__ w,
                            const float* __restrict__ mean, const float* __restrict__ rstd, const T* dadd,
                            int64_t ldadd, T* dx, int64_t lddx, float* __restrict__ part, int64_t rows, int d) {
  __shared__ float sh[2][32][2];
  int turn = 0;
  ops_begin();
  float* mine = part ? part + (size_t)blockIdx.x * 2 * d : nullptr;
  bool begun = false;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x, begun = true) {
    const float mu = gload(mean + r), rs = gload(rstd + r);
    float s[2] = {0.f, 0.f};
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float t = gload_f32(dy + r * lddy + i), g = t * (w ? gload_f32(w + i) : 1.f);
      const float xh = (gload_f32(x + r * ldx + i) - mu) * rs;
      s[0] += g;
      s[1] = fmaf(g, xh, s[1]);
      if (mine) {  // a column is one thread's
        mine[i] = fmaf(t, xh, begun ? mine[i] : 0.f);
        mine[d + i] = (begun ? mine[d + i] : 0.f) + t;
      }
    }
    group_sum<true, false>(s, sh, turn);
    const float m1 = s[0] / (float)d, m2 = s[1] / (float)d;
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      const float g = gload_f32(dy + r * lddy + i) * (w ? gload_f32(w + i) : 1.f);
      const float xh = (gload_f32(x + r * ldx + i) - mu) * rs;
      float v = rs * (g - m1 - xh * m2);
      if (dadd) v += gload_f32(dadd + r * ldadd + i);
      dx[r * lddx + i] = from_f32<T>(v);
    }
  }
}

// dw and db from the blocks' partial sums: 32 columns a block, its 32 warps each a
// run of the partials, joined in order.
template <typename W>
__global__ void __launch_bounds__(1024) ln_reduce_kernel(const float* __restrict__ part, int np, W* __restrict__ dw,
                                                         W* __restrict__ db, int d) {
  __shared__ float sh[32][33];
  ops_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // column of [2 d]: dw's, then db's
  const int per = (np + 31) / 32, p1 = min(np, (warp + 1) * per);
  float s = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int p = warp * per; p < p1; ++p) s += gload(part + (size_t)p * 2 * d + c);
  }
  sh[warp][lane] = s;
  __syncthreads();
  // column `warp` of the block: its 32 sums, one a lane
  const int cc = blockIdx.x * 32 + warp;
  s = warp_sum(sh[lane][warp]);
  if (lane == 0 && cc < 2 * d) {
    if (cc < d) {
      if (dw) dw[cc] = from_f32<W>(s);
    } else if (db) {
      db[cc - d] = from_f32<W>(s);
    }
  }
}

bool ln_args(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d) {
  return dtype_valid(dtype) && (wdtype == dtype || wdtype == MOE_DT_F32) && rows >= 0 &&
         rows <= ((int64_t)1 << 40) && d >= 1 && d <= 65536;
}

// f(T{}, W{}) for the element types of the rows and of the weights.
template <typename F>
cudaError_t ln_types(int dtype, int wdtype, F f) {
  return with_dtype(dtype, [&](auto t) {
    if (wdtype == MOE_DT_F32) return f(t, float());
    return f(t, t);
  });
}

// How a thread moves elements: 16 bytes at once where every row and d allow it, else
// words of 32 bits, else 16-bit elements wherever they lie.  `a`: the or of the
// addresses and row strides in bytes; `aw`: of the weights' addresses, which are read
// 16 bytes at a time too.
enum LnMove { LN_VECTORS, LN_WORDS, LN_LOOSE };
LnMove ln_move(size_t es, int d, uintptr_t a, uintptr_t aw) {
  a |= (uintptr_t)d * es;
  return (a | aw) % 16 == 0 ? LN_VECTORS : a % 4 == 0 ? LN_WORDS : LN_LOOSE;
}
uintptr_t bits(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// Threads of a block that takes a row.
int ln_block_threads(int d) { return ((d + kElems - 1) / kElems + 31) / 32 * 32; }
// Threads launched for each SM.  They are what it holds of the block forms: 64 registers
// a thread in the forward of vectors, up to 128 in the others.  (More blocks than that
// leave a second wave of them: 2048 rows of 2048, backward with 640 threads an SM
// 24.5 us, with 512 20.4.)  The warp forms (d <= 512) take more registers, and some leave
// such a wave: of four blocks two or three fit in the forward of vectors (80 registers,
// 88 in fp32; all four with fp16 weights, 64), of two one in the backward of fp32 rows
// (150 to 165) and of loose ones (159 to 167).  The backward of loose block rows is cut
// to 128 registers and spills: 48 bytes with fp32 weights, 236 with bf16 ones (16384
// rows of 7167: 256 us and 550).
constexpr int kForwardThreads = 1024, kBackwardThreads = 512;
int ln_forward_threads(LnMove v) { return v == LN_VECTORS ? kForwardThreads : kBackwardThreads; }
int ln_blocks_per_sm(int d, int threads) {
  const int t = d <= kWarpRowMax ? 32 * kLnWarps : d <= kBlockRowMax ? ln_block_threads(d) : kLoopThreads;
  return t > threads / 2 ? 1 : threads / t;
}
// Blocks of a call: about as many as fit on the GPU, so that each stays on its rows.
int ln_blocks(int64_t rows, int d, int threads) {
  const int64_t need = d <= kWarpRowMax ? (rows + kLnWarps - 1) / kLnWarps : rows;
  const int64_t most = (int64_t)num_sms() * ln_blocks_per_sm(d, threads);
  return (int)(need < most ? need : most);
}

// The kernel form for the way elements move and the row length, f(tag, ring bytes)
// doing the launch.  Block rows of vectors go through a ring of four rows, three where
// four would not fit into the block's share of shared memory (row_bytes: of all arrays
// that a ring row holds).  Words do not: as many copies and then as many reads as
// elements cost more than the deeper prefetch gives (d = 7166, 16384 rows: forward
// 190 us with the ring, 117 without).
template <int V_, bool LOOSE_, bool BLOCK_, int RING_>
struct LnTag {
  static constexpr int V = V_, RING = RING_;
  static constexpr bool LOOSE = LOOSE_, BLOCK = BLOCK_;
};
template <typename T, typename F>
void ln_pick(LnMove v, int d, int per_sm, size_t row_bytes, F f) {
  constexpr int VF = 16 / sizeof(T), VW = 4 / sizeof(T);
  const bool warp = d <= kWarpRowMax;
  if (v == LN_VECTORS) {
    const size_t share = 225 * 1024 / per_sm - 1024;
    if (warp) f(LnTag<VF, false, false, 0>(), (size_t)0);
    else if (4 * row_bytes <= share) f(LnTag<VF, false, true, 4>(), 4 * row_bytes);
    else f(LnTag<VF, false, true, 3>(), 3 * row_bytes);
  } else if (v == LN_WORDS) {
    if (warp) f(LnTag<VW, false, false, 0>(), (size_t)0);
    else f(LnTag<VW, false, true, 0>(), (size_t)0);
  } else if constexpr (sizeof(T) == 2) {
    if (warp) f(LnTag<2, true, false, 0>(), (size_t)0);
    else f(LnTag<2, true, true, 0>(), (size_t)0);
  }
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layernorm_forward(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d, const void* x,
                                 int64_t ldx, const void* weight, const void* bias, float eps, void* y,
                                 int64_t ldy, float* mean, float* rstd, moe_stream_t stream) {
  if (!ln_args(dtype, wdtype, rows, d) || ldx < d || ldy < d || !(eps >= 0.f) || !isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype), wes = dtype_bytes(wdtype);
  if (!elem_ok_or_null(weight, wes) || !elem_ok_or_null(bias, wes) || (mean == nullptr) != (rstd == nullptr) ||
      !elem_ok_or_null(mean, 4) || !elem_ok_or_null(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!elem_ok(x, es) || !elem_ok(y, es)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LnMove v = ln_move(es, d, bits(x) | bits(y) | (uintptr_t)(ldx * es) | (uintptr_t)(ldy * es),
                       bits(weight) | bits(bias));
  const int threads = ln_forward_threads(v), grid = ln_blocks(rows, d, threads);
  return ops_status(ln_types(dtype, wdtype, [&](auto t, auto wt) {
    using T = decltype(t);
    using W = decltype(wt);
    const T* xp = static_cast<const T*>(x);
    const W *wp = static_cast<const W*>(weight), *bp = static_cast<const W*>(bias);
    T* yp = static_cast<T*>(y);
    cudaError_t e = cudaSuccess;
    if (d > kBlockRowMax)
      e = launch_ops("layernorm_forward", ln_forward_loop_kernel<T, W>, dim3(grid), dim3(kLoopThreads), 0, st, xp, ldx, wp,
                     bp, eps, yp, ldy, mean, rstd, rows, d);
    else
      ln_pick<T>(v, d, ln_blocks_per_sm(d, threads), d * sizeof(T), [&](auto tag, size_t smem) {
        using K = decltype(tag);
        auto kern = ln_forward_kernel<T, W, K::V, K::LOOSE, K::BLOCK, K::RING>;
        static SmemAllowed allowed;
        e = allow_smem(kern, smem, allowed);
        if (e == cudaSuccess) e = launch_ops("layernorm_forward", kern, dim3(grid), dim3(K::BLOCK ? ln_block_threads(d) : 32 * kLnWarps), smem,
                       st, xp, ldx, wp, bp, eps, yp, ldy, mean, rstd, rows, d);
      });
    return e;
  }));
}

size_t moe_layernorm_workspace_bytes(int64_t rows, int32_t d) {
  if (!ln_args(MOE_DT_F32, MOE_DT_F32, rows, d)) return 0;
  return ((size_t)(ln_blocks(rows, d, kBackwardThreads) + 1) * 2 * d * sizeof(float) + 127) / 128 * 128;
}

moe_status moe_layernorm_backward(int32_t dtype, int32_t wdtype, int64_t rows, int32_t d, const void* dy,
                                  int64_t lddy, const void* x, int64_t ldx, const void* weight,
                                  const float* mean, const float* rstd, const void* dadd, int64_t ldadd,
                                  void* dx, int64_t lddx, void* dweight, void* dbias, void* ws,
                                  size_t ws_bytes, moe_stream_t stream) {
  if (!ln_args(dtype, wdtype, rows, d) || lddy < d || ldx < d || lddx < d || (dadd != nullptr && ldadd < d))
    return MOE_ERR_INVALID_ARG;
  const size_t es = dtype_bytes(dtype), wes = dtype_bytes(wdtype);
  if (!elem_ok_or_null(weight, wes) || !elem_ok_or_null(dadd, es) || !elem_ok_or_null(dweight, wes) ||
      !elem_ok_or_null(dbias, wes))
    return MOE_ERR_INVALID_ARG;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (sums && (ws == nullptr || !aligned_to(ws, 128))) return MOE_ERR_INVALID_ARG;
  if (sums && ws_bytes < moe_layernorm_workspace_bytes(rows, d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (rows > 0 && (!elem_ok(dy, es) || !elem_ok(x, es) || !elem_ok(dx, es) || !elem_ok(mean, 4) || !elem_ok(rstd, 4)))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0 && !sums) return MOE_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const LnMove v = ln_move(es, d,
                       bits(dy) | bits(x) | bits(dx) | bits(dadd) | (uintptr_t)(lddy * es) | (uintptr_t)(ldx * es) |
                           (uintptr_t)(lddx * es) | (uintptr_t)((dadd ? ldadd : 0) * es),
                       bits(weight));
  const int grid = ln_blocks(rows, d, kBackwardThreads);
  return ops_status(ln_types(dtype, wdtype, [&](auto t, auto wt) {
    using T = decltype(t);
    using W = decltype(wt);
    const T *dyp = static_cast<const T*>(dy), *xp = static_cast<const T*>(x), *ap = static_cast<const T*>(dadd);
    const W* wp = static_cast<const W*>(weight);
    T* dxp = static_cast<T*>(dx);
    float* part = sums ? static_cast<float*>(ws) : nullptr;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
      if (d > kBlockRowMax)
        e = launch_ops("layernorm_backward", ln_backward_loop_kernel<T, W>, dim3(grid), dim3(kLoopThreads), 0, st, dyp,
                       lddy, xp, ldx, wp, mean, rstd, ap, ldadd, dxp, lddx, part, rows, d);
      else
        ln_pick<T>(v, d, ln_blocks_per_sm(d, kBackwardThreads), 2 * d * sizeof(T), [&](auto tag, size_t smem) {
          using K = decltype(tag);
          auto kern = ln_backward_kernel<T, W, K::V, K::LOOSE, K::BLOCK, K::RING>;
          static SmemAllowed allowed;
          e = allow_smem(kern, smem, allowed);
          if (e == cudaSuccess) e = launch_ops("layernorm_backward", kern, dim3(grid), dim3(K::BLOCK ? ln_block_threads(d) : 32 * kLnWarps),
                         smem, st, dyp, lddy, xp, ldx, wp, mean, rstd, ap, ldadd, dxp, lddx, part, rows, d);
        });
    }
    if (e == cudaSuccess && sums)
      e = launch_ops("layernorm_reduce", ln_reduce_kernel<W>, dim3((2 * d + 31) / 32), dim3(1024), 0, st, part, grid,
                     static_cast<W*>(dweight), static_cast<W*>(dbias), d);
    return e;
  }));
}

}  // extern "C"

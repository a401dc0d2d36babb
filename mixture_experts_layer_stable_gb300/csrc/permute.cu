// permute.cu -- rows sorted by expert and back (include/moe_ops.h:
// moe_sort_rows, moe_permute, moe_unpermute, moe_unpermute_backward).
//
// The sort is a counting sort over E + 1 buckets (the last: rows without an
// expert) and is bound by latency; the moves are bound by HBM.
#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

// ------------------------------------------------------------------ sort
constexpr int kSortIters = 8;                     // rows a lane holds
constexpr int kSortBlockRows = 32 * 32 * kSortIters;
constexpr int kSortCluster = 8;

// Expert of a row, or E for one without an expert.
__device__ __forceinline__ int bucket(int id, int E) { return (unsigned)id < (unsigned)E ? id : E; }

__device__ __forceinline__ int ld_cluster(uint32_t saddr, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(saddr, rank)) : "memory");
  return v;
}

// Rows [blockIdx.x * per_block, ...) of the sort, at most kSortBlockRows, in W
// warps of whole groups of 32 rows.  Each warp counts its rows by bucket while it
// ranks them (the rows of a group that share a bucket by warp match, in order);
// exclusive prefixes over the warps, the blocks and the buckets then give every
// row its place.  No atomics decide a place, so the order is stable.
// The blocks' totals: of the one cluster that does the whole sort, from its shared
// memories; else from `before` [blocks, E + 1], rows in earlier blocks by bucket,
// and `total` [E + 1].
template <bool CLUSTER>
__global__ void __launch_bounds__(1024) sort_kernel(const int* __restrict__ ids, int64_t R, int E, int W, int per_block,
                                                    const int* __restrict__ before, const int* __restrict__ total,
                                                    int* __restrict__ counts, int* __restrict__ offsets,
                                                    int* __restrict__ perm, int* __restrict__ inv) {
  extern __shared__ int sort_mem[];
  int* wcnt = sort_mem;                  // [W][E + 1]
  int* tot = sort_mem + W * (E + 1);     // [E + 1] rows of this block
  int* start = tot + (E + 1);            // [E + 1] place of this block's first row
  __shared__ int wsum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = E + 1;
  for (int i = tid; i < W * nb; i += blockDim.x) wcnt[i] = 0;
  __syncthreads();
  ops_begin();
  const int64_t b0 = blockIdx.x * (int64_t)per_block, b1 = min(R, b0 + per_block);
  const int per_warp = per_block / W;    // a multiple of 32
  const int64_t w0 = b0 + warp * per_warp, w1 = min(b1, w0 + per_warp);
  int e[kSortIters], at[kSortIters];
  if (warp < W) {
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) {
      const int64_t r = w0 + i * 32 + lane;
      e[i] = r < w1 ? bucket(gload(ids + r), E) : -1;
    }
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) {
      if (w0 + i * 32 >= w1) break;
      const uint32_t peers = __match_any_sync(0xffffffffu, e[i]);
      const int first = __ffs(peers) - 1;
      int base = 0;
      if (lane == first && e[i] >= 0) {
        base = wcnt[warp * nb + e[i]];
        wcnt[warp * nb + e[i]] = base + __popc(peers);
      }
      __syncwarp();
      at[i] = __shfl_sync(0xffffffffu, base, first) + __popc(peers & ((1u << lane) - 1u));
    }
  }
  __syncthreads();
  for (int b = tid; b < nb; b += blockDim.x) {
    int run = 0;
    for (int w = 0; w < W; ++w) {
      const int c = wcnt[w * nb + b];
      wcnt[w * nb + b] = run;
      run += c;
    }
    tot[b] = run;
  }
  if constexpr (CLUSTER) cluster_sync();
  else __syncthreads();
  // every bucket's rows in all blocks, and in the blocks before this one
  int all = 0, pre = 0;  // of bucket tid (E <= 1024 threads; the dropped rows' apart)
  if (tid < E) {
    if constexpr (CLUSTER) {
      const uint32_t me = cluster_ctarank(), a = smem_u32(tot + tid);
#pragma unroll
      for (uint32_t c = 0; c < kSortCluster; ++c) {
        const int v = c < gridDim.x ? ld_cluster(a, c) : 0;
        all += v;
        if (c < me) pre += v;
      }
    } else if (total != nullptr) {
      all = gload(total + tid);
      pre = gload(before + (size_t)blockIdx.x * nb + tid);
    } else {
      all = tot[tid];
    }
  }
  int inc = all;  // inclusive scan over the buckets
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  int below = lane < warp && lane < nw ? wsum[lane] : 0;
  below = __reduce_add_sync(0xffffffffu, below);
  const int kept = __reduce_add_sync(0xffffffffu, lane < nw ? wsum[lane] : 0);
  if (tid < E) {
    start[tid] = below + inc - all + pre;
    if (blockIdx.x == 0) {
      counts[tid] = all;
      offsets[tid] = below + inc - all;
    }
  }
  if (tid == 0) {
    int drop = 0;
    if constexpr (CLUSTER) {
      const uint32_t me = cluster_ctarank(), a = smem_u32(tot + E);
      for (uint32_t c = 0; c < me; ++c) drop += ld_cluster(a, c);
    } else if (total != nullptr) {
      drop = gload(before + (size_t)blockIdx.x * nb + E);
    }
    start[E] = kept + drop;
    if (blockIdx.x == 0) offsets[E] = kept;
  }
  if constexpr (CLUSTER) cluster_sync();  // no block leaves while others read its totals
  else __syncthreads();
  if (warp < W) {
#pragma unroll
    for (int i = 0; i < kSortIters; ++i) {
      if (e[i] < 0) continue;
      const int r = (int)(w0 + i * 32 + lane);
      const int p = start[e[i]] + wcnt[warp * nb + e[i]] + at[i];
      perm[p] = r;
      inv[r] = p;
    }
  }
}

// More rows than a cluster takes: the blocks' histograms ...
__global__ void __launch_bounds__(1024) sort_hist_kernel(const int* __restrict__ ids, int64_t R, int E,
                                                         int* __restrict__ hist) {
  __shared__ int sh[kMaxE + 1];
  for (int e = threadIdx.x; e <= E; e += blockDim.x) sh[e] = 0;
  __syncthreads();
  ops_begin();
  const int64_t r0 = blockIdx.x * (int64_t)kSortBlockRows, r1 = min(R, r0 + kSortBlockRows);
  for (int64_t r = r0 + threadIdx.x; r < r1; r += blockDim.x) atomicAdd(&sh[bucket(gload(ids + r), E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) hist[(size_t)blockIdx.x * (E + 1) + e] = sh[e];
}

// ... and their exclusive prefixes over the blocks, in place, with the totals: 32
// buckets a block, its 32 warps each a run of the histograms.
__global__ void __launch_bounds__(1024) sort_scan_kernel(int* __restrict__ hist, int blocks, int nb,
                                                         int* __restrict__ total) {
  __shared__ int sh[32][33];
  ops_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int per = (blocks + 31) / 32, p0 = min(blocks, warp * per), p1 = min(blocks, p0 + per);
  int sum = 0;
  if (e < nb) {
#pragma unroll 8
    for (int p = p0; p < p1; ++p) sum += gload(hist + (size_t)p * nb + e);
  }
  sh[warp][lane] = sum;
  __syncthreads();
  if (e >= nb) return;
  int run = 0, all = 0;
  for (int w = 0; w < 32; ++w) {
    if (w == warp) run = all;
    all += sh[w][lane];
  }
  if (warp == 0) total[e] = all;
  for (int p = p0; p < p1; p += 8) {
    int c[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) c[u] = p + u < p1 ? gload(hist + (size_t)(p + u) * nb + e) : 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (p + u < p1) hist[(size_t)(p + u) * nb + e] = run;
      run += c[u];
    }
  }
}

// ------------------------------------------------------------------ moves
// Threads are laid over (token, unit of its row): a block takes `tpb` tokens, or
// 1 / chunks of one.
struct Lay {
  int nv;      // threads of a token
  int tpb;     // tokens of a block
  int chunks;  // blocks of a token (1 when tpb > 1)
};
__device__ __forceinline__ bool lay_at(const Lay& l, int64_t T, int64_t& t, int& c) {
  if (l.chunks > 1) {
    t = blockIdx.x / l.chunks;
    c = (int)(blockIdx.x - t * l.chunks) * blockDim.x + threadIdx.x;
  } else {
    const int a = threadIdx.x / l.nv;
    t = blockIdx.x * (int64_t)l.tpb + a;
    c = threadIdx.x - a * l.nv;
    if (a >= l.tpb) return false;
  }
  return t < T && c < l.nv;
}

// Rows of whole 16-byte vectors: a token's vector is read once and written to the k
// places.
template <typename T, int V>
__global__ void __launch_bounds__(256) permute_kernel(const T* __restrict__ x, int64_t ldx, const int* __restrict__ inv,
                                                      const int* __restrict__ kept_p, int k, int d, int64_t tokens,
                                                      Lay lay, T* __restrict__ xp) {
  ops_begin();
  int64_t t;
  int c;
  if (!lay_at(lay, tokens, t, c)) return;
  const int kept = gload(kept_p);
  Words<T, V> v, z;
  z.clear();
  v.template load<V>(0, x + t * ldx + c * V);
  const int* pi = inv + t * k;
#pragma unroll 8
  for (int j = 0; j < k; ++j) {
    const int p = gload(pi + j);
    T* dst = xp + (int64_t)p * d + c * V;
    if (p < kept) v.template store<V>(0, dst);
    else z.template store<V>(0, dst);
  }
}

// The k rows' vectors of a token, eight loads in flight, summed in slot order.
template <typename T, int V>
__global__ void __launch_bounds__(256) unpermute_kernel(const T* __restrict__ y, const float* __restrict__ w,
                                                        const int* __restrict__ inv, const int* __restrict__ kept_p,
                                                        int k, int d, int64_t tokens, Lay lay, const T* base,
                                                        int64_t ldbase, T* out, int64_t ldout) {
  constexpr int E = V;
  ops_begin();
  int64_t t;
  int c;
  if (!lay_at(lay, tokens, t, c)) return;
  const int kept = gload(kept_p);
  F2 s[E / 2];
#pragma unroll
  for (int q = 0; q < E / 2; ++q) s[q] = F2(0.f, 0.f);
  Words<T, E> v[8];
  if (base != nullptr) {
    v[0].clear();
    v[0].template load<V>(0, base + t * ldbase + c * V);
#pragma unroll
    for (int q = 0; q < E / 2; ++q) s[q] = v[0].pair(q);
  }
  for (int j0 = 0; j0 < k; j0 += 8) {
    float wj[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u;
      const int p = j < k ? gload(inv + t * k + j) : kept;
      v[u].clear();
      wj[u] = 0.f;
      if (p < kept) {
        v[u].template load<V>(0, y + (int64_t)p * d + c * V);
        wj[u] = w ? gload(w + t * k + j) : 1.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j0 + u >= k) break;
      const F2 ww(wj[u], wj[u]);
#pragma unroll
      for (int q = 0; q < E / 2; ++q) s[q] = fma2(ww, v[u].pair(q), s[q]);
    }
  }
  Words<T, E> o;
#pragma unroll
  for (int q = 0; q < E / 2; ++q) o.set(q, s[q]);
  o.template store<V>(0, out + t * ldout + c * V);
}

// A block a token: its gradient in registers (kBwdVec vectors a thread, in turns
// for wider rows), written to the k places with their weights while the k rows of y
// are read for the scalar products; those are summed over each warp's lanes, then
// over the warps in order.
constexpr int kBwdVec = 2, kBwdThreads = 512;
template <typename T, int V>
__global__ void __launch_bounds__(kBwdThreads, 2) unpermute_backward_kernel(
    const T* __restrict__ dout, int64_t lddout, const T* __restrict__ y, const float* __restrict__ w,
    const int* __restrict__ inv, const int* __restrict__ kept_p, int k, int d, T* __restrict__ dy,
    float* __restrict__ dw) {
  constexpr int E = V;
  __shared__ float sh[kBwdThreads / 32][kMaxK];
  ops_begin();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int kept = gload(kept_p), span = nt * V * kBwdVec;
  const T* spare = kept > 0 ? y : dout + t * lddout;  // d elements that can be read and are not used
  for (int c0 = 0; c0 < d; c0 += span) {
    Words<T, E> g[kBwdVec];
#pragma unroll
    for (int i = 0; i < kBwdVec; ++i) {
      const int c = c0 + (i * nt + tid) * V;
      g[i].clear();
      if (c < d) g[i].template load<V>(0, dout + t * lddout + c);
    }
#pragma unroll 2
    for (int j = 0; j < k; ++j) {
      const int p = gload(inv + t * k + j);
      const bool live = p < kept;
      const float wj = w ? gload(w + t * k + j) : 1.f;
      const float wr = live ? wj : 0.f;
      const int64_t row = (int64_t)p * d;
      Words<T, E> v[kBwdVec];
      if (dw != nullptr) {  // (loads without branches: a dropped row's from `spare`, past d of the row's last vector)
        const T* src = live ? y + row : spare;
#pragma unroll
        for (int i = 0; i < kBwdVec; ++i) v[i].template load<V>(0, src + min(c0 + (i * nt + tid) * V, d - V));
      }
      const F2 w2(wr, wr);
#pragma unroll
      for (int i = 0; i < kBwdVec; ++i) {
        const int c = c0 + (i * nt + tid) * V;
        Words<T, E> o;
#pragma unroll
        for (int q = 0; q < E / 2; ++q) o.set(q, live ? mul2(g[i].pair(q), w2) : F2(0.f, 0.f));
        if (c < d) o.template store<V>(0, dy + row + c);
      }
      if (dw != nullptr) {
        F2 s(0.f, 0.f);
        if (live) {
#pragma unroll
          for (int i = 0; i < kBwdVec; ++i) {
            if (c0 + (i * nt + tid) * V >= d) break;
#pragma unroll
            for (int q = 0; q < E / 2; ++q) s = fma2(g[i].pair(q), v[i].pair(q), s);
          }
        }
        const float r = warp_sum(sum2(s));
        if (lane == 0) sh[warp][j] = c0 ? sh[warp][j] + r : r;
      }
    }
  }
  if (dw == nullptr) return;
  __syncthreads();
  if (tid < k) {
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += sh[i][tid];
    dw[t * k + tid] = s;
  }
}

// ---- rows of any alignment, in 32-bit words: one fp32 element, or two 16-bit ones.
// A row of 16-bit elements may start in the middle of a word.  Its word c (of d / 2 +
// 1) is then elements 2c - 1 and 2c, else 2c and 2c + 1, so that whole words are
// stored; its first and last may hold one element only.  A thread takes kWordsEach
// words, a block apart, so that the lookups of a row's places serve them all.
constexpr int kWordsEach = 4;

// A word as it is loaded: whole, or its two elements apart (the parts are joined
// when the word is used, so that many loads can be under way).
struct RawWord {
  uint32_t lo, hi;
  __device__ __forceinline__ uint32_t join() const { return lo | (hi << 16); }
};
// The word at p; EDGE: only the elements that lo / hi say there are, the others 0.
// `whole`: p is aligned to words.
template <typename T, bool EDGE>
__device__ __forceinline__ RawWord load_word(const T* p, bool whole, bool lo, bool hi) {
  RawWord r{0u, 0u};
  if constexpr (sizeof(T) == 4) {
    if (!EDGE || lo) r.lo = gload(reinterpret_cast<const uint32_t*>(p));
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    if (EDGE || !whole) {
      if (!EDGE || lo) r.lo = gload(h);
      if (!EDGE || hi) r.hi = gload(h + 1);
    } else {
      r.lo = gload(reinterpret_cast<const uint32_t*>(p));
    }
  }
  return r;
}
// The same with 16-bit elements always one by one, without a branch on how p lies.
// Where rows differ in it and stores lie between the loads (the gradient) that took
// 291 us against 388 (4096 tokens, k = 8, d = 7166 or 7167, 16 bit); the unpermute,
// which has only loads, branches (147 us, not 171, at 7166).
template <typename T, bool EDGE>
__device__ __forceinline__ RawWord load_apart(const T* p, bool lo, bool hi) {
  RawWord r{0u, 0u};
  if constexpr (sizeof(T) == 4) {
    if (!EDGE || lo) r.lo = gload(reinterpret_cast<const uint32_t*>(p));
  } else {
    gload_pair(p, !EDGE || lo, !EDGE || hi, r.lo, r.hi);
  }
  return r;
}
template <typename T, bool EDGE>
__device__ __forceinline__ void store_word(T* p, uint32_t w, bool lo, bool hi) {
  if constexpr (!EDGE || sizeof(T) == 4) {
    if (!EDGE || lo) *reinterpret_cast<uint32_t*>(p) = w;
  } else {
    uint16_t* h = reinterpret_cast<uint16_t*>(p);
    if (lo) h[0] = (uint16_t)w;
    if (hi) h[1] = (uint16_t)(w >> 16);
  }
}
template <typename T>
__device__ __forceinline__ F2 word_f32(uint32_t w) {
  if constexpr (sizeof(T) == 4) return F2(__uint_as_float(w), 0.f);
  else return pair_f32<T>(&w);
}
template <typename T>
__device__ __forceinline__ uint32_t f32_word(F2 v) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(v.get().x);
  } else {
    uint32_t w;
    pair_to<T>(&w, v);
    return w;
  }
}
constexpr __host__ __device__ int words_of(int d, size_t es) { return es == 4 ? d : d / 2 + 1; }
// Whether the row at p starts in the middle of a word.
template <typename T>
__device__ __forceinline__ int half_word(const T* p) {
  return sizeof(T) == 4 ? 0 : (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1;
}
// The source elements around word c of a row: pairs (2c, 2c + 1) and (2c - 1, 2c).
template <typename T>
struct Around {
  uint32_t even, odd;
  __device__ __forceinline__ void load(const T* row, int c, int d) {
    if constexpr (sizeof(T) == 4) {
      even = odd = c < d ? gload(reinterpret_cast<const uint32_t*>(row + c)) : 0u;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(row) + 2 * c;
      const uint32_t m = c > 0 && 2 * c - 1 < d ? gload(h - 1) : 0u;
      const uint32_t a = 2 * c < d ? gload(h) : 0u, b = 2 * c + 1 < d ? gload(h + 1) : 0u;
      even = a | (b << 16);
      odd = m | (a << 16);
    }
  }
};
// Whether a thread's words c0, c0 + stride, ... (kWordsEach of n) are inner ones,
// both of whose elements exist however the row lies; f(true_type or false_type) for
// words at the edges or not.
template <typename F>
__device__ __forceinline__ void at_edges(int c0, int stride, int n, size_t es, F f) {
  const bool inner = es == 4 ? c0 + (kWordsEach - 1) * stride < n : c0 > 0 && c0 + (kWordsEach - 1) * stride < n - 1;
  if (inner) f(std::false_type());
  else f(std::true_type());
}

template <typename T>
__global__ void __launch_bounds__(256) permute_words_kernel(const T* __restrict__ x, int64_t ldx,
                                                            const int* __restrict__ inv,
                                                            const int* __restrict__ kept_p, int k, int d,
                                                            int64_t tokens, Lay lay, T* __restrict__ xp) {
  constexpr int E = 4 / sizeof(T);
  ops_begin();
  int64_t t;
  int c0;
  if (!lay_at(lay, tokens, t, c0)) return;
  const int kept = gload(kept_p), n = words_of(d, sizeof(T));
  const int* pi = inv + t * k;
  Around<T> v[kWordsEach];
#pragma unroll
  for (int u = 0; u < kWordsEach; ++u) v[u].load(x + t * ldx, c0 + u * lay.nv, d);
  at_edges(c0, lay.nv, n, sizeof(T), [&](auto edge) {
    constexpr bool EDGE = decltype(edge)::value;
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      const int p = gload(pi + j);
      const bool live = p < kept;
      T* row = xp + (int64_t)p * d;
      const int a = half_word(row), e0 = c0 * E - a;
      T* dst = row + e0;
#pragma unroll
      for (int u = 0; u < kWordsEach; ++u) {
        const int e = e0 + u * lay.nv * E;
        store_word<T, EDGE>(dst + u * lay.nv * E, live ? (a ? v[u].odd : v[u].even) : 0u, e >= 0 && e < d, e + 1 < d);
      }
    }
  });
}

template <typename T>
__global__ void __launch_bounds__(256) unpermute_words_kernel(const T* __restrict__ y, const float* __restrict__ w,
                                                              const int* __restrict__ inv,
                                                              const int* __restrict__ kept_p, int k, int d,
                                                              int64_t tokens, Lay lay, const T* base, int64_t ldbase,
                                                              T* out, int64_t ldout) {
  constexpr int E = 4 / sizeof(T);
  ops_begin();
  int64_t t;
  int c0;
  if (!lay_at(lay, tokens, t, c0)) return;
  const int kept = gload(kept_p), n = words_of(d, sizeof(T)), stride = lay.nv * E;
  const int* pi = inv + t * k;
  const float* pw = w + t * k;
  T* row = out + t * ldout;
  const int e0 = c0 * E - half_word(row);
  const T* spare = kept > 0 ? y : row;  // d elements that can be read and are not used
  at_edges(c0, lay.nv, n, sizeof(T), [&](auto edge) {
    constexpr bool EDGE = decltype(edge)::value;
    auto lo = [&](int u) { return e0 + u * stride >= 0 && e0 + u * stride < d; };
    auto hi = [&](int u) { return e0 + u * stride + 1 < d; };
    F2 s[kWordsEach];
#pragma unroll
    for (int u = 0; u < kWordsEach; ++u) s[u] = F2(0.f, 0.f);
    if (base != nullptr) {
      const T* src = base + t * ldbase + e0;
#pragma unroll
      for (int u = 0; u < kWordsEach; ++u)
        s[u] = word_f32<T>(load_word<T, EDGE>(src + u * stride, !half_word(src), lo(u), hi(u)).join());
    }
    for (int j0 = 0; j0 < k; j0 += 4) {  // four rows' words under way
      RawWord v[4][kWordsEach];
      float wj[4];
      bool live[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // (not behind whether the row was dropped: its words are then spare ones)
        const int jq = min(j0 + q, k - 1), p = gload(pi + jq);
        live[q] = j0 + q < k && p < kept;
        wj[q] = w ? gload(pw + jq) : 1.f;
        const T* src = (live[q] ? y + (int64_t)p * d : spare) + e0;
        const bool whole = !half_word(src);
#pragma unroll
        for (int u = 0; u < kWordsEach; ++u) v[q][u] = load_word<T, EDGE>(src + u * stride, whole, lo(u), hi(u));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const F2 ww(wj[q], wj[q]);
#pragma unroll
        for (int u = 0; u < kWordsEach; ++u)
          if (live[q]) s[u] = fma2(ww, word_f32<T>(v[q][u].join()), s[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kWordsEach; ++u)
      store_word<T, EDGE>(row + e0 + u * stride, f32_word<T>(s[u]), lo(u), hi(u));
  });
}

template <typename T>
__global__ void __launch_bounds__(kBwdThreads, 2) unpermute_backward_words_kernel(
    const T* __restrict__ dout, int64_t lddout, const T* __restrict__ y, const float* __restrict__ w,
    const int* __restrict__ inv, const int* __restrict__ kept_p, int k, int d, T* __restrict__ dy,
    float* __restrict__ dw) {
  constexpr int E = 4 / sizeof(T);
  __shared__ float sh[kBwdThreads / 32][kMaxK];
  ops_begin();
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int kept = gload(kept_p), n = words_of(d, sizeof(T)), stride = nt * E;
  const T* spare = kept > 0 ? y : dout + t * lddout;  // d elements that can be read and are not used
  const int* pi = inv + t * k;
  const float* pw = w + t * k;
  for (int b0 = 0; b0 < n; b0 += nt * kWordsEach) {
    const int c0 = b0 + tid;
    Around<T> g[kWordsEach];
#pragma unroll
    for (int u = 0; u < kWordsEach; ++u) g[u].load(dout + t * lddout, c0 + u * nt, d);
#pragma unroll 2
    for (int j = 0; j < k; ++j) {
      const int p = gload(pi + j);
      const bool live = p < kept;
      const float wj = w ? gload(pw + j) : 1.f, wr = live ? wj : 0.f;
      const F2 w2(wr, wr);
      T* row = dy + (int64_t)p * d;
      const int a = half_word(row), e0 = c0 * E - a;
      const T* src = (live ? y + (int64_t)p * d : spare) + e0;
      F2 s(0.f, 0.f);
      at_edges(c0, nt, n, sizeof(T), [&](auto edge) {
        constexpr bool EDGE = decltype(edge)::value;
        auto lo = [&](int u) { return e0 + u * stride >= 0 && e0 + u * stride < d; };
        auto hi = [&](int u) { return e0 + u * stride + 1 < d; };
        RawWord v[kWordsEach];
#pragma unroll
        for (int u = 0; u < kWordsEach; ++u) v[u] = RawWord{0u, 0u};
        if (dw != nullptr) {
#pragma unroll
          for (int u = 0; u < kWordsEach; ++u) v[u] = load_apart<T, EDGE>(src + u * stride, lo(u), hi(u));
        }
#pragma unroll
        for (int u = 0; u < kWordsEach; ++u) {
          const F2 gu = word_f32<T>(a ? g[u].odd : g[u].even);
          store_word<T, EDGE>(row + e0 + u * stride, live ? f32_word<T>(mul2(gu, w2)) : 0u, lo(u), hi(u));
          s = fma2(gu, word_f32<T>(v[u].join()), s);
        }
      });
      if (dw != nullptr) {
        const float r = live ? warp_sum(sum2(s)) : 0.f;
        if (lane == 0) sh[warp][j] = b0 ? sh[warp][j] + r : r;
      }
    }
  }
  if (dw == nullptr) return;
  __syncthreads();
  if (tid < k) {
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += sh[i][tid];
    dw[t * k + tid] = s;
  }
}

// Whether rows are whole 16-byte vectors: bits is the or of addresses and row
// strides in bytes.
bool pm_vec(size_t es, int d, uintptr_t bits) { return (bits | (uintptr_t)d * es) % 16 == 0; }
uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

struct LayLaunch {
  Lay lay;
  int threads;
  int64_t blocks;
};
// n units of a row, `each` a thread: a token's lay.nv threads take unit c, c + nv, ...
LayLaunch pm_lay(int64_t T, int n, int each) {
  LayLaunch l;
  const int need = (n + each - 1) / each;
  l.lay.chunks = (need + 255) / 256;
  l.lay.nv = need;
  l.lay.tpb = l.lay.chunks > 1 ? 1 : 256 / need;
  if (l.lay.tpb > T) l.lay.tpb = (int)T;
  l.threads = ((l.lay.chunks > 1 ? (need + l.lay.chunks - 1) / l.lay.chunks : need * l.lay.tpb) + 31) / 32 * 32;
  l.blocks = l.lay.chunks > 1 ? T * l.lay.chunks : (T + l.lay.tpb - 1) / l.lay.tpb;
  return l;
}

bool pm_args(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E) {
  return dtype_valid(dtype) && T >= 0 && d >= 1 && d <= (1 << 24) && k >= 1 && k <= kMaxK && E >= 1 && E <= kMaxE &&
         T <= (((int64_t)1 << 28) / k);
}

bool sort_args(int64_t R, int32_t E) { return R >= 0 && R <= ((int64_t)1 << 28) && E >= 1 && E <= kMaxE; }
int64_t sort_blocks(int64_t R) { return (R + kSortBlockRows - 1) / kSortBlockRows; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_sort_workspace_bytes(int64_t R, int32_t E) {
  if (!sort_args(R, E)) return 0;
  return ((size_t)(sort_blocks(R) + 2) * (E + 1) * sizeof(int) + 127) / 128 * 128;
}

moe_status moe_sort_rows(const int32_t* ids, int64_t R, int32_t E, int32_t* counts, int32_t* offsets,
                         int32_t* perm, int32_t* inv, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!sort_args(R, E) || !elem_ok(counts, 4) || !elem_ok(offsets, 4) || ws == nullptr || !aligned_to(ws, 128))
    return MOE_ERR_INVALID_ARG;
  if (R > 0 && (!elem_ok(ids, 4) || !elem_ok(perm, 4) || !elem_ok(inv, 4))) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_sort_workspace_bytes(R, E)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // one block up to 1024 rows, one cluster of 8 up to 65536, else a histogram, its
  // scan and a block for every 8192 rows
  const bool big = R > (int64_t)kSortCluster * kSortBlockRows, cluster = !big && R > 1024;
  const int64_t share = big ? kSortBlockRows : cluster ? (R + kSortCluster - 1) / kSortCluster : R;
  const int groups = (int)((share + 31) / 32);
  const int W = groups < 1 ? 1 : groups < 32 ? groups : 32;
  const int per_block = (groups + W - 1) / W * W * 32;
  const int threads = W * 32 > E ? W * 32 : (E + 31) / 32 * 32;
  const size_t smem = (size_t)(W + 2) * (E + 1) * sizeof(int);
  int* hist = static_cast<int*>(ws);
  cudaError_t e = cudaSuccess;
  if (cluster) {
    auto kern = sort_kernel<true>;
    static SmemAllowed allowed;
    e = allow_smem(kern, smem, allowed);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSortCluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    TraceScope ts("sort_rows", st);
    if (e == cudaSuccess)
      e = cudaLaunchKernelEx(&cfg, kern, (const int*)ids, R, (int)E, W, per_block, (const int*)nullptr,
                             (const int*)nullptr, (int*)counts, (int*)offsets, (int*)perm, (int*)inv);
    return ops_status(e);
  }
  const int blocks = big ? (int)sort_blocks(R) : 1;
  int* total = hist + (size_t)blocks * (E + 1);
  if (big) {
    e = launch_ops("sort_hist", sort_hist_kernel, dim3(blocks), dim3(1024), 0, st, ids, R, E, hist);
    if (e == cudaSuccess)
      e = launch_ops("sort_scan", sort_scan_kernel, dim3((E + 1 + 31) / 32), dim3(1024), 0, st, hist, blocks, E + 1,
                     total);
  }
  auto kern = sort_kernel<false>;
  static SmemAllowed allowed;
  if (e == cudaSuccess) e = allow_smem(kern, smem, allowed);
  if (e == cudaSuccess)
    e = launch_ops("sort_rows", kern, dim3(blocks), dim3(threads), smem, st, ids, R, E, W, per_block,
                   big ? hist : nullptr, big ? total : nullptr, counts, offsets, perm, inv);
  return ops_status(e);
}

moe_status moe_permute(int32_t dtype, int64_t T, int32_t d, int32_t k, int32_t E, const void* x, int64_t ldx,
                       const int32_t* inv, const int32_t* offsets, void* xp, moe_stream_t stream) {
  if (!pm_args(dtype, T, d, k, E) || ldx < d) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const size_t es = dtype_bytes(dtype);
  if (!elem_ok(x, es) || !elem_ok(xp, es) || !elem_ok(inv, 4) || !elem_ok(offsets, 4)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = pm_vec(es, d, addr(x) | addr(xp) | (uintptr_t)(ldx * es));
  return ops_status(with_dtype(dtype, [&](auto t) {
    using U = decltype(t);
    constexpr int V = 16 / sizeof(U);
    const LayLaunch l = vec ? pm_lay(T, d / V, 1) : pm_lay(T, words_of(d, es), kWordsEach);
    return launch_ops("permute", vec ? permute_kernel<U, V> : permute_words_kernel<U>, dim3((unsigned)l.blocks),
                      dim3(l.threads), 0, st, static_cast<const U*>(x), ldx, inv, offsets + E, k, d, T, l.lay,
                      static_cast<U*>(xp));
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
  const bool vec = pm_vec(es, d, addr(y) | addr(out) | (uintptr_t)(ldout * es) | addr(base) |
                                     (uintptr_t)((base ? ldbase : 0) * es));
  return ops_status(with_dtype(dtype, [&](auto t) {
    using U = decltype(t);
    constexpr int V = 16 / sizeof(U);
    const LayLaunch l = vec ? pm_lay(T, d / V, 1) : pm_lay(T, words_of(d, es), kWordsEach);
    return launch_ops("unpermute", vec ? unpermute_kernel<U, V> : unpermute_words_kernel<U>, dim3((unsigned)l.blocks),
                      dim3(l.threads), 0, st, static_cast<const U*>(y), w, inv, offsets + E, k, d, T, l.lay,
                      static_cast<const U*>(base), ldbase, static_cast<U*>(out), ldout);
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
  const bool vec = pm_vec(es, d, addr(dout) | (uintptr_t)(lddout * es) | addr(dy) | (dw ? addr(y) : 0));
  return ops_status(with_dtype(dtype, [&](auto t) {
    using U = decltype(t);
    constexpr int V = 16 / sizeof(U);
    const int need = vec ? (d / V + kBwdVec - 1) / kBwdVec : (words_of(d, es) + kWordsEach - 1) / kWordsEach;
    const int threads = need < kBwdThreads ? (need + 31) / 32 * 32 : kBwdThreads;
    return launch_ops("unpermute_backward", vec ? unpermute_backward_kernel<U, V> : unpermute_backward_words_kernel<U>,
                      dim3((unsigned)T), dim3(threads), 0, st, static_cast<const U*>(dout), lddout,
                      static_cast<const U*>(y), w, inv, offsets + E, k, d, static_cast<U*>(dy), dw);
  }));
}

}  // extern "C"

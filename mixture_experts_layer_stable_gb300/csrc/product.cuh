// product.cuh -- the experts' products: a call's arguments, the numbering of its units of
// work, and the choice of the kernel (product_tc.cuh).
#pragma once

#include "ops_common.cuh"

namespace moe {

constexpr int kMaxG = 1024;

enum ProdForm { PROD_ROWS, PROD_ROWS_T, PROD_DW };  // x w, x w^T, x^T dy

struct ProdArgs {
  const int* off;  // [G + 1], or NULL: one expert with all rows
  const void* a;   // rows x
  const void* b;   // weights, or rows dy
  void* out;
  int64_t lda, ldb, ldo;  // row strides (ldb: of dy, or of a weight matrix)
  int* status;
  int rows, G, K, N;
  int odt;         // type of out
  int accumulate;
  void* ws;        // partial sums
  int splits;      // parts of the contraction, 1: out is the result; else partial sums of
  int64_t split_stride;  // this many floats each
};

// Rows and units of each expert, numbered by the block: s_off [G + 1] first rows, s_unit
// [G + 1] first units; an expert has `per` units for each tile of up to `tile` rows, or
// `per` whatever its rows (tile 0).  (Offsets out of order or range give wrong rows, not
// accesses out of range.)  Returns, in the first warp, the rows of the expert with the
// most and the average of those that have some; ends with a barrier.
__device__ __forceinline__ int2 number_units(const ProdArgs& p, int tile, int per, int* s_off, int* s_unit) {
  int most = 0, average = 0;
  for (int i = threadIdx.x; i <= p.G; i += blockDim.x)
    s_off[i] = p.off ? min(max(gload(p.off + i), 0), p.rows) : (i ? p.rows : 0);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0, with = 0;
    for (int base = 0; base < p.G; base += 32) {
      const int e = base + lane;
      const int c = e < p.G ? max(0, s_off[e + 1] - s_off[e]) : 0;
      most = max(most, c);
      with += __popc(__ballot_sync(0xffffffffu, c > 0));
      const int mine = e < p.G ? (tile ? (c + tile - 1) / tile * per : per) : 0;
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (e < p.G) s_unit[e] = run + inc - mine;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) s_unit[p.G] = run;
    most = __reduce_max_sync(0xffffffffu, most);
    average = with ? max(0, s_off[p.G] - s_off[0]) / with : 0;
  }
  __syncthreads();
  return make_int2(most, average);
}

// Expert of unit u: e with s_unit[e] <= u < s_unit[e + 1]; `at` is a first guess.
__device__ __forceinline__ int expert_of(const int* s_unit, int G, int u, int at) {
  if (u >= s_unit[at] && u < s_unit[at + 1]) return at;
  int lo = 0, hi = G - 1;  // the last e with s_unit[e] <= u (experts without units have none)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s_unit[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// How a call runs: tensor copies, the same by CTA pairs, plain loads, plain loads of fp32 operands
enum TcMode { TC_COPY, TC_PAIR, TC_LOAD, TC_SPLIT };
constexpr bool loads(TcMode mode) { return mode == TC_LOAD || mode == TC_SPLIT; }
constexpr int kBlkM = 128, kBlkK = 64;  // output columns of a CTA's tile, contraction of a stage
// Output rows of a tile at most.  (With loading warps an SM's registers hold the sums of
// half as many.)
constexpr int tile_most(TcMode mode, bool f32) { return loads(mode) && f32 ? 128 : 256; }

inline bool takes_pairs(int64_t rows, int N, int G) { return N > kBlkM && rows >= 64 * (int64_t)G; }

// Units of a call at most.
inline int64_t units_of(ProdForm form, TcMode mode, bool f32, int64_t rows, int K, int N, int G) {
  const int tile = tile_most(mode, f32), cols = mode == TC_PAIR ? 2 * kBlkM : kBlkM;
  const int64_t tiles = form == PROD_DW ? (int64_t)((K + tile - 1) / tile) * G : rows / tile + (G < rows ? G : rows);
  return tiles * ((N + cols - 1) / cols);
}

// Parts that the contraction is cut into, their sums joined by a second kernel: as many as
// leave every worker a unit where there are at most half as many units as workers, of four
// stages at least.  (8 bf16 rows, 7168 to 256, two tiles: 29 us whole, 16 in parts; 3636
// rows' gradient of 84 columns through 6373, 15 tiles of unaligned rows: 47 us in parts.)
constexpr int kSplitStages = 16;  // shorter contractions stay whole
inline int splits_of(ProdForm form, TcMode mode, int64_t rows, int K, int N, int G) {
  const int64_t units = units_of(form, mode, true, rows, K, N, G), workers = mode == TC_PAIR ? num_sms() / 2 : num_sms();
  const int64_t stages = ((form == PROD_DW ? rows / G : K) + kBlkK - 1) / kBlkK;
  if (units < 1 || 2 * units > workers || stages < kSplitStages) return 1;
  const int64_t most = stages / 4, want = workers / units;
  return (int)(want < most ? want : most);
}
inline int64_t results_of(ProdForm form, int64_t rows, int K, int N, int G) {
  return form == PROD_DW ? (int64_t)G * K * N : rows * N;
}

cudaError_t launch_product_rows(int dtype, const ProdArgs& p, cudaStream_t st);
cudaError_t launch_product_rows_t(int dtype, const ProdArgs& p, cudaStream_t st);
cudaError_t launch_product_dw(int dtype, const ProdArgs& p, cudaStream_t st);

}  // namespace moe

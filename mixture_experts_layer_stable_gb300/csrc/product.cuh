// product.cuh -- what the two kernels of the experts' products share: the call's
// arguments and the numbering of its units of work.
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
};

// Rows and units of each expert, numbered by the block: s_off [G + 1] first rows, s_unit
// [G + 1] first units; an expert has per units for each tile of `tile` rows, or `per`
// whatever its rows (tile 0).  (Offsets out of order or range give wrong rows, not
// accesses out of range.)  Ends with a barrier.
__device__ __forceinline__ void number_units(const ProdArgs& p, int tile, int per, int* s_off, int* s_unit) {
  for (int i = threadIdx.x; i <= p.G; i += blockDim.x)
    s_off[i] = p.off ? min(max(gload(p.off + i), 0), p.rows) : (i ? p.rows : 0);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0;
    for (int base = 0; base < p.G; base += 32) {
      const int e = base + lane;
      const int c = e < p.G ? max(0, s_off[e + 1] - s_off[e]) : 0;
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
  }
  __syncthreads();
}

// Units of a call at most, for D tiles of bm x bn.
inline int64_t most_units(ProdForm form, const ProdArgs& p, int bm, int bn) {
  const int64_t nt = (p.N + bn - 1) / bn;
  if (form == PROD_DW) return nt * ((p.K + bm - 1) / bm) * p.G;
  return nt * ((int64_t)p.rows / bm + (p.G < p.rows ? p.G : p.rows));
}

// 16-bit operands on the tensor cores (product_tc.cu).
cudaError_t launch_product_tc(ProdForm form, int dtype, const ProdArgs& p, cudaStream_t st);

}  // namespace moe

// product.cu -- the calls of the experts' products and their weights' gradients
// (include/moe_ops.h, moe_grouped_product, moe_grouped_product_dw; the kernel is in
// product_tc.cuh).
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

// (No array has more than 2^40 elements, so units are numbered in 32 bits.)
bool prod_sizes(int64_t rows, int32_t K, int32_t N, int32_t G) {
  constexpr int64_t most = (int64_t)1 << 40;
  return rows >= 0 && rows <= ((int64_t)1 << 28) && K >= 1 && K <= (1 << 22) && N >= 1 && N <= (1 << 22) && G >= 1 &&
         G <= kMaxG && (int64_t)K * N <= most / G && rows <= most / (K > N ? K : N);
}

// The stride of `rows` rows of n: one row's says nothing (and may be past what a tensor map
// holds, or keep it off 16 bytes).
int64_t row_stride(int64_t rows, int64_t ld, int n) { return rows > 1 ? ld : (n + 7) / 8 * 8; }

// Bytes of workspace: a status, and partial sums.
size_t ws_bytes_of(int64_t floats) { return 128 + ((size_t)floats * sizeof(float) + 127) / 128 * 128; }

// What a call needs, however its operands lie.
size_t needed_bytes(ProdForm form, int64_t rows, int K, int N, int G) {
  int splits = 1;
  for (const TcMode mode : {TC_COPY, TC_PAIR, TC_LOAD}) {  // (fp32 operands' tiles are TC_LOAD's)
    if (mode == TC_PAIR && !takes_pairs(rows, N, G)) continue;
    const int s = splits_of(form, mode, rows, K, N, G);
    splits = s > splits ? s : splits;
  }
  return ws_bytes_of(splits > 1 ? splits * results_of(form, rows, K, N, G) : 0);
}

// At least what any call of up to `rows` rows needs.  (One call's need has no order in the
// rows: fewer leave more workers without a unit.)  The parts are at most a quarter of the
// stages, and so many that every worker has one tile at most.
int64_t partials_most(ProdForm form, int64_t rows, int K, int N, int G) {
  const int64_t stages = ((form == PROD_DW ? rows / G : K) + kBlkK - 1) / kBlkK;
  if (stages < kSplitStages) return 0;
  const int64_t tiles = (int64_t)num_sms() * 256 * kBlkM, results = results_of(form, rows, K, N, G);
  return results >= tiles / (stages / 4) ? tiles : results * (stages / 4);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_product_workspace_bytes(int64_t rows, int32_t K, int32_t N, int32_t G) {
  if (!prod_sizes(rows, K, N, G)) return 0;
  // every form, K and N also in each other's place: both orders need the same
  int64_t most = 0;
  for (const ProdForm form : {PROD_ROWS, PROD_ROWS_T, PROD_DW}) {
    const int64_t a = partials_most(form, rows, K, N, G), b = partials_most(form, rows, N, K, G);
    most = most < a ? a : most;
    most = most < b ? b : most;
  }
  return ws_bytes_of(most);
}

moe_status moe_grouped_product(int32_t dtype, int32_t odtype, int64_t rows, int32_t K, int32_t N, int32_t G,
                               const int32_t* offsets, const void* x, int64_t ldx, const void* w, int32_t transposed,
                               void* out, int64_t ldo, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_valid(dtype) || (odtype != dtype && odtype != MOE_DT_F32) || !prod_sizes(rows, K, N, G) || ldx < K ||
      ldo < N || (offsets == nullptr && G != 1) || ws == nullptr || !aligned_to(ws, 128))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < needed_bytes(transposed ? PROD_ROWS_T : PROD_ROWS, rows, K, N, G)) return MOE_ERR_WORKSPACE_TOO_SMALL;
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
  p.lda = row_stride(rows, ldx, K);
  p.ldb = transposed ? K : N;
  p.ldo = row_stride(rows, ldo, N);
  p.status = static_cast<int*>(ws);
  p.ws = static_cast<char*>(ws) + 128;
  p.splits = 1;
  p.rows = (int)rows;
  p.G = G;
  p.K = K;
  p.N = N;
  p.odt = odtype;
  return ops_status(transposed ? launch_product_rows_t(dtype, p, st) : launch_product_rows(dtype, p, st));
}

moe_status moe_grouped_product_dw(int32_t dtype, int32_t wdtype, int64_t rows, int32_t K, int32_t N, int32_t G,
                                  const int32_t* offsets, const void* x, int64_t ldx, const void* dy, int64_t lddy,
                                  void* dw, int32_t accumulate, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!dtype_valid(dtype) || (wdtype != dtype && wdtype != MOE_DT_F32) || !prod_sizes(rows, K, N, G) || ldx < K ||
      lddy < N || (offsets == nullptr && G != 1) || ws == nullptr || !aligned_to(ws, 128))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < needed_bytes(PROD_DW, rows, K, N, G)) return MOE_ERR_WORKSPACE_TOO_SMALL;
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
  p.lda = row_stride(rows, ldx, K);
  p.ldb = row_stride(rows, lddy, N);
  p.ldo = N;
  p.status = static_cast<int*>(ws);
  p.ws = static_cast<char*>(ws) + 128;
  p.splits = 1;
  p.rows = (int)rows;
  p.G = G;
  p.K = K;
  p.N = N;
  p.odt = wdtype;
  p.accumulate = accumulate != 0;
  return ops_status(launch_product_dw(dtype, p, st));
}

}  // extern "C"

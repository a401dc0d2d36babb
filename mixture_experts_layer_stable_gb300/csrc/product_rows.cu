// product_rows.cu -- rows times their expert's weights (product_tc.cuh).
#include "product_tc.cuh"

namespace moe {

cudaError_t launch_product_rows(int dtype, const ProdArgs& p, cudaStream_t st) {
  return p.odt == MOE_DT_F32 ? launch_form<PROD_ROWS, true>(dtype, p, st) : launch_form<PROD_ROWS, false>(dtype, p, st);
}

}  // namespace moe

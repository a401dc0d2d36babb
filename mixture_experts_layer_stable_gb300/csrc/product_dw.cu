// product_dw.cu -- the weights' gradients (product_tc.cuh).
#include "product_tc.cuh"

namespace moe {

cudaError_t launch_product_dw(int dtype, const ProdArgs& p, cudaStream_t st) {
  return p.odt == MOE_DT_F32 ? launch_form<PROD_DW, true>(dtype, p, st) : launch_form<PROD_DW, false>(dtype, p, st);
}

}  // namespace moe

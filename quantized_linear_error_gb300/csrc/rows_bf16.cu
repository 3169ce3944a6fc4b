// The norm and the 8-bit quantiser of rows of bf16.
#include "rows_kernel.cuh"

namespace spear {

spear_status_t rows_launch_bf16(const RowsParams& p, bool norm, int sms, cudaStream_t stream) {
  return norm ? launch_rows<__nv_bfloat16, true>(p, sms, stream) : launch_rows<__nv_bfloat16, false>(p, sms, stream);
}

}  // namespace spear

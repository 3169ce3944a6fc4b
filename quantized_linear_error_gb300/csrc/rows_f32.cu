// The norm and the 8-bit quantiser of rows of f32.
#include "rows_kernel.cuh"

namespace spear {

spear_status_t rows_launch_f32(const RowsParams& p, bool norm, int sms, cudaStream_t stream) {
  return norm ? launch_rows<float, true>(p, sms, stream) : launch_rows<float, false>(p, sms, stream);
}

}  // namespace spear

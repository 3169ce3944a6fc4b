// Rows of a decoder layer: arguments of the norm and the 8-bit quantiser, which rows_bf16.cu, rows_f16.cu and rows_f32.cu
// compile for one element type each.
#pragma once
#include "kv.h"
#include "w8.h"

namespace spear {

struct RowsParams {
  const void* x;
  int64_t ld_x;
  const void* res;  // or null
  int64_t ld_res;
  void* res_out;
  int64_t ld_res_out;
  const void* weight;
  void* y;  // or null
  int64_t ld_y;
  int8_t* q;  // or null
  int64_t ld_q;
  float* scales;
  int M, K;
  float eps;
  int res_f32, weight_f32;
  int vec_x, vec_res, vec_res_out, vec_w, vec_y, vec_q;  // rows may be moved in wide accesses
  int ring;        // rows on their way (of kernels that go through several)
  int staging_at;  // where the warps' shared memory for other stores begins
};

spear_status_t rows_launch_bf16(const RowsParams& p, bool norm, int sms, cudaStream_t stream);
spear_status_t rows_launch_f16(const RowsParams& p, bool norm, int sms, cudaStream_t stream);
spear_status_t rows_launch_f32(const RowsParams& p, bool norm, int sms, cudaStream_t stream);

}  // namespace spear

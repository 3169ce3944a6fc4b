// Rows in 8 bits: the entry points and their checks, and the read-back kernels. (The norm and the quantiser: rows_kernel.cuh.)
#include <atomic>

#include "rows.h"
#include "rows_device.cuh"

namespace spear {
namespace {

spear_status_t launch_rows(const RowsParams& p, bool norm, spear_dtype_t type, cudaStream_t stream) {
  int sms = 0;
  const spear_status_t st = sm_count_of_current(&sms);
  if (st != SPEAR_OK) return st;
  switch (type) {
    case SPEAR_BF16: return rows_launch_bf16(p, norm, sms, stream);
    case SPEAR_F16: return rows_launch_f16(p, norm, sms, stream);
    default: return rows_launch_f32(p, norm, sms, stream);
  }
}

// Values of 16 codes a thread and turn, along the rows. Bound by memory: 12289 x 8192 to bf16 45 us, a plain copy's
// rate (in 16-byte stores, half sectors, 52 us), 12289 x 8191 46. A code's byte (code + 128) under the exponent of 2^23 is 2^23 +
// 128 + code, exactly.
SPEAR_DEVINL void values8(uint32_t lo, uint32_t hi, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __uint_as_float(__byte_perm((j < 4 ? lo : hi) ^ kW8Bias, 0x4B000000u, 0x7440 + (j & 3))) - 8388736.f;
}
constexpr int kTurns = 2;
// 16 values to p, of which n exist; vec: all do and p is 16-byte aligned, 2: 32-byte aligned.
template <class T>
SPEAR_DEVINL void store16(T* p, int n, int vec, const float (&lo)[8], const float (&hi)[8]) {
  if (vec == 2) {
    T e[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) e[j] = rounded<T>(j < 8 ? lo[j] : hi[j - 8]);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      uint32_t w[8];
      memcpy(w, reinterpret_cast<const char*>(e) + 32 * i, 32);
      store32(reinterpret_cast<char*>(p) + 32 * i, w);
    }
  } else {
    store8(p, n, vec, lo);
    store8(p + 8, n - 8, vec, hi);
  }
}
template <class T>
__global__ void __launch_bounds__(256) dequantize_kernel(const int8_t* __restrict__ q, int64_t ld_q,
                                                         const float* __restrict__ scales, int M, int K,
                                                         T* __restrict__ out, int64_t ld_out, int vec) {
  kv_follow();
  const int groups = (K - 1) / 16 + 1;
  uint4 w[kTurns];
  float s[kTurns];
  int64_t row[kTurns];
  int k[kTurns];
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t g = ((int64_t)blockIdx.x * kTurns + i) * 256 + threadIdx.x;
    row[i] = div_u64(g, groups);
    k[i] = (int)(g - row[i] * groups) * 16;
    w[i] = make_uint4(0, 0, 0, 0);
    s[i] = 0.f;
    if (row[i] >= M) continue;
    const int8_t* src = q + row[i] * ld_q + k[i];
    s[i] = scales[row[i]];
    if (vec && K - k[i] >= 16) {
      w[i] = __ldcs(reinterpret_cast<const uint4*>(src));
    } else {
      int8_t c[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) c[j] = j < K - k[i] ? src[j] : (int8_t)0;
      memcpy(&w[i], c, 16);
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    if (row[i] >= M) continue;
    float v[2][8];
    values8(w[i].x, w[i].y, v[0]), values8(w[i].z, w[i].w, v[1]);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j >> 3][j & 7] *= s[i];
    store16(out + row[i] * ld_out + k[i], K - k[i], K - k[i] >= 16 ? vec : 0, v[0], v[1]);
  }
}

// The same where rows follow each other without gaps, as one long row of n elements in wide accesses, whatever K >= 16:
// 16 elements then belong to one row or two.
template <class T>
__global__ void __launch_bounds__(256) dequantize_flat_kernel(const int8_t* __restrict__ q, const float* __restrict__ scales,
                                                              int M, int K, T* __restrict__ out, int vec) {
  kv_follow();
  const int64_t n = (int64_t)M * K;
  uint4 w[kTurns];
  float s[kTurns][2];
  int in[kTurns];  // elements of the first row
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t at = (((int64_t)blockIdx.x * kTurns + i) * 256 + threadIdx.x) * 16;
    w[i] = make_uint4(0, 0, 0, 0);
    if (at >= n) continue;
    const int64_t row = div_u64(at, K);
    in[i] = (int)min((int64_t)16, (row + 1) * K - at);
    s[i][0] = scales[row];
    s[i][1] = in[i] < 16 && row + 1 < M ? scales[row + 1] : 0.f;
    if (at + 16 <= n) {
      w[i] = __ldcs(reinterpret_cast<const uint4*>(q + at));
    } else {
      int8_t c[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) c[j] = at + j < n ? q[at + j] : (int8_t)0;
      memcpy(&w[i], c, 16);
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t at = (((int64_t)blockIdx.x * kTurns + i) * 256 + threadIdx.x) * 16;
    if (at >= n) continue;
    float v[2][8];
    values8(w[i].x, w[i].y, v[0]), values8(w[i].z, w[i].w, v[1]);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j >> 3][j & 7] *= j < in[i] ? s[i][0] : s[i][1];
    store16(out + at, (int)min(n - at, (int64_t)16), at + 16 <= n ? vec : 0, v[0], v[1]);
  }
}

template <class T>
spear_status_t launch_dequantize(bool flat, dim3 grid, cudaStream_t stream, const int8_t* q, int64_t ld_q, const float* scales,
                                 int M, int K, T* out, int64_t ld_out, int vec) {
  return flat ? kv_launch(dequantize_flat_kernel<T>, grid, 256, 0, stream, q, scales, M, K, out, vec)
              : kv_launch(dequantize_kernel<T>, grid, 256, 0, stream, q, ld_q, scales, M, K, out, ld_out, vec);
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(spear_dtype_t t) { return t == SPEAR_BF16 || t == SPEAR_F16 || t == SPEAR_F32; }
unsigned size_of(spear_dtype_t t) { return t == SPEAR_F32 ? 4 : 2; }
// 16-byte accesses of whole groups of eight elements
bool vec_ok(const void* p, int64_t ld, int M, unsigned size) {
  return aligned(p, 16) && (M == 1 || ld * size % 16 == 0);
}
bool rows_ok(const void* p, int64_t ld, int K, unsigned size) { return p && ld >= K && aligned(p, size); }

// Whether rows [M][K] of two arrays (elements of sa and sb bytes) share bytes; the same rows count as apart if `same_ok`.
bool rows_overlap(const void* a, int64_t ld_a, unsigned sa, const void* b, int64_t ld_b, unsigned sb, int M, int K,
                  bool same_ok) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t la = (uintptr_t)ld_a * sa, lb = (uintptr_t)ld_b * sb;
  if (same_ok && a0 == b0 && sa == sb && (la == lb || M == 1)) return false;
  const uintptr_t a1 = a0 + (uintptr_t)(M - 1) * la + (uintptr_t)K * sa, b1 = b0 + (uintptr_t)(M - 1) * lb + (uintptr_t)K * sb;
  if (a1 <= b0 || b1 <= a0) return false;
  if (la != lb) return true;
  // the same distance from row to row: other columns of the same rows are apart
  const uintptr_t d = a0 <= b0 ? (b0 - a0) % la : (a0 - b0) % la;  // of the later one behind a row of the earlier one
  const uintptr_t first = a0 <= b0 ? (uintptr_t)K * sa : (uintptr_t)K * sb, second = a0 <= b0 ? (uintptr_t)K * sb : (uintptr_t)K * sa;
  return d < first || d + second > la;
}

// Whether the bytes from a's first to its last row meet those of b's.
bool extents_meet(const void* a, int64_t ld_a, unsigned sa, int Ma, int Ka, const void* b, int64_t ld_b, unsigned sb,
                  int Mb, int Kb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + (uintptr_t)(Mb - 1) * ld_b * sb + (uintptr_t)Kb * sb &&
         b0 < a0 + (uintptr_t)(Ma - 1) * ld_a * sa + (uintptr_t)Ka * sa;
}

}  // namespace

spear_status_t sm_count_of_current(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEAR_ERR_CUDA;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return SPEAR_OK;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SPEAR_ERR_CUDA;
  if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return SPEAR_OK;
}

}  // namespace spear

using namespace spear;

extern "C" spear_status_t spear_rms_norm(const void* x, int64_t ld_x, spear_dtype_t type, const void* residual,
                                         int64_t ld_residual, void* residual_out, int64_t ld_residual_out,
                                         spear_dtype_t residual_type, const void* weight, spear_dtype_t weight_type,
                                         float eps, int32_t M, int32_t K, void* y, int64_t ld_y, int8_t* q, int64_t ld_q,
                                         float* scales, cudaStream_t stream) {
  if (!type_ok(type) || M < 0 || K < 1 || !(eps >= 0.f && eps < INFINITY)) return SPEAR_ERR_INVALID_ARG;
  if (weight_type != type && weight_type != SPEAR_F32) return SPEAR_ERR_INVALID_ARG;
  const unsigned sx = size_of(type), sw = size_of(weight_type);
  if (!rows_ok(weight, K, K, sw)) return SPEAR_ERR_INVALID_ARG;
  if (M == 1) ld_x = ld_residual = ld_residual_out = ld_y = ld_q = K;  // of no account
  if (M > 0) {
    if (q && scales &&
        (extents_meet(x, ld_x, sx, M, K, scales, 1, 4, M, 1) || extents_meet(weight, K, sw, 1, K, scales, 1, 4, M, 1) ||
         (residual && extents_meet(residual, ld_residual, size_of(residual_type), M, K, scales, 1, 4, M, 1))))
      return SPEAR_ERR_INVALID_ARG;
    if (!rows_ok(x, ld_x, K, sx) || (!y && !q) || (q && (!scales || !aligned(scales, 4) || ld_q < K)) ||
        (y && !rows_ok(y, ld_y, K, sx)))
      return SPEAR_ERR_INVALID_ARG;
    const struct { const void* p; int64_t ld; unsigned s; } in[] = {{x, ld_x, sx}, {residual, ld_residual, size_of(residual_type)}},
        out[] = {{residual ? residual_out : nullptr, ld_residual_out, size_of(residual_type)}, {y, ld_y, sx}, {q, ld_q, 1}};
    if (residual) {
      if ((residual_type != type && residual_type != SPEAR_F32) || !rows_ok(residual, ld_residual, K, in[1].s) ||
          !rows_ok(residual_out, ld_residual_out, K, in[1].s))
        return SPEAR_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 3; ++i) {
      if (!out[i].p) continue;
      if (extents_meet(out[i].p, out[i].ld, out[i].s, M, K, weight, K, sw, 1, K) ||
          (q && extents_meet(out[i].p, out[i].ld, out[i].s, M, K, scales, 1, 4, M, 1)))
        return SPEAR_ERR_INVALID_ARG;
      for (const auto& a : in)
        if (a.p && rows_overlap(out[i].p, out[i].ld, out[i].s, a.p, a.ld, a.s, M, K, true)) return SPEAR_ERR_INVALID_ARG;
      for (int j = 0; j < i; ++j)
        if (out[j].p && rows_overlap(out[i].p, out[i].ld, out[i].s, out[j].p, out[j].ld, out[j].s, M, K, false))
          return SPEAR_ERR_INVALID_ARG;
    }
  }
  if (K > kRowsMaxWidth) return SPEAR_ERR_UNSUPPORTED;
  if (M == 0) return SPEAR_OK;
  RowsParams p = {};
  p.x = x, p.ld_x = ld_x, p.weight = weight, p.y = y, p.ld_y = ld_y, p.q = q, p.ld_q = ld_q, p.scales = scales;
  p.res = residual, p.ld_res = ld_residual, p.res_out = residual_out, p.ld_res_out = ld_residual_out;
  p.M = M, p.K = K, p.eps = eps;
  p.res_f32 = residual_type == SPEAR_F32, p.weight_f32 = weight_type == SPEAR_F32;
  p.vec_x = vec_ok(x, ld_x, M, sx), p.vec_w = aligned(weight, 16), p.vec_y = y && vec_ok(y, ld_y, M, sx);
  p.vec_res = residual && vec_ok(residual, ld_residual, M, size_of(residual_type));
  p.vec_res_out = residual && vec_ok(residual_out, ld_residual_out, M, size_of(residual_type));
  p.vec_q = aligned(q, 8) && (M == 1 || ld_q % 8 == 0);
  return launch_rows(p, true, type, stream);
}

extern "C" spear_status_t spear_quantize_rows(const void* x, int64_t ld_x, spear_dtype_t type, int32_t M, int32_t K,
                                              int8_t* q, int64_t ld_q, float* scales, cudaStream_t stream) {
  if (!type_ok(type) || M < 0 || K < 1) return SPEAR_ERR_INVALID_ARG;
  if (M == 1) ld_x = ld_q = K;  // of no account
  if (M > 0 && (!rows_ok(x, ld_x, K, size_of(type)) || !q || ld_q < K || !scales || !aligned(scales, 4) ||
                rows_overlap(q, ld_q, 1, x, ld_x, size_of(type), M, K, false) ||
                extents_meet(q, ld_q, 1, M, K, scales, 1, 4, M, 1) ||
                extents_meet(x, ld_x, size_of(type), M, K, scales, 1, 4, M, 1)))
    return SPEAR_ERR_INVALID_ARG;
  if (K > kRowsMaxWidth) return SPEAR_ERR_UNSUPPORTED;
  if (M == 0) return SPEAR_OK;
  RowsParams p = {};
  p.x = x, p.ld_x = ld_x, p.q = q, p.ld_q = ld_q, p.scales = scales, p.M = M, p.K = K;
  p.vec_x = vec_ok(x, ld_x, M, size_of(type)), p.vec_q = aligned(q, 8) && (M == 1 || ld_q % 8 == 0);
  return launch_rows(p, false, type, stream);
}

extern "C" spear_status_t spear_dequantize_rows(const int8_t* q, int64_t ld_q, const float* scales, int32_t M, int32_t K,
                                                void* out, int64_t ld_out, spear_dtype_t type, cudaStream_t stream) {
  if (!type_ok(type) || M < 0 || K < 1) return SPEAR_ERR_INVALID_ARG;
  const unsigned s = size_of(type);
  if (M == 1) ld_q = ld_out = K;  // of no account
  if (M > 0 && (!q || ld_q < K || !scales || !aligned(scales, 4) || !rows_ok(out, ld_out, K, s) ||
                rows_overlap(out, ld_out, s, q, ld_q, 1, M, K, false) ||
                extents_meet(out, ld_out, s, M, K, scales, 1, 4, M, 1)))
    return SPEAR_ERR_INVALID_ARG;
  if (M == 0) return SPEAR_OK;
  const bool wide = vec_ok(out, ld_out, M, s) && vec_ok(q, ld_q, M, 1);
  const bool flat = !wide && K >= 16 && (M == 1 || (ld_q == K && ld_out == K)) && aligned(q, 16) && aligned(out, 16);
  const int vec = !wide && !flat ? 0 : aligned(out, 32) && (flat || M == 1 || ld_out * s % 32 == 0) ? 2 : 1;
  const int64_t groups = flat ? ((int64_t)M * K + 15) / 16 : (int64_t)M * ((K - 1) / 16 + 1);
  const int64_t blocks = (groups + 256 * kTurns - 1) / (256 * kTurns);
  if (blocks > 0x7FFFFFFF) return SPEAR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks);
  switch (type) {
    case SPEAR_BF16: return launch_dequantize(flat, grid, stream, q, ld_q, scales, M, K, static_cast<__nv_bfloat16*>(out), ld_out, vec);
    case SPEAR_F16: return launch_dequantize(flat, grid, stream, q, ld_q, scales, M, K, static_cast<__half*>(out), ld_out, vec);
    default: return launch_dequantize(flat, grid, stream, q, ld_q, scales, M, K, static_cast<float*>(out), ld_out, vec);
  }
}

extern "C" spear_status_t spear_rms_norm_args(const spear_rms_norm_args_t* a) {
  if (!a) return SPEAR_ERR_INVALID_ARG;
  return spear_rms_norm(a->x, a->ld_x, (spear_dtype_t)a->type, a->residual, a->ld_residual, a->residual_out,
                        a->ld_residual_out, (spear_dtype_t)a->residual_type, a->weight, (spear_dtype_t)a->weight_type, a->eps,
                        a->M, a->K, a->y, a->ld_y, a->q, a->ld_q, a->scales, a->stream);
}

extern "C" spear_status_t spear_quantize_rows_args(const spear_quantize_rows_args_t* a) {
  if (!a) return SPEAR_ERR_INVALID_ARG;
  return spear_quantize_rows(a->x, a->ld_x, (spear_dtype_t)a->type, a->M, a->K, a->q, a->ld_q, a->scales, a->stream);
}

extern "C" spear_status_t spear_dequantize_rows_args(const spear_dequantize_rows_args_t* a) {
  if (!a) return SPEAR_ERR_INVALID_ARG;
  return spear_dequantize_rows(a->q, a->ld_q, a->scales, a->M, a->K, a->out, a->ld_out, (spear_dtype_t)a->type, a->stream);
}

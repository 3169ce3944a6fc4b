// Rows of a decoder layer between its linears: the root-mean-square norm with
// the residual's addition and an output in 8 bits, the 8-bit quantisation of
// rows, and the read-back.
//
// A row v in 8 bits is codes and one fp32 scale:
//   a = max |v|, scale = a / 127, code = clamp(rint(v * (127 / a)), -127, 127).
// The norm v = h * rstd * w, rstd = 1 / sqrt(mean h^2 + eps), needs the sum of
// squares before anything can be written; the codes need max |v| as well. Since
// rstd > 0 is one factor of the whole row, max |v| = rstd max |h w| and
// v / max |v| = h w / max |h w|: both reductions run over the same registers at
// once, and a row is read once and written once.
//
// Bound by memory: a row stays in registers (8 to 32 elements a thread) between
// the loads and the stores. Measured: 12289 rows of 8192, bf16 with a bf16
// residual, 134 us, 6.0 TB/s or 90% of a plain copy's rate; with an fp32 residual
// and 8 bits 199 us, 83%; 8-bit rows of 12289 x 8192 bf16 48 us, 94%, of 4096 x
// 14336 fp32 47 us, 92%; read back 52 us, 86%. One row 2.4 us, a launch's latency.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kv_device.cuh"
#include "w8_device.cuh"

namespace spear {
namespace {

SPEAR_DEVINL float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Eight elements from p (of which `n` exist) as fp32; `vec`: p is 16-byte aligned and all eight exist.
// kOnce: rows that nobody reads again, out of the caches' way.
template <bool kOnce, class T>
SPEAR_DEVINL void load8(const T* p, int n, bool vec, float (&x)[8]) {
  if (vec) {
    constexpr int words = sizeof(T) / 2;
    uint4 w[words];
#pragma unroll
    for (int i = 0; i < words; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(p) + i;
      w[i] = kOnce ? __ldcs(src) : *src;
    }
    T e[8];
    memcpy(e, w, sizeof(e));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? (float)p[i] : 0.f;
  }
}

template <class T>
SPEAR_DEVINL T rounded(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

template <class T>
SPEAR_DEVINL void store8(T* p, int n, bool vec, const float (&x)[8]) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = rounded<T>(x[i]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      uint4 w;
      memcpy(&w, reinterpret_cast<const char*>(e) + 16 * i, 16);
      *(reinterpret_cast<uint4*>(p) + i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
}

// Eight elements from k on of a row of K, by every lane of a warp, lane i + 1 the next eight behind lane i's. fp32 ones
// are 32 bytes a lane: neighbours trade halves, so that each instruction writes whole sectors.
template <class T>
SPEAR_DEVINL void put8(T* row, int k, int K, bool vec, const float (&x)[8]) {
  if (sizeof(T) == 4 && vec && K % 8 == 0) {
    const bool odd = threadIdx.x & 1;
    float4 own, got;
    float* g = &got.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = __shfl_xor_sync(0xffffffffu, odd ? x[j] : x[4 + j], 1);
    own = odd ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(x[0], x[1], x[2], x[3]);
    const int k0 = k & ~8;  // the pair's first element
    // even lanes: the first halves, of their own eight and of the neighbour's; odd lanes: the second halves
    float4* to = reinterpret_cast<float4*>(row + k0 + (odd ? 4 : 0));
    if (k0 < K) to[0] = odd ? got : own;
    if (k0 + 8 < K) to[2] = odd ? own : got;
  } else if (k < K) {
    store8(row + k, K - k, vec && k + 8 <= K, x);
  }
}

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
  int vec_x, vec_res, vec_res_out, vec_w, vec_y, vec_q;
};

// Sum of a and maximum of b over the row's threads, in every one of them.
template <bool kWarp>
SPEAR_DEVINL void reduce_row(float& a, float& b, float2* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  if (kWarp) return;
  const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
  if (lane == 0) part[threadIdx.x / 32] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  a = v.x, b = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
}

// 16 bytes to a shared address, past the registers.
SPEAR_DEVINL void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
SPEAR_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SPEAR_DEVINL void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <class T>
SPEAR_DEVINL void lds8(uint32_t from, float (&x)[8]) {
  constexpr int words = sizeof(T) / 2;
  uint4 w[words];
#pragma unroll
  for (int i = 0; i < words; ++i) w[i] = lds128(from + 16 * i);
  T e[8];
  memcpy(e, w, sizeof(e));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
}

// How rows are handed out: a warp (K <= 256 NV) or a block a row, or warps or blocks that go through rows of their own
// with the next kRing rows on their way: a thread copies what it will work on to shared memory, so that it waits for
// its own copies alone. Measured, one row after the other / with rows on their way, shares of a plain copy's rate:
// 12289 rows of 8192 with the residual, bf16, 61 / 94%; 8-bit rows of 12289 x 8192 77 / 97%.
enum RowsBy { kWarpRow, kBlockRow, kWarpRows, kBlockRows };
constexpr int kRing = 2, kPartBytes = 3 * 32 * 8;

// NV groups of eight elements a thread, `stride` groups apart.
// R: the residual's type (kWarpRows and kBlockRows; the others ask each time).
template <class T, int NV, bool kNorm, int kBy, class R>
__global__ void __launch_bounds__(kBy == kBlockRow || kBy == kBlockRows ? 1024 : 256) rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr bool kWarp = kBy == kWarpRow || kBy == kWarpRows, kAhead = kBy == kWarpRows || kBy == kBlockRows;
  extern __shared__ __align__(16) uint8_t smem[];
  auto part = reinterpret_cast<float2(*)[32]>(smem);  // [3][32], not for kWarpRow
  kv_follow();
  const int64_t first = kWarp ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  if (first >= p.M) return;  // whole warps, or nobody
  const int at = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
  const int64_t next = kWarp ? (int64_t)gridDim.x * (blockDim.x / 32) : gridDim.x;

  // [stage][word][thread] of 16 bytes: x's words, group after group, then the residual's. The two words of eight fp32
  // elements lie as in the row for a warp's 1 KB, and its lanes copy 512 bytes of it side by side.
  const int words = sizeof(T) / 2 + (kNorm && p.res ? sizeof(R) / 2 : 0);
  const int lane = threadIdx.x & 31;
  const uint32_t step = blockDim.x * 16, ring = smem_u32(smem) + kPartBytes;
  const uint32_t mine = threadIdx.x * 16, mine32 = (threadIdx.x & ~31) * 32 + lane * 32;
  // eight elements from k on of `row`, `size` bytes each, to the words at `to`
  auto copy8 = [&](uint32_t to, const char* row, int k, int size) {
    if (size == 2) {
      if (k < p.K) cp_async16(to + mine, row + (uint32_t)(k * 2));
    } else {
      const int k0 = k - 4 * lane;  // the warp's first element, and this lane's four from there
      to += mine32 - lane * 16;
      const char* src = row + (uint32_t)(k0 * 4);
      if (k0 < p.K) cp_async16(to, src);
      if (k0 + 128 < p.K) cp_async16(to + 512, src + 512);
    }
  };
  auto read8 = [&](uint32_t from, int size, float (&v)[8]) {
    if (size == 4) lds8<float>(from + mine32, v);
    else lds8<T>(from + mine, v);
  };
  const char* const x0 = static_cast<const char*>(p.x);
  const char* const r0 = static_cast<const char*>(p.res);
  auto copy = [&](int64_t row, int stage) {
    if (row < p.M) {
      const char *x = x0 + row * p.ld_x * (int)sizeof(T), *r = r0 + row * p.ld_res * (int)sizeof(R);
      uint32_t to = ring + stage * (NV * words) * step;
#pragma unroll
      for (int i = 0; i < NV; ++i, to += words * step) {
        const int k = (at + i * stride) * 8;  // K is a multiple of 8 here
        copy8(to, x, k, sizeof(T));
        if (kNorm && p.res) copy8(to + sizeof(T) / 2 * step, r, k, sizeof(R));
      }
    }
    cp_async_commit();
  };
  const uint32_t weight_at = ring + kRing * NV * words * step, weight_words = p.weight_f32 ? 2 : sizeof(T) / 2;
  if constexpr (kAhead) {
    if (kNorm)  // the weight's groups behind the ring, for all of the rows
#pragma unroll
      for (int i = 0; i < NV; ++i)
        copy8(weight_at + i * weight_words * step, static_cast<const char*>(p.weight), (at + i * stride) * 8,
              p.weight_f32 ? 4 : sizeof(T));
#pragma unroll
    for (int i = 0; i < kRing; ++i) copy(first + i * next, i);
  }

  float h[NV][8];
  // h w stays in registers beside one or two groups; of more it is made again.
  constexpr bool kHold = kNorm && NV <= 2;
  float hw[kHold ? NV : 1][8];
  auto load_w = [&](int i, float (&w)[8]) {
    const int k = (at + i * stride) * 8;
    if constexpr (kAhead) {
      read8(weight_at + i * weight_words * step, p.weight_f32 ? 4 : sizeof(T), w);
    } else {
      const bool vec = p.vec_w && k + 8 <= p.K;
      if (p.weight_f32) load8<false>(static_cast<const float*>(p.weight) + k, p.K - k, vec, w);
      else load8<false>(static_cast<const T*>(p.weight) + k, p.K - k, vec, w);
    }
  };
  if constexpr (kHold && !kAhead) {  // beside x, not after it
#pragma unroll
    for (int i = 0; i < NV; ++i) load_w(i, hw[i]);
  }
  // h w of group i; `loaded`: w is in hw
  auto weighted = [&](int i, float (&v)[8], bool loaded) {
    if constexpr (kHold && !kAhead) {
      if (loaded) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = hw[i][j];
      } else {
        load_w(i, v);
      }
    } else if constexpr (kNorm) {
      load_w(i, v);
    }
    const bool in = !kAhead || (at + i * stride) * 8 < p.K;  // past the row there may be anything
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = !kNorm ? h[i][j] : in ? v[j] * h[i][j] : 0.f;
  };
  auto statistics = [&](float& ss, float& top, float2* scratch, bool loaded) {
    ss = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
      weighted(i, v, loaded);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (kNorm) ss += h[i][j] * h[i][j];
        if (p.q) top = max_nan(top, fabsf(v[j]));
        if constexpr (kHold) hw[i][j] = v[j];
      }
    }
    reduce_row<kWarp>(ss, top, scratch);
  };
  int stage = 0, turn = 0;
  for (int64_t row = first; row < p.M; row += next) {
    if constexpr (kAhead) {
      cp_async_wait<kRing - 1>();
      __syncwarp();  // what the warp's other lanes have copied
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = (at + i * stride) * 8;
      if constexpr (kAhead) {
        if (k < p.K) read8(ring + (stage * NV + i) * words * step, sizeof(T), h[i]);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      } else {
        load8<true>(static_cast<const T*>(p.x) + row * p.ld_x + k, p.K - k, p.vec_x && k + 8 <= p.K, h[i]);
      }
    }
    if (kNorm && p.res) {
      float r[NV][8];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = (at + i * stride) * 8;
        if constexpr (kAhead) {
          if (k < p.K) read8(ring + ((stage * NV + i) * words + sizeof(T) / 2) * step, sizeof(R), r[i]);
        } else {
          const bool vec = p.vec_res && k + 8 <= p.K;
          if (p.res_f32) load8<true>(static_cast<const float*>(p.res) + row * p.ld_res + k, p.K - k, vec, r[i]);
          else load8<true>(static_cast<const T*>(p.res) + row * p.ld_res + k, p.K - k, vec, r[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = (at + i * stride) * 8;
        if (k < p.K)  // beyond, h stays zero
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[i][j];
        if (kAhead ? sizeof(R) == 4 : p.res_f32) put8(static_cast<float*>(p.res_out) + row * p.ld_res_out, k, p.K, p.vec_res_out, h[i]);
        else put8(static_cast<T*>(p.res_out) + row * p.ld_res_out, k, p.K, p.vec_res_out, h[i]);
      }
    }
    if constexpr (kAhead) {
      __syncwarp();  // all lanes have read the stage
      copy(row + kRing * next, stage);
      if (++stage == kRing) stage = 0;
    }
    float ss, top, rstd = 1.f;
    statistics(ss, top, part[turn], true);  // a thread may still read what the row before left there: two in turn
    turn ^= 1;
    if (kNorm) {
      float eps = p.eps;
      // squares beyond fp32 (the same for the whole row): h times a power of two, which rstd takes back
      if (ss > 0x1p120f || (ss < 0x1p-60f && eps < 0x1p-60f)) {
        const float by = ss > 0x1p120f ? 0x1p-96f : 0x1p80f;
        eps = eps * by * by;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] *= by;
        statistics(ss, top, part[2], false);
        if (!kWarp) __syncthreads();
      }
      rstd = __frsqrt_rn(__fdiv_rn(ss, (float)p.K) + eps);
      if (!(ss < INFINITY)) rstd = NAN;  // an element that is not finite: the whole row
    }
    const float a = kNorm ? top * rstd : top;
    const bool finite = a < INFINITY, held = finite && a >= 0x1p-100f && top >= 0x1p-110f;
    const float inv = held ? __fdiv_rn(127.f, top) : 0.f;
    if (p.q && at == 0) p.scales[row] = held ? __fdiv_rn(a, 127.f) : finite ? 0.f : NAN;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = (at + i * stride) * 8;
      float v[8];
      if constexpr (kHold) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = hw[i][j];
      } else {
        weighted(i, v, false);
      }
      if (p.q) {
        // rint by adding 1.5 * 2^23, whose last byte is the code (|v inv| < 127.5); conversions take four times as long
        uint32_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.f));
        uint2 o;
        o.x = held ? __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410) : 0u;
        o.y = held ? __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410) : 0u;
        int8_t* dst = p.q + row * p.ld_q + k;
        if (p.vec_q && k + 8 <= p.K) {
          *reinterpret_cast<uint2*>(dst) = o;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k + j < p.K) dst[j] = (int8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
        }
      }
      if (kNorm && p.y) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= rstd;
        put8(static_cast<T*>(p.y) + row * p.ld_y, k, p.K, p.vec_y, v);
      }
    }
    if constexpr (!kAhead) break;
  }
}

template <class T, int NV, bool kNorm, bool kWarp>
spear_status_t launch_rows(const RowsParams& p, int sms, int threads, cudaStream_t stream) {
  constexpr int kOne = kWarp ? kWarpRow : kBlockRow, kMany = kWarp ? kWarpRows : kBlockRows;
  const int per = kWarp ? threads / 32 : 1;  // rows of a block at a time
  const int words = sizeof(T) / 2 + (kNorm && p.res ? (p.res_f32 ? 2 : sizeof(T) / 2) : 0);
  const size_t smem = ((size_t)kRing * words + (kNorm ? (p.weight_f32 ? 2 : sizeof(T) / 2) : 0)) * NV * threads * 16 + kPartBytes;
  // Rows that take wide copies, and more than one for each of the blocks that the SMs hold.
  const int blocks = std::min(1024 / threads, (int)(228 * 1024 / (smem + 1024)));  // of an SM
  if (blocks > 0 && p.M > (int64_t)blocks * sms * per && p.K % 8 == 0 && p.vec_x && (!p.res || p.vec_res) &&
      (!kNorm || p.vec_w)) {
    const bool f32 = kNorm && p.res && p.res_f32 && sizeof(T) == 2;
    constexpr void (*kernels[2])(RowsParams) = {
        rows_kernel<T, NV, kNorm, kMany, T>, rows_kernel<T, NV, kNorm, kMany, std::conditional_t<kNorm, float, T>>};
    static std::atomic<uint64_t> configured[2];
    if (smem_limit_once(reinterpret_cast<const void*>(kernels[f32]), configured[f32]) != cudaSuccess) return SPEAR_ERR_CUDA;
    return kv_launch(kernels[f32], dim3(blocks * sms), threads, smem, stream, p);
  }
  return kv_launch(rows_kernel<T, NV, kNorm, kOne, T>, dim3((unsigned)(((int64_t)p.M + per - 1) / per)), threads, kPartBytes,
                   stream, p);
}

template <class T, bool kNorm>
spear_status_t launch_rows(const RowsParams& p, int sms, cudaStream_t stream) {
  const int groups = (p.K + 7) / 8;
  if (groups <= 32) return launch_rows<T, 1, kNorm, true>(p, sms, 256, stream);
  if (groups <= 64) return launch_rows<T, 2, kNorm, true>(p, sms, 256, stream);
  if (groups <= 128) return launch_rows<T, 4, kNorm, true>(p, sms, 256, stream);
  // A block a row: as many threads as it takes where there are few rows, else at most 512, so that two blocks fit an SM.
  const int nv = p.M <= sms ? (groups + 1023) / 1024 : std::min(4, std::max(2, (groups + 511) / 512));
  const int threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
  switch (nv) {
    case 1: return launch_rows<T, 1, kNorm, false>(p, sms, threads, stream);
    case 2: return launch_rows<T, 2, kNorm, false>(p, sms, threads, stream);
    case 3: return launch_rows<T, 3, kNorm, false>(p, sms, threads, stream);
    default: return launch_rows<T, 4, kNorm, false>(p, sms, threads, stream);
  }
}

template <bool kNorm>
spear_status_t launch_rows(const RowsParams& p, spear_dtype_t type, cudaStream_t stream) {
  int sms = 0;
  const spear_status_t st = sm_count_of_current(&sms);
  if (st != SPEAR_OK) return st;
  switch (type) {
    case SPEAR_BF16: return launch_rows<__nv_bfloat16, kNorm>(p, sms, stream);
    case SPEAR_F16: return launch_rows<__half, kNorm>(p, sms, stream);
    default: return launch_rows<float, kNorm>(p, sms, stream);
  }
}

// Values of 16 codes a thread and turn, along the rows. A code's byte (code + 128) under the exponent of 2^23 is 2^23 +
// 128 + code, exactly.
constexpr int kTurns = 2;
template <class T>
__global__ void __launch_bounds__(256) dequantize_kernel(const int8_t* __restrict__ q, int64_t ld_q,
                                                         const float* __restrict__ scales, int M, int K,
                                                         T* __restrict__ out, int64_t ld_out, int vec) {
  kv_follow();
  const int groups = (K + 15) / 16;
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
    if (vec && k[i] + 16 <= K) {
      w[i] = __ldcs(reinterpret_cast<const uint4*>(src));
    } else {
      int8_t c[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) c[j] = k[i] + j < K ? src[j] : (int8_t)0;
      memcpy(&w[i], c, 16);
    }
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    if (row[i] >= M) continue;
    T* dst = out + row[i] * ld_out + k[i];
    const uint32_t c[4] = {w[i].x ^ kW8Bias, w[i].y ^ kW8Bias, w[i].z ^ kW8Bias, w[i].w ^ kW8Bias};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = (__uint_as_float(__byte_perm(c[2 * h + j / 4], 0x4B000000u, 0x7440 + (j & 3))) - 8388736.f) * s[i];
      store8(dst + 8 * h, K - k[i] - 8 * h, vec && k[i] + 16 <= K, v);
    }
  }
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(spear_dtype_t t) { return t == SPEAR_BF16 || t == SPEAR_F16 || t == SPEAR_F32; }
unsigned size_of(spear_dtype_t t) { return t == SPEAR_F32 ? 4 : 2; }
// 16-byte accesses of whole groups of eight elements
int vec_ok(const void* p, int64_t ld, int M, unsigned size) {
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
  return launch_rows<true>(p, type, stream);
}

extern "C" spear_status_t spear_quantize_rows(const void* x, int64_t ld_x, spear_dtype_t type, int32_t M, int32_t K,
                                              int8_t* q, int64_t ld_q, float* scales, cudaStream_t stream) {
  if (!type_ok(type) || M < 0 || K < 1) return SPEAR_ERR_INVALID_ARG;
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
  return launch_rows<false>(p, type, stream);
}

extern "C" spear_status_t spear_dequantize_rows(const int8_t* q, int64_t ld_q, const float* scales, int32_t M, int32_t K,
                                                void* out, int64_t ld_out, spear_dtype_t type, cudaStream_t stream) {
  if (!type_ok(type) || M < 0 || K < 1) return SPEAR_ERR_INVALID_ARG;
  const unsigned s = size_of(type);
  if (M > 0 && (!q || ld_q < K || !scales || !aligned(scales, 4) || !rows_ok(out, ld_out, K, s) ||
                rows_overlap(out, ld_out, s, q, ld_q, 1, M, K, false) ||
                extents_meet(out, ld_out, s, M, K, scales, 1, 4, M, 1)))
    return SPEAR_ERR_INVALID_ARG;
  if (M == 0) return SPEAR_OK;
  const int64_t blocks = ((int64_t)M * ((K + 15) / 16) + 256 * kTurns - 1) / (256 * kTurns);
  if (blocks > 0x7FFFFFFF) return SPEAR_ERR_UNSUPPORTED;
  const int vec = vec_ok(out, ld_out, M, s) && vec_ok(q, ld_q, M, 1);
  const dim3 grid((unsigned)blocks);
  switch (type) {
    case SPEAR_BF16:
      return kv_launch(dequantize_kernel<__nv_bfloat16>, grid, 256, 0, stream, q, ld_q, scales, M, K,
                       static_cast<__nv_bfloat16*>(out), ld_out, vec);
    case SPEAR_F16:
      return kv_launch(dequantize_kernel<__half>, grid, 256, 0, stream, q, ld_q, scales, M, K,
                       static_cast<__half*>(out), ld_out, vec);
    default:
      return kv_launch(dequantize_kernel<float>, grid, 256, 0, stream, q, ld_q, scales, M, K, static_cast<float*>(out),
                       ld_out, vec);
  }
}

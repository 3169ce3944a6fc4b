// Rows of a decoder layer between its linears: the root-mean-square norm with
// the residual's addition and an output in 8 bits, and the 8-bit quantisation of
// rows.
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
// residual, 143 us, 5.6 TB/s or 84% of a plain copy's rate; with an fp32 residual
// and 8 bits 168 us, 98%; 4096 x 14336 bf16 79 us, 89%; 8-bit rows of 12289 x 8192
// bf16 46 us, 98%, of 4096 x 14336 fp32 44 us, 99%. One row of 4096 2.3 us in a graph
// (1.9 without a residual), a launch's latency. Rows that start at any byte are bound
// by the instructions that shift their words: 12289 x 8191 in 8 bits 117 us (39%;
// element by element 24%), the norm of 4096 x 4097 47 us (43%; 20%). More than 16384
// channels: the registers of 1024 threads, 2048 x 28672 109 us, 64%. Four groups a
// thread with the norm spill: up to 296 bytes a thread in the kernels of one row, 84 in
// those of several (wide rows of 16 bits: 24).
#pragma once
#include <algorithm>

#include "rows.h"
#include "rows_device.cuh"

namespace spear {
namespace {

SPEAR_DEVINL float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 bytes from byte `at` (0 .. 15) of two words on.
SPEAR_DEVINL uint4 bytes16(const uint4& a, const uint4& b, uint32_t at) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {  // at / 4 words on
    const uint32_t lo = at & 4 ? w[i + 1 > 7 ? 7 : i + 1] : w[i], hi = at & 4 ? w[i + 3 > 7 ? 7 : i + 3] : w[i + 2];
    v[i] = at & 8 ? hi : lo;
  }
  const uint32_t by = 0x3210u + 0x1111u * (at & 3);
  return make_uint4(__byte_perm(v[0], v[1], by), __byte_perm(v[1], v[2], by), __byte_perm(v[2], v[3], by),
                    __byte_perm(v[3], v[4], by));
}

// 16 bytes of shared memory from any byte on.
SPEAR_DEVINL uint4 lds_bytes16(uint32_t addr) {
  uint32_t w[6];
#pragma unroll
  for (int i = 0; i < 3; ++i)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[2 * i]), "=r"(w[2 * i + 1]) : "r"((addr & ~7u) + 8 * i));
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = addr & 4 ? w[i + 1] : w[i];
  const uint32_t by = 0x3210u + 0x1111u * (addr & 3);
  return make_uint4(__byte_perm(v[0], v[1], by), __byte_perm(v[1], v[2], by), __byte_perm(v[2], v[3], by),
                    __byte_perm(v[3], v[4], by));
}

// Eight elements from p (of which `n` exist) as fp32; `vec`: p is 16-byte aligned and all eight exist. Else the aligned
// words that hold them are read (in full, so up to 15 bytes beside them, too). kOnce: rows that nobody reads again, out
// of the caches' way.
template <bool kOnce, class T>
SPEAR_DEVINL void load8(const T* p, int n, bool vec, float (&x)[8]) {
  constexpr int words = sizeof(T) / 2;
  uint4 w[words];
  if (vec) {
#pragma unroll
    for (int i = 0; i < words; ++i) {
      const uint4* src = reinterpret_cast<const uint4*>(p) + i;
      w[i] = kOnce ? __ldcs(src) : *src;
    }
  } else {
    const uint32_t at = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - at);
    const int bytes = (int)at + min(max(n, 0), 8) * (int)sizeof(T);  // from src on
    uint4 a[words + 1];
#pragma unroll
    for (int i = 0; i <= words; ++i) a[i] = n > 0 && 16 * i < bytes ? src[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < words; ++i) w[i] = bytes16(a[i], a[i + 1], at);
  }
  T e[8];
  memcpy(e, w, sizeof(e));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = vec || i < n ? (float)e[i] : 0.f;
}

// Bytes `at` .. of a row that starts anywhere: what a warp's lanes have, `size` bytes each side by side (16 or 32, or 8
// for codes), of which `bytes` belong to the row, elements of E. Through 1 KB of shared memory, so that all but the first
// and last few bytes go out in aligned words.
constexpr int kStageBytes = 1024 + 32;
template <class E, int kSize>
SPEAR_DEVINL void put_any(char* to, int bytes, uint32_t stage, const uint32_t (&v)[kSize / 4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kSize / 8; ++i)
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(stage + lane * kSize + 8 * i), "r"(v[2 * i]), "r"(v[2 * i + 1]) : "memory");
  __syncwarp();
  constexpr int S = sizeof(E);
  const int head = min(bytes, (int)(-reinterpret_cast<intptr_t>(to) & 15)), words = (bytes - head) / 16, tail = head + 16 * words;
  auto one = [&](int at) {
    if constexpr (S == 4) {
      uint32_t e;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(e) : "r"(stage + at));
      *reinterpret_cast<uint32_t*>(to + at) = e;
    } else if constexpr (S == 2) {
      uint16_t e;
      asm volatile("ld.shared.b16 %0, [%1];" : "=h"(e) : "r"(stage + at));
      *reinterpret_cast<uint16_t*>(to + at) = e;
    } else {
      uint32_t e;
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(stage + at));
      *reinterpret_cast<uint8_t*>(to + at) = (uint8_t)e;
    }
  };
  if (lane * S < head) one(lane * S);
  for (int i = lane; i < words; i += 32)
    *reinterpret_cast<uint4*>(to + head + 16 * i) = lds_bytes16(stage + head + 16 * i);
  if (tail + lane * S < bytes) one(tail + lane * S);
  __syncwarp();
}

// Eight elements from k on of a row of K, by every lane of a warp, lane i + 1 the next eight behind lane i's. fp32 ones
// are 32 bytes a lane: neighbours trade halves, so that each instruction writes whole sectors.
// kAny: rows that take no wide stores (vec false) are possible.
template <bool kAny, class T>
SPEAR_DEVINL void put8(T* row, int k, int K, bool vec, uint32_t stage, const float (&x)[8]) {
  const int lane = threadIdx.x & 31;
  if (kAny && !vec) {
    const int k0 = k - 8 * lane;
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = rounded<T>(x[i]);
    uint32_t v[2 * sizeof(T)];
    memcpy(v, e, sizeof(e));
    if (k0 < K)
      put_any<T, 8 * sizeof(T)>(reinterpret_cast<char*>(row + k0), min(K - k0, 256) * (int)sizeof(T), stage, v);
  } else if (sizeof(T) == 4 && K % 8 == 0) {
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
    store8(row + k, K - k, k + 8 <= K, x);
  }
}

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

// The same from byte `at` (0 .. 15) on.
template <class T>
SPEAR_DEVINL void lds8_any(uint32_t from, uint32_t at, float (&x)[8]) {
  constexpr int words = sizeof(T) / 2;
  uint4 w[words];
  if constexpr (words == 1) {
    w[0] = lds_bytes16(from + at);
  } else {  // 32 bytes a lane: whole words, which meet fewer lanes in a bank
    uint4 a[words + 1];
#pragma unroll
    for (int i = 0; i <= words; ++i) a[i] = lds128(from + 16 * i);
#pragma unroll
    for (int i = 0; i < words; ++i) w[i] = bytes16(a[i], a[i + 1], at);
  }
  T e[8];
  memcpy(e, w, sizeof(e));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)e[i];
}

// How rows are handed out: a warp (K <= 256 NV) or a block a row, or warps or blocks that go through rows of their own
// with the next one or two rows on their way (p.ring): a warp copies what it will work on to shared memory, so that it
// waits for its own copies alone. Measured, one row after the other / with rows on their way, shares of a plain copy's rate:
// 12289 rows of 8192 with the residual, bf16, 61 / 94%; 8-bit rows of 12289 x 8192 77 / 97%.
enum RowsBy { kWarpRow, kBlockRow, kWarpRows, kBlockRows };
constexpr int kPartBytes = 3 * 32 * 8;

// Blocks of eight warps that go through several rows, of an SM: four groups a lane of the norm need more registers (20000
// x 517 with four blocks 70 us, with two 52).
template <int NV, bool kNorm>
constexpr int kWarpBlocks = kNorm && NV == 4 ? 2 : 4;

// NV groups of eight elements a thread, `stride` groups apart.
// R: the residual's type (kWarpRows and kBlockRows; the others ask each time).
// kOdd: rows of any alignment and width (the kernels of one row take them as they come).
template <class T, int NV, bool kNorm, int kBy, class R, bool kOdd>
__global__ void __launch_bounds__(kBy == kBlockRow || kBy == kBlockRows ? 1024 : 256, kBy == kWarpRows ? (kNorm ? 2 : 4) : kBy == kWarpRow ? 4 : 1)
    rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr bool kWarp = kBy == kWarpRow || kBy == kWarpRows, kAhead = kBy == kWarpRows || kBy == kBlockRows, kAny = !kAhead || kOdd;
  extern __shared__ __align__(16) uint8_t smem[];
  auto part = reinterpret_cast<float2(*)[32]>(smem);  // [3][32], not for kWarpRow
  kv_follow();
  const int64_t first = kWarp ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  if (first >= p.M) return;  // whole warps, or nobody
  const int at = kWarp ? threadIdx.x & 31 : threadIdx.x, stride = kWarp ? 32 : blockDim.x;
  const int64_t next = kWarp ? (int64_t)gridDim.x * (blockDim.x / 32) : gridDim.x;

  // [stage][group][x, residual], each a warp's 32 x 8 elements after the other as they lie in the row, which its lanes
  // copy in 16-byte words side by side; a little more where the row does not start at a word (kOdd).
  constexpr int kX = 256 * sizeof(T) + (kOdd ? 32 : 0), kR = 256 * sizeof(R) + (kOdd ? 32 : 0);
  const int lane = threadIdx.x & 31, warps = blockDim.x / 32, warp = threadIdx.x / 32;
  const int group_bytes = (kX + (kNorm && p.res ? kR : 0)) * warps, weight_bytes = 256 * (p.weight_f32 ? 4 : (int)sizeof(T));
  const uint32_t ring = smem_u32(smem) + kPartBytes, weight_at = ring + p.ring * NV * group_bytes;
  const uint32_t staging = smem_u32(smem) + p.staging_at + warp * kStageBytes;
  // the warp's elements from k0 on of `row`, `size` bytes each, to `to`
  auto copy_warp = [&](uint32_t to, const char* row, int k0, int size) {
    if (k0 >= p.K) return;
    const char* src = row + (uint32_t)(k0 * size);
    if (kOdd) {
      const int at = (int)(reinterpret_cast<uintptr_t>(src) & 15), bytes = at + min(p.K - k0, 256) * size;
      src -= at;
      for (int i = 16 * lane; i < bytes; i += 512) cp_async16(to + i, src + i);
    } else {  // K is a multiple of 8
      const int per = 16 / size;
      if (k0 + lane * per < p.K) cp_async16(to + 16 * lane, src + 16 * lane);
      if (size == 4 && k0 + 128 + lane * per < p.K) cp_async16(to + 512 + 16 * lane, src + 512 + 16 * lane);
    }
  };
  // eight elements of this lane; `row`: where they came from
  auto read8 = [&](uint32_t from, const char* row, int size, float (&v)[8]) {
    if (kOdd) {
      const uint32_t at = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15);
      if (size == 4) lds8_any<float>(from + 32 * lane, at, v);
      else lds8_any<T>(from + 16 * lane, at, v);
    } else {
      if (size == 4) lds8<float>(from + 32 * lane, v);
      else lds8<T>(from + 16 * lane, v);
    }
  };
  const char* const x0 = static_cast<const char*>(p.x);
  const char* const r0 = static_cast<const char*>(p.res);
  auto copy = [&](int64_t row, int stage) {
    if (row < p.M) {
      const char *x = x0 + row * p.ld_x * (int)sizeof(T), *r = r0 + row * p.ld_res * (int)sizeof(R);
      uint32_t to = ring + stage * NV * group_bytes;
#pragma unroll
      for (int i = 0; i < NV; ++i, to += group_bytes) {
        const int k0 = (at - lane + i * stride) * 8;
        copy_warp(to + warp * kX, x, k0, sizeof(T));
        if (kNorm && p.res) copy_warp(to + warps * kX + warp * kR, r, k0, sizeof(R));
      }
    }
    cp_async_commit();
  };
  if constexpr (kAhead) {
    if (kNorm)  // the weight's groups behind the ring, for all of the rows; it starts at a word
#pragma unroll
      for (int i = 0; i < NV; ++i)
        copy_warp(weight_at + (i * warps + warp) * weight_bytes, static_cast<const char*>(p.weight), (at - lane + i * stride) * 8,
                  p.weight_f32 ? 4 : sizeof(T));
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < p.ring) copy(first + i * next, i);
  }

  float h[NV][8];
  // h w stays in registers beside one or two groups; of more it is made again.
  constexpr bool kHold = kNorm && NV <= 2;
  float hw[kHold ? NV : 1][8];
  auto load_w = [&](int i, float (&w)[8]) {
    const int k = (at + i * stride) * 8;
    if constexpr (kAhead) {
      if (p.weight_f32) lds8<float>(weight_at + (i * warps + warp) * weight_bytes + 32 * lane, w);
      else lds8<T>(weight_at + (i * warps + warp) * weight_bytes + 16 * lane, w);
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
  // Zeros for what lies past the row (kAhead: there may be anything). Most groups lie within.
  auto inside = [&](int i, float (&v)[8]) {
    if (!kAhead || (at - lane + i * stride) * 8 + 256 <= p.K) return;
    const int n = p.K - (at + i * stride) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (kOdd ? j < n : n > 0) ? v[j] : 0.f;
  };
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
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = kNorm ? v[j] * h[i][j] : h[i][j];
    if constexpr (kNorm) inside(i, v);
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
      if (p.ring == 2) cp_async_wait<1>();
      else cp_async_wait<0>();
      __syncwarp();  // what the warp's other lanes have copied
    }
    auto sum_out = [&](int k, float (&sum)[8]) {
      if (kAhead ? sizeof(R) == 4 : p.res_f32) put8<kAny>(static_cast<float*>(p.res_out) + row * p.ld_res_out, k, p.K, p.vec_res_out, staging, sum);
      else put8<kAny>(static_cast<T*>(p.res_out) + row * p.ld_res_out, k, p.K, p.vec_res_out, staging, sum);
    };
    if constexpr (kAhead) {  // group by group: all of the residual's beside h would not fit the registers
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t from = ring + (stage * NV + i) * group_bytes;
        read8(from + warp * kX, x0 + row * p.ld_x * (int)sizeof(T), sizeof(T), h[i]);
        inside(i, h[i]);
        if (kNorm && p.res) {
          float r[8];
          read8(from + warps * kX + warp * kR, r0 + row * p.ld_res * (int)sizeof(R), sizeof(R), r);
          inside(i, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[j];
          sum_out((at + i * stride) * 8, h[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = (at + i * stride) * 8;
        load8<true>(static_cast<const T*>(p.x) + row * p.ld_x + k, p.K - k, p.vec_x && k + 8 <= p.K, h[i]);
      }
      if (kNorm && p.res) {
        float r[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int k = (at + i * stride) * 8;
          const bool vec = p.vec_res && k + 8 <= p.K;
          if (p.res_f32) load8<true>(static_cast<const float*>(p.res) + row * p.ld_res + k, p.K - k, vec, r[i]);
          else load8<true>(static_cast<const T*>(p.res) + row * p.ld_res + k, p.K - k, vec, r[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += r[i][j];
          sum_out((at + i * stride) * 8, h[i]);
        }
      }
    }
    if constexpr (kAhead) {
      __syncwarp();  // all lanes have read the stage
      copy(row + p.ring * next, stage);
      if (++stage == p.ring) stage = 0;
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
        if (kAny && !p.vec_q) {
          const uint32_t c2[2] = {o.x, o.y};
          const int k0 = k - 8 * lane;
          if (k0 < p.K) put_any<int8_t, 8>(reinterpret_cast<char*>(dst - 8 * lane), min(p.K - k0, 256), staging, c2);
        } else if (k + 8 <= p.K) {
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
        put8<kAny>(static_cast<T*>(p.y) + row * p.ld_y, k, p.K, p.vec_y, staging, v);
      }
    }
    if constexpr (!kAhead) break;
  }
}

template <class T, int NV, bool kNorm, bool kWarp>
spear_status_t launch_rows(RowsParams p, int sms, int threads, cudaStream_t stream) {
  constexpr int kOne = kWarp ? kWarpRow : kBlockRow, kMany = kWarp ? kWarpRows : kBlockRows;
  const int per = kWarp ? threads / 32 : 1;  // rows of a block at a time
  const bool wide = p.vec_x && (!p.y || p.vec_y) && (!p.q || p.vec_q) && (!p.res || (p.vec_res && p.vec_res_out));
  const bool odd = !wide || p.K % 8 != 0, f32 = kNorm && p.res && p.res_f32 && sizeof(T) == 2;
  const size_t more = odd ? 32 : 0, stages = wide ? 0 : (size_t)threads / 32 * kStageBytes;
  const size_t group = 256 * sizeof(T) + more + (kNorm && p.res ? 256 * (p.res_f32 ? 4 : sizeof(T)) + more : 0);
  const size_t weight = kNorm ? 256 * (p.weight_f32 ? 4 : sizeof(T)) : 0, warps = threads / 32;
  auto bytes = [&](int ring) { return (ring * group + weight) * NV * warps + kPartBytes + stages; };
  // More than one row for each of the blocks that the SMs hold. (A block a row with NV = 1: M <= sms.)
  if constexpr (kWarp || NV > 1) {
    const int most = kWarp ? kWarpBlocks<NV, kNorm> : 1024 / threads, room = 227 * 1024;  // blocks of an SM: registers
    p.ring = bytes(2) <= (size_t)room ? 2 : 1;
    const int blocks = std::min(most, (int)((room + 1024) / (bytes(p.ring) + 1024)));
    if (blocks > 0 && p.M > (int64_t)blocks * sms * per && (!kNorm || p.vec_w)) {
      using F = std::conditional_t<kNorm, float, T>;
      constexpr void (*kernels[4])(RowsParams) = {
          rows_kernel<T, NV, kNorm, kMany, T, false>, rows_kernel<T, NV, kNorm, kMany, F, false>,
          rows_kernel<T, NV, kNorm, kMany, T, true>, rows_kernel<T, NV, kNorm, kMany, F, true>};
      static std::atomic<uint64_t> configured[4];
      const int which = 2 * odd + f32;
      if (smem_limit_once(reinterpret_cast<const void*>(kernels[which]), configured[which]) != cudaSuccess) return SPEAR_ERR_CUDA;
      p.staging_at = (int)(bytes(p.ring) - stages);
      return kv_launch(kernels[which], dim3(blocks * sms), threads, bytes(p.ring), stream, p);
    }
  }
  p.staging_at = kPartBytes;
  return kv_launch(rows_kernel<T, NV, kNorm, kOne, T, true>, dim3((unsigned)(((int64_t)p.M + per - 1) / per)), threads,
                   kPartBytes + stages, stream, p);
}

template <class T, bool kNorm>
spear_status_t launch_rows(const RowsParams& p, int sms, cudaStream_t stream) {
  const int groups = (p.K + 7) / 8;
  if (groups <= 32) return launch_rows<T, 1, kNorm, true>(p, sms, 256, stream);
  if (groups <= 64) return launch_rows<T, 2, kNorm, true>(p, sms, 256, stream);
  if (groups <= 128) return launch_rows<T, 4, kNorm, true>(p, sms, 256, stream);
  // A block a row: as many threads as it takes; where there are many rows two groups a thread at least, so that two blocks
  // fit an SM. (Three and four groups a thread spill: norm of 4096 x 11008 in 480 threads 65 us, in 704 59; of 4096 x
  // 14336, bf16, 171 in two blocks of 448, 77 in one with more registers, 79 in one of 896.)
  const int nv = p.M <= sms ? (groups + 1023) / 1024 : std::max(2, (groups + 1023) / 1024);
  const int threads = ((groups + nv - 1) / nv + 31) / 32 * 32;
  switch (nv) {
    case 1: return launch_rows<T, 1, kNorm, false>(p, sms, threads, stream);
    case 2: return launch_rows<T, 2, kNorm, false>(p, sms, threads, stream);
    case 3: return launch_rows<T, 3, kNorm, false>(p, sms, threads, stream);
    default: return launch_rows<T, 4, kNorm, false>(p, sms, threads, stream);
  }
}

}  // namespace
}  // namespace spear

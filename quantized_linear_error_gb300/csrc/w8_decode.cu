// Few tokens (up to 32, or 16 where weights are many) through 8-bit integer
// weights: a kernel that streams the weights once.
//
//   y[m][n] = round(s_x[m] s_w[n] sum_k q_x[m][k] q_w[n][k])
//
// Bound by the weights' bytes. Each warp streams blocks of its own through a
// private ring in shared memory (bulk copies; it waits for nothing but them),
// turns the codes into f16 in registers and feeds warp MMAs whose A operand is
// 16 weight rows and whose columns are 8 tokens. Products of codes and their
// sums below 2^24 are exact in the fp32 accumulators.
//
// A warp takes 4 KB at a time, RS strips of 16 rows by KU blocks of 64 channels,
// so that what a turn costs beside the arithmetic (a wait, copies to issue, the
// tokens' codes) is spread over as much (a token through 14336 x 4096 with 1, 2,
// 4 KB a turn: 19.3, 14.6, 12.5 us); the warps of a CTA take the units of the
// same rows along K in turn, and their sums are added in shared memory in a
// fixed order. Measured: 8 tokens x 28672 x 8192 (235 MB) 38 us, 6.1 TB/s or 91% of
// a plain copy's rate; 16 tokens 41 us, 85%; a token through 4096 x 4096 5.2 us, of
// which the bytes take 2.5 and a launch's latency the rest. From 17 tokens on a unit
// is 2 KB and its tokens' codes are as many as its weights', loaded and converted
// for every two strips anew: 32 tokens through 4096 x 8192 (34 MB) 13.2 us, 38% of
// HBM, with the tensor pipe active 32% of the cycles, the integer pipe 42% and an
// issue slot used 49% by 16 warps, which wait for results of a few cycles and for
// tokens most. (28672 x 8192 63 us; such layers take the other kernel.)
#include <algorithm>

#include "w8_device.cuh"

namespace spear {
namespace {

struct StreamParams {
  const uint8_t* w;
  const float* w_scales;
  const int8_t* x;
  int64_t ld_x;
  const float* x_scales;
  void* y;
  int64_t ld_y;
  float* part;
  unsigned *counters, *status;
  uint64_t wait_ns;
  int type, M, K, N, kq, gated, act;  // kq: units of a row group
  int units, balanced, per;           // units in all; split evenly, or `per` whole row groups a CTA
  int skip_arrive;                    // the first barrier of the first warp expects an arrival that never comes
};

SPEAR_DEVINL void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// First unit of CTA c.
__host__ __device__ inline int range_start(int c, int grid, int units, int balanced, int per, int kq) {
  if (balanced) return (int)((int64_t)c * units / grid);
  const int64_t u = (int64_t)c * per * kq;
  return u < units ? (int)u : units;
}

// MT tiles of 8 tokens, RS strips of 16 rows x KU blocks a unit, NW warps, D units of a warp on their way.
template <int MT, int RS, int KU, int NW, int D>
struct Plan {
  static constexpr int kStage = RS * KU * kW8Block;           // a unit
  static constexpr int kRing = NW * D * kStage;
  static constexpr int kElems = RS * MT * 128;                // sums of a row group
  // a second buffer of the warps' sums, where there is room: one barrier less a row group
  static constexpr int kBufs = kRing + 2 * NW * kElems * 4 + NW * D * 8 + 16 <= 227 * 1024 ? 2 : 1;
  static constexpr int kBars = kRing + kBufs * NW * kElems * 4;
  static constexpr int kSmem = kBars + NW * D * 8 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

template <int MT, int RS, int KU, int NW, int D>
__global__ void __launch_bounds__(NW * 32, 1) stream_kernel(const __grid_constant__ StreamParams p) {
  using P = Plan<MT, RS, KU, NW, D>;
  constexpr int kRuns = RS / 2, kRun = 2 * KU * kW8Block;  // a unit's pairs of strips, and the bytes of one
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u0 = range_start(blockIdx.x, gridDim.x, p.units, p.balanced, p.per, p.kq);
  const int u1 = range_start(blockIdx.x + 1, gridDim.x, p.units, p.balanced, p.per, p.kq);
  uint8_t* ring = smem + warp * D * P::kStage;
  float* red = reinterpret_cast<float*>(smem + P::kRing);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBars) + warp * D;
  volatile int& last = *reinterpret_cast<volatile int*>(smem + P::kSmem - 16);

  grid_launch_dependents();
  // The unit to be copied next: fu = row group fg, unit fk of it; lane i copies its run i.
  const int64_t pair_bytes = (int64_t)p.kq * kRun;  // of a pair of strips
  int fg = u0 / p.kq, fk = u0 - fg * p.kq + warp, fu = u0 + warp, copied = u1;
  while (fk >= p.kq) fk -= p.kq, ++fg;
  auto fetch = [&](int stage) {
    if (fu < copied) {
      if (lane == 0) mbar_arrive_expect_tx(bars + stage, P::kStage);
      if (lane < kRuns)
        bulk_g2s(ring + stage * P::kStage + lane * kRun, p.w + (fg * kRuns + lane) * pair_bytes + (int64_t)fk * kRun, kRun,
                 bars + stage);
    }
    fu += NW, fk += NW;
    while (fk >= p.kq) fk -= p.kq, ++fg;
  };
  uint4 xr[KU][MT];  // of the unit that is worked on next
  int xk = u0 % p.kq + warp;
  while (xk >= p.kq) xk -= p.kq;
  const int8_t* xrow = p.x + g * p.ld_x + t * 16;
  auto fetch_x = [&](int u) {
#pragma unroll
    for (int q = 0; q < KU; ++q) {
      const int k = (xk * KU + q) * kW8K;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        xr[q][j] = make_uint4(0, 0, 0, 0);
        if (u < u1 && j * 8 + g < p.M && k + t * 16 < p.K)  // K is a multiple of 16
          xr[q][j] = *reinterpret_cast<const uint4*>(xrow + j * 8 * p.ld_x + k);
      }
    }
    xk += NW;
    while (xk >= p.kq) xk -= p.kq;
  };
  if (lane == 0) {
#pragma unroll
    for (int d = 0; d < D; ++d) mbar_init(bars + d, d == 0 && warp == 0 && blockIdx.x == 0 && p.skip_arrive ? 2 : 1);
    fence_mbar_init();
  }
  __syncwarp();
#pragma unroll
  for (int d = 0; d < D; ++d) fetch(d);  // the handle's own weights, while the kernel before this one ends
  grid_wait();
  fetch_x(u0 + warp);

  int u = u0 + warp, stage = 0, buf = 0;
  unsigned phase = 0;
  const uint32_t place = w8_place(g, t) * 16;
  for (int seg = u0; seg < u1;) {
    const int group = seg / p.kq, end = min(u1, (group + 1) * p.kq);
    float acc[RS][MT][4];
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][j][i] = 0.f;
    for (; u < end; u += NW) {
      uint32_t b[KU][MT][8];
#pragma unroll
      for (int q = 0; q < KU; ++q)
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          w8_unpack(xr[q][j].x ^ kW8Bias, b[q][j][0], b[q][j][1]);
          w8_unpack(xr[q][j].y ^ kW8Bias, b[q][j][2], b[q][j][3]);
          w8_unpack(xr[q][j].z ^ kW8Bias, b[q][j][4], b[q][j][5]);
          w8_unpack(xr[q][j].w ^ kW8Bias, b[q][j][6], b[q][j][7]);
        }
      fetch_x(u + NW);
      if (u < copied && !__all_sync(0xffffffffu, mbar_wait_bounded(bars + stage, phase, p.wait_ns))) {
        copied = min(copied, fu);  // no further copies; those in flight are still waited for
        if (lane == 0) atomicOr(p.status, kStatusTimeoutPipe);
      }
      // strip r of k block q: run r / 2, [q][r % 2]
      const uint32_t at = smem_u32(ring + stage * P::kStage) + place;
      uint4 v[KU][RS][2];
#pragma unroll
      for (int q = 0; q < KU; ++q)
#pragma unroll
        for (int r = 0; r < RS; ++r)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            v[q][r][half] = lds128(at + (r / 2) * kRun + (2 * q + r % 2) * kW8Block + half * 512);
#pragma unroll
      for (int q = 0; q < KU; ++q)
#pragma unroll
        for (int r = 0; r < RS; ++r) {
          const uint32_t lo[4] = {v[q][r][0].x, v[q][r][0].y, v[q][r][0].z, v[q][r][0].w};
          const uint32_t hi[4] = {v[q][r][1].x, v[q][r][1].y, v[q][r][1].z, v[q][r][1].w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t a0, a1, a2, a3;
            w8_unpack(lo[s], a0, a2);
            w8_unpack(hi[s], a1, a3);
#pragma unroll
            for (int j = 0; j < MT; ++j) mma_f16_16816(acc[r][j], a0, a1, a2, a3, b[q][j][2 * s], b[q][j][2 * s + 1]);
          }
        }
      __syncwarp();  // every lane has read its part
      fetch(stage);
      if (++stage == D) stage = 0, phase ^= 1;
    }
    if (P::kBufs == 1) __syncthreads();  // the sums of the group before have been read
    float* sums = red + buf * NW * P::kElems;
    float* mine = sums + warp * P::kElems;
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[((r * MT + j) * 4 + i) * 32 + lane] = acc[r][j][i];
    __syncthreads();
    auto own_sum = [&](int e) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) a += sums[w * P::kElems + e];
      return a;
    };
    // element e: [r][j][i][lane] -> row 16 r + lane / 4 + 8 (i / 2), token 8 j + 2 (lane % 4) + i % 2
    auto finish = [&](auto&& sum) {
      const int outs = p.gated ? P::kElems / 2 : P::kElems;
      for (int o = threadIdx.x; o < outs; o += NW * 32) {
        const int e = p.gated ? (o >> 6) * 128 + (o & 63) : o;
        const int l = e & 31, i = (e >> 5) & 3, j = (e >> 7) % MT, r = (e >> 7) / MT;
        const int m = j * 8 + 2 * (l & 3) + (i & 1);
        const int row = (group * RS + r) * kW8Strip + (l >> 2) + 8 * (i >> 1);
        const int n = p.gated ? (group * RS + r) * 8 + (l >> 2) : row;
        if (m >= p.M || n >= p.N) continue;
        const float sx = p.x_scales[m];
        float v = sum(e) * sx * p.w_scales[row];
        if (p.gated) v = (p.type == SPEAR_F32 ? w8_act<true>(v, p.act) : w8_act<false>(v, p.act)) * (sum(e + 64) * sx * p.w_scales[row + 8]);
        w8_store(p.y, m * p.ld_y + n, p.type, v);
      }
    };
    if (seg == group * p.kq && end == (group + 1) * p.kq) {
      finish(own_sum);
    } else {
      // shared with other CTAs: the last one to arrive adds the parts in the CTAs' order
      auto slot = [&](int c, int first) { return p.part + ((int64_t)2 * c + (first >= group * p.kq ? 1 : 0)) * P::kElems; };
      float* part = slot(blockIdx.x, u0);
      for (int e = threadIdx.x; e < P::kElems; e += NW * 32) part[e] = own_sum(e);
      __threadfence();
      __syncthreads();
      // CTAs that hold a block of the group: from the one with its first to the one with its last
      int c0 = blockIdx.x, c1 = blockIdx.x;
      while (range_start(c0, gridDim.x, p.units, 1, 0, 0) > group * p.kq) --c0;
      while (range_start(c1 + 1, gridDim.x, p.units, 1, 0, 0) < (group + 1) * p.kq) ++c1;
      if (threadIdx.x == 0) {
        last = atomicAdd(p.counters + group, 1u) == (unsigned)(c1 - c0);
        if (last) p.counters[group] = 0;
      }
      __syncthreads();
      if (last) {
        __threadfence();
        finish([&](int e) {
          float a = 0.f;
          for (int c = c0; c <= c1; ++c)
            a += __ldcg(slot(c, range_start(c, gridDim.x, p.units, 1, 0, 0)) + e);
          return a;
        });
      }
    }
    seg = end;
    if (P::kBufs == 2) buf ^= 1;
  }
}

struct Split {
  int groups, kq, per, grid, balanced;
  int64_t cost;  // blocks of the CTA with the most, and what joining takes
};

// Whole row groups of RS strips need no joining between CTAs; an even split does, about the time of 200 blocks (4.5 us).
Split split(const spear_w8_s* h, int RS, int KU, int NW) {
  Split s;
  const int used = h->gated ? (h->N + 7) / 8 : (h->N + 15) / 16;
  s.groups = (used + RS - 1) / RS;
  s.kq = h->kb / KU;
  s.per = (s.groups + h->sm_count - 1) / h->sm_count;
  s.grid = (s.groups + s.per - 1) / s.per;
  s.balanced = 0;
  s.cost = (int64_t)s.per * s.kq * RS * KU;
  const int64_t units = (int64_t)s.groups * s.kq;
  const int even = (int)std::min<int64_t>(h->sm_count, std::max<int64_t>(1, units / NW));
  const int64_t cost = (units + even - 1) / even * RS * KU + 200;
  if (cost < s.cost) s.balanced = 1, s.grid = even, s.cost = cost;
  return s;
}

template <int MT, int RS, int KU, int NW, int D>
spear_status_t launch(const spear_w8_s* h, const W8Call& c, const Split& sp, cudaStream_t stream) {
  using P = Plan<MT, RS, KU, NW, D>;
  static std::atomic<uint64_t> configured{0};
  if (smem_limit_once(reinterpret_cast<const void*>(&stream_kernel<MT, RS, KU, NW, D>), configured) != cudaSuccess)
    return SPEAR_ERR_CUDA;
  StreamParams p = {h->w, h->w_scales, c.x, c.ld_x, c.x_scales, c.y, c.ld_y, h->part, h->counters, h->status, h->wait_ns};
  p.type = c.type, p.M = c.M, p.K = h->K, p.N = h->N, p.kq = sp.kq, p.gated = h->gated, p.act = h->act;
  p.units = sp.groups * sp.kq, p.per = sp.per, p.balanced = sp.balanced, p.skip_arrive = h->skip_arrive;
  return kv_launch(stream_kernel<MT, RS, KU, NW, D>, dim3(sp.grid), NW * 32, P::kSmem, stream, p);
}

// Two strips by two blocks, or four strips where that costs no balance: half the tokens' codes.
template <int MT, int NW, int D>
spear_status_t launch(const spear_w8_s* h, const W8Call& c, cudaStream_t stream) {
  const Split s2 = split(h, 2, 2, NW), s4 = split(h, 4, 1, NW);
  if (s4.cost * 16 <= s2.cost * 17) return launch<MT, 4, 1, NW, D>(h, c, s4, stream);
  return launch<MT, 2, 2, NW, D>(h, c, s2, stream);
}

}  // namespace

// Two parts a CTA, of the variant with the most sums.
size_t w8_decode_workspace(const spear_w8_s* h) { return (size_t)2 * h->sm_count * Plan<2, 4, 1, 16, 2>::kElems * sizeof(float); }

spear_status_t w8_launch_decode(const spear_w8_s* h, const W8Call& c, cudaStream_t stream) {
  if (c.M <= 8) return launch<1, 16, 3>(h, c, stream);
  if (c.M <= 16) return launch<2, 16, 2>(h, c, stream);
  // more tokens: 2 KB a turn, in the registers of 16 warps (4 KB and 8 warps: 76 us against 63 for 32 x 28672 x 8192)
  return launch<4, 2, 1, 16, 4>(h, c, split(h, 2, 1, 16), stream);
}

}  // namespace spear

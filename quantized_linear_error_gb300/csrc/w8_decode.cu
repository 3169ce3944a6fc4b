// Few tokens (up to 32) through 8-bit integer weights: a kernel that streams
// the weights once.
//
//   y[m][n] = round(s_x[m] s_w[n] sum_k q_x[m][k] q_w[n][k])
//
// Bound by the weights' bytes. Each warp streams blocks of its own through a
// private ring in shared memory (asynchronous 16-byte copies; a lane reads back
// only what it copied, so nothing but its own copies has to be waited for),
// turns the codes into f16 in registers and feeds warp MMAs whose A operand is
// 16 weight rows and whose columns are 8 tokens. Products of codes and their
// sums below 2^24 are exact in the fp32 accumulators.
//
// The warps of a CTA take blocks of the same rows along K in turn; their sums
// are added in shared memory in a fixed order.
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
  unsigned* counters;
  int type, M, K, N, kb, gated, act;
  int units, balanced, per;  // blocks in all; split evenly, or `per` whole row groups a CTA
};

SPEAR_DEVINL void cp_async16(uint32_t dst, const void* src, unsigned bytes) {  // zeros past `bytes`
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
SPEAR_DEVINL void cp_async16_stream(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
SPEAR_DEVINL void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SPEAR_DEVINL void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

SPEAR_DEVINL void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// First block of CTA c.
__host__ __device__ inline int range_start(int c, int grid, int units, int balanced, int per, int kb) {
  if (balanced) return (int)((int64_t)c * units / grid);
  const int64_t u = (int64_t)c * per * kb;
  return u < units ? (int)u : units;
}

// MT tiles of 8 tokens, RS strips of 16 rows a warp, NW warps, D blocks in flight a warp.
template <int MT, int RS, int NW, int D>
struct Plan {
  static constexpr int kStage = RS * kW8Block + MT * 512;     // a warp's
  static constexpr int kRing = NW * D * kStage;
  static constexpr int kElems = RS * MT * 128;                // sums of a row group
  static constexpr int kSmem = kRing + 2 * NW * kElems * 4 + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

template <int MT, int RS, int NW, int D>
__global__ void __launch_bounds__(NW * 32, 1) stream_kernel(const __grid_constant__ StreamParams p) {
  using P = Plan<MT, RS, NW, D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u0 = range_start(blockIdx.x, gridDim.x, p.units, p.balanced, p.per, p.kb);
  const int u1 = range_start(blockIdx.x + 1, gridDim.x, p.units, p.balanced, p.per, p.kb);
  const uint32_t ring = smem_u32(smem) + warp * D * P::kStage + lane * 16;
  float* red = reinterpret_cast<float*>(smem + P::kRing);
  volatile int& last = *reinterpret_cast<volatile int*>(smem + P::kSmem - 16);

  grid_launch_dependents();
  // a row group's strips follow each other, kb blocks each
  int fg = u0 / p.kb, fk = u0 - fg * p.kb + warp, fu = u0 + warp;  // the block to be copied next
  while (fk >= p.kb) fk -= p.kb, ++fg;
  auto fetch_w = [&](int stage) {
    if (fu < u1) {
      const uint8_t* src = p.w + ((int64_t)fg * RS * p.kb + fk) * kW8Block + w8_place(g, t) * 16;
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          cp_async16_stream(ring + stage * P::kStage + r * kW8Block + half * 512,
                            src + (int64_t)r * p.kb * kW8Block + half * 512);
    }
  };
  auto fetch_x = [&](int stage, int u, int kblock) {
    if (u < u1) {
      const int k = kblock * kW8K + t * 16;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int m = j * 8 + g;
        const bool real = m < p.M && k < p.K;  // K is a multiple of 16
        cp_async16(ring + stage * P::kStage + RS * kW8Block + j * 512, real ? p.x + m * p.ld_x + k : p.x, real ? 16 : 0);
      }
    }
  };
  auto advance = [&] {
    fu += NW, fk += NW;
    while (fk >= p.kb) fk -= p.kb, ++fg;
  };
  const int u_first = fu, k_first = fk;
#pragma unroll
  for (int d = 0; d < D; ++d) {  // the handle's own weights, while the kernel before this one ends
    fetch_w(d);
    advance();
  }
  grid_wait();
  {
    int u = u_first, k = k_first;
#pragma unroll
    for (int d = 0; d < D; ++d) {
      fetch_x(d, u, k);
      cp_async_commit();
      u += NW, k += NW;
      while (k >= p.kb) k -= p.kb;
    }
  }

  int u = u0 + warp, stage = 0, buf = 0;
  for (int seg = u0; seg < u1;) {
    const int group = seg / p.kb, end = min(u1, (group + 1) * p.kb);
    float acc[RS][MT][4];
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][j][i] = 0.f;
    for (; u < end; u += NW) {
      cp_async_wait<D - 1>();
      const uint32_t at = ring + stage * P::kStage;
      uint32_t b[MT][8];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const uint4 v = lds128(at + RS * kW8Block + j * 512);
        w8_unpack(v.x ^ kW8Bias, b[j][0], b[j][1]);
        w8_unpack(v.y ^ kW8Bias, b[j][2], b[j][3]);
        w8_unpack(v.z ^ kW8Bias, b[j][4], b[j][5]);
        w8_unpack(v.w ^ kW8Bias, b[j][6], b[j][7]);
      }
#pragma unroll
      for (int r = 0; r < RS; ++r) {
        const uint4 v0 = lds128(at + r * kW8Block), v1 = lds128(at + r * kW8Block + 512);
        const uint32_t lo[4] = {v0.x, v0.y, v0.z, v0.w}, hi[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t a0, a1, a2, a3;
          w8_unpack(lo[s], a0, a2);
          w8_unpack(hi[s], a1, a3);
#pragma unroll
          for (int j = 0; j < MT; ++j) mma_f16_16816(acc[r][j], a0, a1, a2, a3, b[j][2 * s], b[j][2 * s + 1]);
        }
      }
      fetch_w(stage);
      fetch_x(stage, fu, fk);
      cp_async_commit();
      advance();
      stage = stage + 1 == D ? 0 : stage + 1;
    }
    float* mine = red + (buf * NW + warp) * P::kElems;
#pragma unroll
    for (int r = 0; r < RS; ++r)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[((r * MT + j) * 4 + i) * 32 + lane] = acc[r][j][i];
    __syncthreads();
    const float* sums = red + buf * NW * P::kElems;
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
        if (p.gated) v = w8_act(v, p.act) * (sum(e + 64) * sx * p.w_scales[row + 8]);
        w8_store(p.y, m * p.ld_y + n, p.type, v);
      }
    };
    if (seg == group * p.kb && end == (group + 1) * p.kb) {
      finish(own_sum);
    } else {
      // shared with other CTAs: the last one to arrive adds the parts in the CTAs' order
      auto slot = [&](int c, int first) { return p.part + ((int64_t)2 * c + (first >= group * p.kb ? 1 : 0)) * P::kElems; };
      float* part = slot(blockIdx.x, u0);
      for (int e = threadIdx.x; e < P::kElems; e += NW * 32) part[e] = own_sum(e);
      __threadfence();
      __syncthreads();
      // CTAs that hold a block of the group: from the one with its first to the one with its last
      int c0 = blockIdx.x, c1 = blockIdx.x;
      while (range_start(c0, gridDim.x, p.units, 1, 0, 0) > group * p.kb) --c0;
      while (range_start(c1 + 1, gridDim.x, p.units, 1, 0, 0) < (group + 1) * p.kb) ++c1;
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
    buf ^= 1;
    seg = end;
  }
}

template <int MT, int RS, int NW, int D>
spear_status_t launch(const spear_w8_s* h, const W8Call& c, cudaStream_t stream) {
  using P = Plan<MT, RS, NW, D>;
  static std::atomic<uint64_t> configured{0};
  if (smem_limit_once(reinterpret_cast<const void*>(&stream_kernel<MT, RS, NW, D>), configured) != cudaSuccess)
    return SPEAR_ERR_CUDA;
  StreamParams p = {h->w, h->w_scales, c.x, c.ld_x, c.x_scales, c.y, c.ld_y, h->part, h->counters};
  p.type = c.type, p.M = c.M, p.K = h->K, p.N = h->N, p.kb = h->kb, p.gated = h->gated, p.act = h->act;
  const int groups = h->strips / RS;
  p.units = groups * h->kb;
  p.per = (groups + h->sm_count - 1) / h->sm_count;
  int grid = (groups + p.per - 1) / p.per;
  // Whole row groups need no joining between CTAs; an even split does (about the time of 64 KB a CTA).
  const int even = std::min(h->sm_count, std::max(1, p.units / NW));
  if ((int64_t)p.per * h->kb - p.units / even > 64 / RS) {
    p.balanced = 1;
    grid = even;
  }
  return kv_launch(stream_kernel<MT, RS, NW, D>, dim3(grid), NW * 32, P::kSmem, stream, p);
}

}  // namespace

// Two parts a CTA, of the variant with the most sums.
size_t w8_decode_workspace(const spear_w8_s* h) { return (size_t)2 * h->sm_count * Plan<4, 2, 8, 4>::kElems * sizeof(float); }

spear_status_t w8_launch_decode(const spear_w8_s* h, const W8Call& c, cudaStream_t stream) {
  if (c.M <= 8) return launch<1, 1, 16, 6>(h, c, stream);
  if (c.M <= 16) return launch<2, 2, 16, 3>(h, c, stream);
  return launch<4, 2, 8, 4>(h, c, stream);
}

}  // namespace spear

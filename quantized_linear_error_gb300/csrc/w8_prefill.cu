// Many tokens (more than 32, or 16 where weights are many) through 8-bit integer
// weights on the tcgen05 tensor cores.
//
//   y[m][n] = round(s_x[m] s_w[n] sum_k q_x[m][k] q_w[n][k])
//
// sm_103a has no integer MMA of tcgen05's rate, and codes are exact in f16, their
// products and sums below 2^24 in fp32: the contraction runs at the f16 rate and
// is bound by it (2 M N K operations).
//
// A small kernel turns the tokens' codes into f16 tiles in the order that the
// tensor cores read (64 channels x 8 tokens, 1 KB, 128-byte swizzle) and the
// copies run through, so that a stage's tokens are one bulk copy; every row tile
// reads them again, from L2. The weights stay in 8 bits until they reach the SM.
//
// A pair of CTAs (a cluster, cta_group::2) works on 256 weight rows x TN tokens:
// each CTA holds 128 of the rows and half of the tokens, and the MMAs read both
// halves of the tokens, which halves the shared memory traffic of a single CTA's
// tile. A stage is 128 channels. Roles of a CTA:
//   warp 0       copies the weights' codes, 16 KB a stage
//   warp 1       issues the MMAs of the pair (in the first CTA): A from tensor
//                memory, B from both CTAs' shared memory
//   warps 2-9    codes -> f16 -> tensor memory: two warps 32 rows, every other stage each
//   warps 10-13  epilogue, from the accumulator that the MMAs have left, while they
//                fill the other one
//   warp 14      copies the tokens, TN / 2 of them a stage
// What each role does a stage is fixed cost next to the MMAs' 4 TN cycles: with 64
// channels a stage and one thread for both copies, a stage took 530 cycles of
// that thread, 350 of the dequantising warps and 325 of the issuing one.
//
// Measured: 4096 tokens through 2 x 28672 x 8192 (3.85 TFLOP) 1.93 to 2.00 ms in bursts,
// 100 to 104% of a library product's burst rate, 2.00 to 2.05 ms call after call, 98 to
// 100% (112 to 115% of its sustained rate); 2048 tokens
// x 14336 x 4096 135 us, 93%; tensor pipe active 90% of the time (profile of this
// case). Small calls are bound by stages of 580 cycles, whatever TN up to 128 (the
// eight MMAs of a stage then take some 64 cycles each), and by some 9 us of start,
// tokens' preparation, epilogue and end: 320 tokens x 4096 x 6144 20 us, of which 10
// in the MMAs' loop. Far from their floors (bytes or operations at a plain copy's and
// the library product's rates): few outputs, whose row tile is 256 all the same, while
// the tokens' f16 tiles are written and read back (4096 x 28672 into 64 outputs 129 us,
// floor 18; 5000 x 8192 into 16 60, 6), and few channels, where four epilogue warps take
// longer than the MMAs (4096 tokens of 64, 256 and 512 channels into 8192 outputs 43, 46
// and 50 us, floors 10, 10 and 18).
//
// Work is split in whole tiles as long as they fill all pairs; what does not come
// out even is split along K. The pairs that share a tile add their parts, as 32-bit
// integers, in memory: no order of the additions changes the sum, so that a
// repeated call gives the same bits. The last one to finish takes the sum, adds its
// own part from tensor memory and leaves zeros; nobody waits for another pair.
// (fp32 parts, read one after the other by the last pair: 20 us for 128 tokens.)
//
// Barriers between the CTAs of a pair order tensor memory and shared memory that
// copies have filled, each with the tcgen05 fences or by the copies' own
// completion; no ordinary memory goes through them, so that the arrivals need no
// wider scope than they have (cluster scope on both sides: 4 times the time).
#include <algorithm>

#include "tcgen05.cuh"
#include "w8_device.cuh"

namespace spear {
namespace {

constexpr int kThreads = 15 * 32;
constexpr int kRawBytes = 2 * kW8Tile * kW8Block;  // 128 rows x 128 channels
constexpr int kMaxTokens = 192;                    // of a tile: two accumulators and two A slots in 512 columns
constexpr int kSmem = 225 * 1024;
constexpr int kMaxStages = 8, kMaxSlots = 4;

struct GemmParams {
  const uint8_t *w, *x16;
  const float *w_scales, *x_scales;
  void* y;
  int64_t ld_y;
  int* sums;              // [tile][rank][token][row] of shared tiles, zero between calls
  unsigned *counters, *status, *spoilt;
  uint64_t wait_ns;
  int type, vec;          // vec: results may be stored 16 bytes at a time
  int M, N, ks, act, w_tiles;  // ks: stages of a tile
  int TN, n_tok;               // tokens of a tile, token tiles
  int tiles, sk_tiles, sk_pairs;  // tiles in all; those split along K, over that many pairs
  int stages, slots, stage_bytes, acc_stride;
  int skip_arrive;  // the first pair's first barrier of the dequantising warps expects an arrival that never comes
};

// Add `bytes` of 32-bit integers in shared memory to those at dst; waits for such copies by the thread that issued them.
SPEAR_DEVINL void bulk_add_s32(int* dst, const int* src, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.s32 [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
SPEAR_DEVINL void bulk_wait_read() {  // all but N have read their source
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
SPEAR_DEVINL void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct Segment {
  int tile, k0, k1;
};

// The pair's segments in order: its share of the tiles that are split, then whole ones.
struct Segments {
  int u, end, next, step;
  SPEAR_DEVINL Segments(const GemmParams& p, int pair, int pairs) {
    const int64_t units = (int64_t)p.sk_tiles * p.ks;
    u = pair < p.sk_pairs ? (int)(pair * units / p.sk_pairs) : 0;
    end = pair < p.sk_pairs ? (int)((pair + 1) * units / p.sk_pairs) : 0;
    next = p.sk_tiles + pair;
    step = pairs;
  }
  SPEAR_DEVINL bool get(const GemmParams& p, Segment& s) {
    if (u < end) {
      s.tile = u / p.ks;
      s.k0 = u - s.tile * p.ks;
      s.k1 = min(p.ks, s.k0 + end - u);
      u += s.k1 - s.k0;
      return true;
    }
    if (next >= p.tiles) return false;
    s.tile = next, s.k0 = 0, s.k1 = p.ks;
    next += step;
    return true;
  }
};

SPEAR_DEVINL uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
SPEAR_DEVINL void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Address of the first CTA's barrier at the same place, and an arrival on it.
SPEAR_DEVINL uint32_t leader_bar(uint64_t* bar) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(bar)));
  return r;
}
SPEAR_DEVINL void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
SPEAR_DEVINL bool mbar_test(uint32_t bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait of a whole warp; most phases are over when they are asked for, which a test shows sooner than a try.
SPEAR_DEVINL bool wait_bar(uint64_t* bar, unsigned parity, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, mbar_test(smem_u32(bar), parity))) return true;
  return warp_wait(bar, parity, limit_ns, 0);
}
// By the elected lane of a warp whose control flow is uniform.
SPEAR_DEVINL void expect_and_copy(uint32_t leader, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%3], %2;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "r"(leader)
      : "memory");
}

// Eight k steps of 16: A from tensor memory, 8 columns a step; B from two tiles of 64 channels, 32 bytes a step.
SPEAR_DEVINL void umma2_stage(uint32_t leader, uint32_t d, uint32_t a, uint64_t b0, uint64_t b1, uint32_t idesc, uint32_t accumulate) {
#define SPEAR_MMA(A, B, P) "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [" A "], " B ", %4, " P ";\n\t"
#define SPEAR_NEXT "add.u32 a, a, 8;\n\tadd.u64 b, b, 2;\n\t"
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b32 a, %1;\n\tmov.b64 b, %2;\n\t"
      SPEAR_MMA("a", "b", "p") SPEAR_NEXT SPEAR_MMA("a", "b", "t") SPEAR_NEXT SPEAR_MMA("a", "b", "t") SPEAR_NEXT
      SPEAR_MMA("a", "b", "t") "add.u32 a, a, 8;\n\tmov.b64 b, %3;\n\t"
      SPEAR_MMA("a", "b", "t") SPEAR_NEXT SPEAR_MMA("a", "b", "t") SPEAR_NEXT SPEAR_MMA("a", "b", "t") SPEAR_NEXT
      SPEAR_MMA("a", "b", "t") "}" ::"r"(d), "r"(a), "l"(b0), "l"(b1), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
#undef SPEAR_MMA
#undef SPEAR_NEXT
}
// Arrive on both CTAs' barriers when the MMAs issued so far have completed.
SPEAR_DEVINL void umma2_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "mov.b16 m, 3;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// A wait ran out. Parts that other pairs have added may stay in the sums, which other handles share.
SPEAR_DEVINL void gave_up(const GemmParams& p) {
  atomicOr(p.status, kStatusTimeoutPipe);
  if (p.sk_tiles) atomicOr(p.spoilt, 1u);
}

SPEAR_DEVINL void lds(uint16_t& v, uint32_t addr) { asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr)); }
SPEAR_DEVINL void lds(uint32_t& v, uint32_t addr) { asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr)); }

// 32 rows x 16 columns of an accumulator: v[8 h + 4 i + e] is row 16 h + lane / 4 + 8 (e / 2), column 8 i + 2 (lane % 4)
// + e % 2, the fragment of 8 x 8 matrices, so that a store of transposed matrices gives rows of tokens, and both
// projections of a gated output stand in one lane.
SPEAR_DEVINL void acc_load(uint32_t taddr, uint32_t (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[8 * h]), "=r"(v[8 * h + 1]), "=r"(v[8 * h + 2]), "=r"(v[8 * h + 3]), "=r"(v[8 * h + 4]),
                   "=r"(v[8 * h + 5]), "=r"(v[8 * h + 6]), "=r"(v[8 * h + 7])
                 : "r"(taddr + ((uint32_t)(16 * h) << 16)));
}
SPEAR_DEVINL void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// What an epilogue warp keeps in shared memory.
struct EpilogueShared {
  int sums[2][512];           // two parts of 16 columns on their way, or 16 tokens' results
  float scales[kMaxTokens];   // of the tile's tokens
};

// One warp's 32 rows of an accumulator, 16 tokens at a time: scaled, rounded and stored.
template <bool kGated, bool kF32>
struct Epilogue {
  const GemmParams& p;
  EpilogueShared& sh;
  int lane, n0;      // n0: first output of the warp's
  float sw[4];       // scales of the rows lane / 4 + 8 i

  SPEAR_DEVINL Epilogue(const GemmParams& p, EpilogueShared& sh, int lane, int row0, int tok) : p(p), sh(sh), lane(lane) {
    n0 = kGated ? row0 / 2 : row0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sw[i] = row0 < p.w_tiles * 128 ? p.w_scales[row0 + 8 * i + (lane >> 2)] : 0.f;
    __syncwarp();
    for (int c = lane; c < p.TN; c += 32) {
      const int m = tok * p.TN + c;
      sh.scales[c] = m < p.M ? p.x_scales[m] : 0.f;
    }
    __syncwarp();
  }

  SPEAR_DEVINL uint32_t pack(float a, float b) const {
    if (p.type == SPEAR_BF16) return pack_bf16x2(a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  // kOuts neighbouring outputs of each of 16 tokens, `step` bytes apart in shared memory from `from` on. E: as wide.
  template <int kOuts, class E>
  SPEAR_DEVINL void store(uint32_t from, uint32_t step, int m0) const {
    E* const y = static_cast<E*>(p.y);
    if (p.vec && n0 + kOuts <= p.N) {  // 16 bytes a lane
      constexpr int kOf = 16 / sizeof(E), kLanes = kOuts / kOf, kTurns = kLanes / 2;
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int t = i * (32 / kLanes) + lane / kLanes, q = lane % kLanes;
        if (m0 + t < p.M) *reinterpret_cast<uint4*>(y + (m0 + t) * p.ld_y + n0 + kOf * q) = lds128(from + t * step + 16 * q);
      }
    } else {  // rows of any alignment: an output a lane, side by side
      constexpr int kAtOnce = 32 / kOuts;
      const int q = lane % kOuts;
#pragma unroll 4
      for (int t = lane / kOuts; t < 16; t += kAtOnce)
        if (m0 + t < p.M && n0 + q < p.N) {
          E e;
          lds(e, from + t * step + sizeof(E) * q);
          y[(m0 + t) * p.ld_y + n0 + q] = e;
        }
    }
  }

  // Columns c .. c + 15 of the tile, tokens m0 ..
  SPEAR_DEVINL void columns(float (&v)[16], int c, int m0) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 sx = *reinterpret_cast<const float2*>(&sh.scales[c + 8 * i + 2 * (lane & 3)]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float& x = v[8 * h + 4 * i + e];
          x = x * (e & 1 ? sx.y : sx.x) * sw[2 * h + (e >> 1)];
        }
    }
    if constexpr (kGated) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) v[4 * q + e] = w8_act<kF32>(v[4 * q + e], p.act) * v[4 * q + e + 2];
    }
    const uint32_t at = smem_u32(sh.sums);
    __syncwarp();
    if constexpr (kF32) {  // 128 (64 gated) bytes a token, 16 more apart: no bank conflicts
      constexpr int kStep = kGated ? 80 : 144;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (kGated && (j & 2)) continue;
        const int t = 2 * (j & 4) + 2 * (lane & 3) + (j & 1);
        const int n = kGated ? 8 * (j >> 3) + (lane >> 2) : 16 * (j >> 3) + 8 * ((j >> 1) & 1) + (lane >> 2);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + t * kStep + 4 * n), "f"(v[j]) : "memory");
      }
      __syncwarp();
      store<kGated ? 16 : 32, uint32_t>(at, kStep, m0);
    } else {
      if constexpr (kGated) {  // 32 bytes a token, 48 apart: no bank conflicts
        store_transposed(at + (8 * (lane >> 4) + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16, pack(v[0], v[1]), pack(v[8], v[9]),
                         pack(v[4], v[5]), pack(v[12], v[13]));
        __syncwarp();
        store<16, uint16_t>(at, 48, m0);
      } else {                 // 64 bytes a token, 80 apart
#pragma unroll
        for (int i = 0; i < 2; ++i)
          store_transposed(at + (8 * i + (lane & 7)) * 80 + (lane >> 3) * 16, pack(v[4 * i], v[4 * i + 1]),
                           pack(v[4 * i + 2], v[4 * i + 3]), pack(v[8 + 4 * i], v[8 + 4 * i + 1]),
                           pack(v[8 + 4 * i + 2], v[8 + 4 * i + 3]));
        __syncwarp();
        store<32, uint16_t>(at, 80, m0);
      }
    }
  }
};

struct Shared {
  uint64_t raw[kMaxStages];    // a stage's copies have landed (this CTA)
  uint64_t a[kMaxStages];      // its codes stand in tensor memory, in both CTAs (the first CTA's)
  uint64_t empty[kMaxStages];  // its MMAs have run (both CTAs)
  uint64_t acc_full[2];        // an accumulator is complete (both CTAs)
  uint64_t acc_empty[2];       // it has been read, in both CTAs (the first CTA's)
  alignas(16) EpilogueShared epilogue[4];
  uint32_t tmem;
};

// (Registers for 608 threads: a block of convert_kernel runs beside this one.)
template <bool kGated, bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads + 128, 1) gemm_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;  // the swizzle goes by the address
  Shared& sh = *reinterpret_cast<Shared*>(smem + p.stages * p.stage_bytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sh.raw[s], 2);
      mbar_init(&sh.a[s], s == 0 && blockIdx.x == 0 && p.skip_arrive ? 9 : 8);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], 8);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before_sync();
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after_sync();
  // Not before tensor memory is held: a kernel that follows may want it too, and would then hold it while it waits for this one.
  grid_launch_dependents();
  const uint32_t tmem = sh.tmem;
  const uint32_t a_base = tmem + 2 * p.acc_stride;
  const int b_bytes = p.TN * 128;  // half the tokens x 128 channels

  Segments segs(p, pair, pairs);
  Segment sg;
  bool ok = true;
  if (warp == 0 || warp == 14) {
    // Copies: the handle's own weights ahead of the kernel before this one, the tokens' tiles behind it.
    const bool tokens = warp == 14;
    bool follows = tokens;  // from here on a wait's time is limited, so not while the kernel before this one may run
    if (tokens) grid_wait();
    const uint32_t leader = elect_leader();
    const int64_t run = (int64_t)p.ks * 4096;  // of a pair of strips
    const uint32_t dst = smem_u32(smem) + (tokens ? 0 : b_bytes);
    int s = 0, issued = 0;
    unsigned phase = 1;  // the first pass through the ring finds every stage empty
    while (ok && segs.get(p, sg)) {
      const int row = sg.tile / p.n_tok, tok = sg.tile - row * p.n_tok;
      const uint8_t* src = tokens ? p.x16 + ((int64_t)(tok * 2 + rank) * p.ks + sg.k0) * b_bytes
                                  : p.w + min(row * 2 + rank, p.w_tiles - 1) * 4 * run + (int64_t)sg.k0 * 4096;
      for (int k = sg.k0; k < sg.k1; ++k) {
        if (!follows && issued == p.stages) {
          grid_wait();
          follows = true;
        }
        ok = wait_bar(&sh.empty[s], phase, p.wait_ns);
        if (!ok) break;
        if (tokens) {
          expect_and_copy(leader, dst + s * p.stage_bytes, src, b_bytes, smem_u32(&sh.raw[s]));
          src += b_bytes;
        } else {
          if (leader) mbar_arrive_expect_tx(&sh.raw[s], kRawBytes);
          // lane i < 4: a pair of strips' 4 KB
          if (lane < 4) bulk_g2s_shared_u32(dst + s * p.stage_bytes + lane * 4096, src + lane * run, 4096, &sh.raw[s]);
          src += 4096;
        }
        ++issued;
        if (++s == p.stages) s = 0, phase ^= 1;
      }
    }
    if (!follows) grid_wait();
    if (!ok && lane == 0) gave_up(p);
    // every stage's MMAs have run before the CTA may leave (or, given up, its copies have landed)
    const int left = min(issued, p.stages);
    if (issued < p.stages) s = 0, phase = 0;
    for (int i = 0; i < left; ++i) {
      if (ok) ok = wait_bar(&sh.empty[s], phase, p.wait_ns);
      else warp_wait(&sh.raw[s], phase, kW8WaitNs / 10, 0);
      if (++s == p.stages) s = 0, phase ^= 1;
    }
  } else if (warp == 1) {
    grid_wait();
    if (rank == 0) {
      const uint32_t leader = elect_leader();
      const uint32_t idesc = idesc_f16_f32(256, p.TN);
      int s = 0, slot = 0, buf = 0;
      unsigned phase = 0, acc_phase = 1;
      while (ok && segs.get(p, sg)) {
        ok = wait_bar(&sh.acc_empty[buf], acc_phase, p.wait_ns);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t d = tmem + buf * p.acc_stride;
        for (int k = sg.k0; k < sg.k1; ++k) {
          ok = wait_bar(&sh.a[s], phase, p.wait_ns);
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t desc = sw128_kmajor_desc(smem_u32(smem + s * p.stage_bytes));
          const uint64_t desc2 = desc + (p.TN * 64 >> 4);  // the second 64 channels
          umma2_stage(leader, d, a_base + slot * 64, desc, desc2, idesc, k > sg.k0);
          umma2_commit(leader, &sh.empty[s]);
          if (++s == p.stages) s = 0, phase ^= 1;
          if (++slot == p.slots) slot = 0;
        }
        if (!ok) break;
        umma2_commit(leader, &sh.acc_full[buf]);
        if ((buf ^= 1) == 0) acc_phase ^= 1;
      }
      if (!ok && lane == 0) gave_up(p);
    } else if (blockIdx.x == 1 && lane == 0 && p.sk_tiles && __ldcg(p.spoilt)) {
      atomicOr(p.status, kStatusTimeoutPipe);  // the sums of this call's shared tiles are wrong
    }
  } else if (warp < 10) {
    grid_wait();
    const int quarter = warp & 3, turn = (warp - 2) >> 2;  // every other stage
    const int r = 32 * quarter + lane;
    const uint32_t base = smem_u32(smem) + b_bytes + (r >> 5) * 4 * kW8Block + ((r >> 4) & 1) * kW8Block;  // quarter's pair
    uint32_t at[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) at[t] = base + w8_place(r & 15, t) * 16;
    const uint32_t dst = a_base + ((uint32_t)(32 * quarter) << 16);
    const uint32_t full = leader_bar(&sh.a[0]);
    // s, slot: of stage n; es: the stage whose MMAs free the slot, stage n - slots
    int n = 0, s = 0, slot = 0, es = 0;
    unsigned phase = 0, e_phase = 0;
    auto next = [&] {
      if (++n > p.slots && ++es == p.stages) es = 0, e_phase ^= 1;
      if (++s == p.stages) s = 0, phase ^= 1;
      if (++slot == p.slots) slot = 0;
    };
    if (turn) next();
    int skip = turn;  // stages to pass before the next one of this warp's
    while (ok && segs.get(p, sg)) {
      int k = sg.k0 + skip;
      for (; k < sg.k1; k += 2) {
        ok = wait_bar(&sh.raw[s], phase, p.wait_ns);
        if (!ok) break;
        const uint32_t from = s * p.stage_bytes;
        uint4 v[8];  // all loads ahead of the first conversion
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = lds128(at[t & 3] + from + (t >> 2) * 2 * kW8Block);
        uint32_t f[32];
        auto convert = [&](int half) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint4 w = v[4 * half + t];
            w8_unpack(w.x, f[8 * t], f[8 * t + 1]), w8_unpack(w.y, f[8 * t + 2], f[8 * t + 3]);
            w8_unpack(w.z, f[8 * t + 4], f[8 * t + 5]), w8_unpack(w.w, f[8 * t + 6], f[8 * t + 7]);
          }
        };
        convert(0);
        if (n >= p.slots) {
          ok = wait_bar(&sh.empty[es], e_phase, p.wait_ns);
          if (!ok) break;
          tc_fence_after_sync();
        }
        tmem_st_x32(dst + slot * 64, f);
        convert(1);
        tmem_st_x32(dst + slot * 64 + 32, f);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full + 8 * s);
        next();
        next();
      }
      skip = k - sg.k1;
    }
    if (!ok && lane == 0) gave_up(p);
  } else {
    grid_wait();  // the tokens' scales, and what the kernel before this one may still read of y
    const int quarter = warp & 3;
    const uint32_t emptied = leader_bar(&sh.acc_empty[0]);
    EpilogueShared& mine = sh.epilogue[warp - 10];
    const int64_t units = (int64_t)p.sk_tiles * p.ks;
    int buf = 0;
    unsigned phase = 0;
    while (segs.get(p, sg)) {
      const int row = sg.tile / p.n_tok, tok = sg.tile - row * p.n_tok;
      const Epilogue<kGated, kF32> out(p, mine, lane, (row * 2 + rank) * 128 + 32 * quarter, tok);
      ok = wait_bar(&sh.acc_full[buf], phase, p.wait_ns);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t acc = tmem + buf * p.acc_stride + ((uint32_t)(32 * quarter) << 16);
      const bool whole = sg.k0 == 0 && sg.k1 == p.ks;
      // [16 columns][4][lane][4]: a lane's 16 values of acc_load as four vectors
      int* sums = p.sums + ((int64_t)(sg.tile * 2 + rank) * 4 + quarter) * p.TN * 32;
      bool held = true, last = true;  // this pair's part is in tensor memory; the tile is complete with it
      if (!whole) {
        // The pairs that share the tile: from the one with its first stage to the one with its last.
        const int64_t t0 = (int64_t)sg.tile * p.ks, t1 = t0 + p.ks;
        int c0 = pair, c1 = pair;
        while (c0 * units / p.sk_pairs > t0) --c0;
        while ((c1 + 1) * units / p.sk_pairs < t1) ++c1;
        unsigned* counter = p.counters + (sg.tile * 2 + rank) * 4 + quarter;
        const unsigned others = c1 - c0;
        // Where all others have added theirs, this part need not go through memory.
        held = __shfl_sync(0xffffffffu, ld_acquire_gpu(counter), 0) == others;
        if (!held) {
#pragma unroll 1
          for (int c = 0, b = 0; c < p.TN; c += 16, b ^= 1) {
            float v[16];
            acc_load(acc + c, reinterpret_cast<uint32_t(&)[16]>(v));
            tmem_ld_wait();
            if (lane == 0) bulk_wait_read<1>();  // the copy before the last one has left shared memory
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<int4*>(&mine.sums[b][(j * 32 + lane) * 4]) =
                  make_int4(__float2int_rn(v[4 * j]), __float2int_rn(v[4 * j + 1]), __float2int_rn(v[4 * j + 2]),
                            __float2int_rn(v[4 * j + 3]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bulk_add_s32(sums + c * 32, mine.sums[b], 2048);
          }
          unsigned n = 0;
          if (lane == 0) {
            bulk_wait_all();
            __threadfence();
            n = atomicAdd(counter, 1u);
          }
          last = __shfl_sync(0xffffffffu, n, 0) == others;
        }
        if (last) {
          __threadfence();
          if (lane == 0) *counter = 0;
        }
      }
      if (whole) {
#pragma unroll 1  // a call with few tiles runs this from a cold instruction cache
        for (int c = 0; c < p.TN; c += 16) {
          float v[16];
          acc_load(acc + c, reinterpret_cast<uint32_t(&)[16]>(v));
          tmem_ld_wait();
          out.columns(v, c, tok * p.TN + c);
        }
      } else if (last) {
        constexpr int kAhead = 2;  // groups of 16 columns on their way
        int4 g[kAhead][4];
        auto load = [&](int c, int4 (&to)[4]) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c < p.TN) to[j] = __ldcg(reinterpret_cast<const int4*>(sums + c * 32) + j * 32 + lane);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load(16 * i, g[i]);
#pragma unroll 1
        for (int c0 = 0; c0 < p.TN; c0 += 16 * kAhead) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int c = c0 + 16 * i;
            if (c >= p.TN) break;
            float v[16];
            if (held) {
              acc_load(acc + c, reinterpret_cast<uint32_t(&)[16]>(v));
              tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int* e = reinterpret_cast<const int*>(&g[i][j / 4]);
              v[j] = (float)(e[j % 4] + (held ? __float2int_rn(v[j]) : 0));
            }
            load(c + 16 * kAhead, g[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *(reinterpret_cast<int4*>(sums + c * 32) + j * 32 + lane) = make_int4(0, 0, 0, 0);
            out.columns(v, c, tok * p.TN + c);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(emptied + 8 * buf);
      if ((buf ^= 1) == 0) phase ^= 1;
    }
    if (!ok && lane == 0) gave_up(p);
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Tokens' codes -> f16 tiles of 8 tokens x 64 channels (1 KB), ordered [half of a token tile][k block][tile of the
// half]: a warp a tile, lane 4 r + t the 16 channels 16 t .. of token r. The order of channels within 16 is that of
// w8_unpack, as for the weights. Tokens past M and channels past K are zeros.
// Blocks go through the work with the next loads on their way: one fits an SM beside the main kernel's.
constexpr int kConvertThreads = 256, kConvertTiles = 4;  // k blocks a warp and turn
__global__ void __launch_bounds__(kConvertThreads) convert_kernel(const int8_t* __restrict__ x, int64_t ld_x, int M, int K,
                                                                  int kb, int half_groups, int groups,
                                                                  uint8_t* __restrict__ x16) {
  kv_follow();
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int step = gridDim.x * (kConvertThreads / 32), turns = (kb + kConvertTiles - 1) / kConvertTiles, tasks = turns * groups;
  auto load = [&](int task, uint4 (&v)[kConvertTiles]) {
    const int group = task / turns, k0 = (task - group * turns) * kConvertTiles, m = group * 8 + r;
#pragma unroll
    for (int i = 0; i < kConvertTiles; ++i) {
      const int k = (k0 + i) * kW8K + t * 16;
      v[i] = make_uint4(0, 0, 0, 0);
      if (m < M && k < K) v[i] = *reinterpret_cast<const uint4*>(x + m * ld_x + k);
    }
  };
  int task = blockIdx.x * (kConvertThreads / 32) + threadIdx.x / 32;
  uint4 v[kConvertTiles], next[kConvertTiles];
  if (task < tasks) load(task, v);
  for (; task < tasks; task += step) {
    if (task + step < tasks) load(task + step, next);
    const int group = task / turns, k0 = (task - group * turns) * kConvertTiles, half = group / half_groups;
    uint8_t* tile = x16 + (((int64_t)half * kb + k0) * half_groups + (group - half * half_groups)) * 1024 + r * 128;
#pragma unroll
    for (int i = 0; i < kConvertTiles; ++i) {
      uint4 a, b;
      w8_unpack(v[i].x ^ kW8Bias, a.x, a.y), w8_unpack(v[i].y ^ kW8Bias, a.z, a.w);
      w8_unpack(v[i].z ^ kW8Bias, b.x, b.y), w8_unpack(v[i].w ^ kW8Bias, b.z, b.w);
      if (k0 + i < kb) {
        uint8_t* at = tile + (int64_t)i * half_groups * 1024;
        // the lane's two chunks are one sector, the other way round in odd rows (16 bytes a store, half sectors: 320
        // tokens of 4096 x 6144 20.8 us instead of 19.7)
        const bool swap = r & 1;
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at + (t ^ (r >> 1)) * 32),
                     "r"(swap ? b.x : a.x), "r"(swap ? b.y : a.y), "r"(swap ? b.z : a.z), "r"(swap ? b.w : a.w),
                     "r"(swap ? a.x : b.x), "r"(swap ? a.y : b.y), "r"(swap ? a.z : b.z), "r"(swap ? a.w : b.w)
                     : "memory");
      }
      v[i] = next[i];
    }
  }
}

// How a call is cut: n_tok tiles of TN tokens; sk_tiles of all the tiles split along K over sk_pairs pairs.
struct Cut {
  int TN, n_tok, tiles, sk_tiles, sk_pairs;
  int64_t cycles;
};

// The cut with the least estimated time, where the MMAs of the next tile hide every epilogue but the last: below some 700
// channels they do not, the estimate is too low and its choice there was not measured.
// Measured, in cycles of an SM: a stage takes the MMAs' 4 TN and 40 more; its 16 KB of codes and 128 TN bytes of tokens come from L2 at 50 bytes a cycle when all SMs ask (1088 tokens through 22016 x
// 4096: a stage 423 ns with TN 192, 396 with 160, 410 with 128; the call 104, 110, 137 us); 580 at least
// (8 MMAs of 64 cycles, whatever TN, and the hand-over); the last tile's epilogue 25 TN; adding up a
// split tile 3000 and 110 TN, which whole tiles that follow it hide (61 tokens through 22016 x 4096, 86 tiles on 76
// pairs: 23.9 us; with all of them split 25.0); 8000 then (2048 tokens through 4096 x 4096, 13 x 160: 52.1 us with
// a split, 51.1 without, although that is 96 stages against 88). Chunk of 320 tokens, 6144 x 4096: 2 x 160 split 26
// us, 2 x 160 whole 21, 3 x 112 21, 4 x 80 27; 512 tokens, 8192 x 8192: 3 x 176 split 54, whole 62, 4 x 128 59 and 58.
Cut cut(const spear_w8_s* h, int M, size_t room) {
  const int pairs = h->sm_count / 2, ks = h->kb / 2, rows = (h->strips / kW8Tile + 1) / 2;
  Cut best = {};
  for (int n = (M + kMaxTokens - 1) / kMaxTokens, most = n + 4; n <= most; ++n) {
    Cut c = {((M + n - 1) / n + 15) / 16 * 16, n, rows * n, 0, pairs, 0};
    if (n < most - 4 + 1 || (size_t)c.TN * n <= room) {
      const int64_t stage = std::max({4 * c.TN + 40, (kRawBytes + 128 * c.TN) / 50, 580});
      c.cycles = (c.tiles + pairs - 1) / pairs * ks * stage + 25 * c.TN;
      if (best.TN == 0 || c.cycles < best.cycles) best = c;
      const int over = c.tiles % pairs;
      if (over && h->K <= 65536) {  // a sum of K products of codes has to fit 32 bits
        // what is over goes first, at least four stages a pair; whole tiles hide its adding up
        c.sk_tiles = over;
        const int64_t units = (int64_t)over * ks, whole = c.tiles / pairs * ks * stage, join = 3000 + 110 * c.TN;
        c.sk_pairs = (int)std::min<int64_t>(pairs, std::max<int64_t>(c.tiles < pairs ? over : 1, units / 4));
        c.cycles = (units + c.sk_pairs - 1) / c.sk_pairs * stage + (c.tiles < pairs ? join : std::max(join, whole + 25 * c.TN) + 8000);
        if (c.cycles < best.cycles) best = c;
      }
    }
  }
  return best;
}

// Room for whole token tiles: 16 n_tok tokens more than M at most.
size_t x16_tokens(const spear_w8_s* h) { return (size_t)h->max_tokens + h->max_tokens / 8 + 256; }

}  // namespace

// Arrival counters (2 CTAs x 4 warps a shared tile, fewer than one tile a pair) and sums of shared tiles: zero between calls.
// The sums follow a word that says that they may not be.
size_t w8_prefill_counters(const spear_w8_s* h) { return w8_many(h, h->max_tokens) ? (size_t)h->sm_count * 4 : 0; }
size_t w8_prefill_sums(const spear_w8_s* h) {
  return w8_many(h, h->max_tokens) ? kW8SumsAt + (size_t)h->sm_count * kMaxTokens * 128 * sizeof(int) : 0;
}
// The tokens in f16.
size_t w8_prefill_workspace(const spear_w8_s* h) {
  return w8_many(h, h->max_tokens) ? (size_t)h->kb * 128 * x16_tokens(h) : 0;
}

spear_status_t w8_launch_prefill(const spear_w8_s* h, const W8Call& c, cudaStream_t stream) {
  GemmParams p = {};
  p.w = h->w, p.x16 = h->x16, p.w_scales = h->w_scales, p.x_scales = c.x_scales;
  p.y = c.y, p.ld_y = c.ld_y, p.sums = h->sums, p.counters = h->gemm_counters, p.status = h->status, p.spoilt = h->spoilt;
  p.type = c.type, p.M = c.M, p.N = h->N, p.ks = h->kb / 2, p.act = h->act, p.w_tiles = h->strips / kW8Tile;
  p.vec = (reinterpret_cast<uintptr_t>(c.y) & 15) == 0 && (c.ld_y % (c.type == SPEAR_F32 ? 4 : 8) == 0 || c.M == 1);
  p.wait_ns = h->wait_ns, p.skip_arrive = h->skip_arrive;
  const int pairs = h->sm_count / 2;
  const Cut k = cut(h, c.M, x16_tokens(h));
  p.TN = k.TN, p.n_tok = k.n_tok, p.tiles = k.tiles, p.sk_tiles = k.sk_tiles, p.sk_pairs = k.sk_pairs;
  p.acc_stride = (p.TN + 31) / 32 * 32;
  p.slots = std::min(kMaxSlots, (512 - 2 * p.acc_stride) / 64);
  p.stage_bytes = kRawBytes + p.TN * 128;
  p.stages = std::min(kMaxStages, (int)(kSmem - sizeof(Shared) - 1024) / p.stage_bytes);
  const size_t smem = std::max((size_t)p.stages * p.stage_bytes + sizeof(Shared) + 1024, (size_t)120 * 1024);  // one CTA an SM

  const int grid = 2 * std::min(pairs, std::max(p.sk_tiles ? p.sk_pairs : 0, p.tiles - p.sk_tiles));

  static std::atomic<uint64_t> configured[4];
  constexpr void (*kernels[4])(GemmParams) = {gemm_kernel<false, false>, gemm_kernel<false, true>, gemm_kernel<true, false>,
                                              gemm_kernel<true, true>};
  const int which = 2 * h->gated + (c.type == SPEAR_F32);
  if (smem_limit_once(reinterpret_cast<const void*>(kernels[which]), configured[which]) != cudaSuccess) return SPEAR_ERR_CUDA;
  const int groups = p.n_tok * p.TN / 8, per = kConvertThreads / 32;
  const int64_t tasks = (int64_t)groups * ((h->kb + kConvertTiles - 1) / kConvertTiles);
  const spear_status_t st = kv_launch(convert_kernel, dim3((unsigned)std::min<int64_t>((tasks + per - 1) / per, h->sm_count)),
                                      kConvertThreads, 0, stream, c.x, c.ld_x, c.M, h->K, h->kb, p.TN / 16, groups, h->x16);
  if (st != SPEAR_OK) return st;
  return kv_launch(kernels[which], dim3(grid), kThreads, smem, stream, p);
}

}  // namespace spear

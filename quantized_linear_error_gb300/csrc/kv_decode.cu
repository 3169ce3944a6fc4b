// Attention of a few query rows over the paged 4-bit cache: one new token a
// sequence, or a few drafted ones.
//
// For each (sequence, key/value head) the R = 8 NT RG rows (query tokens x the
// heads that share the key/value head) meet every visible key once:
//   s = scale (q . k),  out = sum 2^(s - m) v / sum 2^(s - m)   (s in log2),
// so the cache is read once, (D + 8) bytes a key for 4 D R flops: bound by
// memory as long as the instructions that unpack the codes keep up. Measured,
// D = 128: 8 heads a key/value head, 128 sequences of 500 to 8192 keys (607 MB)
// in 115 us, 5.3 TB/s, 78% of a plain copy; one head each, 64 sequences of 100
// to 4096 keys and 32 heads (601 MB) in 118 us, 76%; one sequence of 262143
// keys (285 MB) in 62.5 us, 68%; a call of little work takes 6.5 us, most of it
// launch, look-up of lengths and pages, first copy and join.
//
//  - Products run on warp MMAs (m16n8k16) with the cache as the A operand and
//    the rows as the 8 columns of B, so that no tensor work is spent on padding
//    a single token's few heads to 16 rows. (tcgen05 would want 128 rows of
//    dequantised keys written to tensor or shared memory for 8 columns.)
//  - K: four lanes hold a key's codes, D / 4 channels each, in the order of its
//    bytes. A masked nibble, or byte, reads as an f16 subnormal, c 2^-24, which
//    the MMA takes as it is: no arithmetic on K at all. A byte is lo + 16 hi, so
//    q0 lo + q1 hi = (q0 - q1 / 16) lo + (q1 / 16) byte: four masks a word. The
//    rows of q are scaled by a power of two into f16, once a segment. Then s =
//    S (q . c) + O sum(q) with the key's scale S and offset O.
//  - V: transposed matrix loads of 16-bit words put four channels of two keys
//    in a register, as the A operand of out^T = V^T p^T wants it; again the low
//    nibbles and whole bytes enter, and the high nibbles are their difference,
//    taken at the end. Codes are centred, lo - 8 and byte - 136, exact in 16
//    bits (small magnitudes: neither the fp32 sums nor the rounding of p S lose
//    to a large common term); sum p (O + 8 S) is kept beside it in fp32. p S is
//    rounded to f16, 11 bits (its range: see the reference, below); 32 keys with
//    a scale far below the largest so far go through bf16, 8 bits, with the same
//    accumulators.
//    The scores' accumulator layout becomes p^T's operand layout by one 8 x 8
//    transpose (movmatrix).
//  - The reference m of the weights p = 2^(s - m) is free, and does two things.
//    It follows the maximum lazily: sums are only rescaled when some score passes
//    it by 8 more than at first. And it lies k below the maximum, k such that the
//    warp's largest value scale so far times 2^k is in 2^6 .. 2^7: then p S is
//    below 2^15, and all of f16's range beneath serves small weights, which keep
//    8 bits down to some 2^-22 of the largest and are lost below 2^-31. (With k =
//    0 weights of 2^-17 of values of size 0.01 were lost: thousands of keys
//    behind one that has most of the weight.)
//
// Work: (sequence, head, tile of 128 keys) units, in this order, are split
// evenly over the CTAs, whatever the lengths, which only the device knows. A
// CTA's run is a list of segments, one an item (sequence, head). Partial
// results of items that several CTAs share go to the workspace; the last CTA
// of an item to arrive joins them in CTA order (the same bits every time) and
// resets the counter. No CTA waits for another.
//
// Variants: up to 8 rows one MMA tile a warp (NT = 1), up to 16 two, up to 32 two
// groups of warps (RG = 2) with 16 rows each over the same tiles: 32 sequences x
// 4000 keys x 8 heads with 8 / 16 / 32 rows take 36 / 60 / 102 us. The rows'
// instructions, not the bytes, bound the last two. (Four tiles in a warp's
// registers instead of two groups: 180 us; eight rows a group, so that 16 and 32
// rows get 16 warps an SM: 67 and 122 us, the registers spill and each group
// unpacks again.)
//
// A CTA: four warps, 32 keys of a tile each with a state of their own, joined
// at the end of a segment; a warp more copies the tiles' 16-token blocks (one
// bulk copy each, whatever the page size) into a ring of stages.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv_device.cuh"

namespace spear {
namespace {

constexpr int kKeyWarps = 4;                   // consumer warps along the keys of a tile
constexpr int kTile = 32 * kKeyWarps;          // keys of a unit
constexpr int kBlocksPerTile = kTile / 16;
constexpr int kMaxStages = 16;
constexpr int kItemCost = 3;                   // units: rows of q in, states joined, results out (64 ragged sequences: 158 us
                                               // with 0, 119 with 3 when it came in)
constexpr int kMinUnits = 4;                   // a CTA's, where there are few of them (4 sequences of 1000 tokens: 13.4 us
                                               // without the rule, 11.8 with it)
constexpr int kScan = 10;                      // warps at most
constexpr float kLazy = 8.f;
// Value scales, by their exponent fields. Largest ones of 2^-34 .. 2^46 choose k (beyond, 2^k and the sums could leave fp32);
// f16 takes this many binades from the largest down.
constexpr uint32_t kScaleMin = 93, kScaleMax = 173, kScaleBinades = 10;
constexpr uint32_t kNoScale = 255u << 23;
// A variant: NT 8-row MMA tiles a warp, RG groups of warps with rows of their own over the same keys (four tiles in one
// warp's registers spill and leave four warps an SM). CTAs an SM: the accumulators and the rows of q take 3 D NT / 8
// registers a thread.
constexpr int per_sm(int D, int NT, int RG) { return RG > 1 ? 1 : (D * NT <= 128 ? 3 : 2); }

struct DecodeParams {
  KvView v;
  KvAttnArgs a;
  int max_rows;        // sequences with more rows of a key/value head are left to the other kernel
  int NS;              // stages
  uint32_t stage_bytes;
  float* part;         // [grid][2][R D + 2 R]
  unsigned* counters;  // [grid]
  uint64_t wait_ns;
};

template <int N>
SPEAR_DEVINL void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

SPEAR_DEVINL void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// D = A(16x16, row) * B(16x8, col) + C, f16 inputs, fp32 accumulate.
SPEAR_DEVINL void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with C = 0.
SPEAR_DEVINL void mma_f16_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Bytes 1 and 3 of x as two 16-bit halves.
SPEAR_DEVINL uint32_t odd_bytes(uint32_t x) { return __byte_perm(x, 0, 0x4341); }

SPEAR_DEVINL uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int kThreads>
SPEAR_DEVINL void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// Units of a sequence: per head its tiles and kItemCost for what an item costs beside them.
SPEAR_DEVINL int64_t seq_units(const DecodeParams& p, const KvSeq& s) {
  return s.n > 0 && s.n * p.v.group <= p.max_rows ? (int64_t)(kItemCost + s.tiles) * p.v.n_kv_heads : 0;
}

// A position in the list of units: unit `off` of an item, the first kItemCost of which are no tiles.
struct Cursor {
  int64_t u;
  int b, h, off;
  KvSeq s;
};

// A CTA's share of the item that its cursor stands at (or at the end of): tiles [t0, t1), counted from s.lo.
struct Segment {
  int t0, t1;
};

// (The cursor goes on to the next item only when that is asked for, so that an item's numbers are held once.)
SPEAR_DEVINL bool next_segment(const DecodeParams& p, Cursor& c, int64_t u1, Segment& g) {
  while (c.u < u1) {
    if (c.off == kItemCost + c.s.tiles) {
      c.off = 0;
      if (++c.h == p.v.n_kv_heads) {
        c.h = 0;
        do {
          ++c.b;
          c.s = kv_seq(p.v, p.a, c.b, kTile);
        } while (seq_units(p, c.s) == 0);
      }
    }
    const int end = (int)min((int64_t)kItemCost + c.s.tiles, c.off + (u1 - c.u));
    g.t0 = max(0, c.off - kItemCost);
    g.t1 = max(0, end - kItemCost);
    c.u += end - c.off;
    c.off = end;
    if (g.t1 > g.t0) return true;
  }
  return false;
}

SPEAR_DEVINL unsigned add_acq_rel(unsigned* p, unsigned x) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(x) : "memory");
  return old;
}

SPEAR_DEVINL void ldcg_row(const float* p, float (&v)[4]) {
  const float4 x = __ldcg(reinterpret_cast<const float4*>(p));
  v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
SPEAR_DEVINL void ldcg_row(const float* p, float (&v)[2]) {
  const float2 x = __ldcg(reinterpret_cast<const float2*>(p));
  v[0] = x.x, v[1] = x.y;
}

SPEAR_DEVINL int64_t scan_inclusive(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

template <int D, int NT, int RG>
__global__ void __launch_bounds__(32 * (kKeyWarps * RG + 1), per_sm(D, NT, RG))
    decode_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kWarps = kKeyWarps * RG, kThreads = 32 * (kWarps + 1);
  constexpr int R = 8 * NT * RG;
  constexpr int BB = 16 * (D + 8);
  constexpr int KW = D / 32;       // code words of a K row a lane
  constexpr int VW = D / 64;       // code words of a V row a lane
  constexpr int E = D / 32;        // elements of a result row a lane
  constexpr int OS = D + 4;        // row stride of the joined results
  constexpr int kPart = R * D + 2 * R;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kMaxStages;
  int64_t* scan = reinterpret_cast<int64_t*>(empty + kMaxStages);  // [kScan] sums
  int* found = reinterpret_cast<int*>(scan + kScan);
  static_assert(kWarps < kScan, "");
  float* ml = reinterpret_cast<float*>(smem + 512);                // [kKeyWarps][R][2]
  float* om = ml + kKeyWarps * R * 2;                              // [kKeyWarps][R][OS]
  const uint32_t om_bytes = (kKeyWarps * R * (2 + OS)) * 4;
  const uint32_t stages_at = smem_u32(smem) + 512 + (om_bytes + 127) / 128 * 128;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < p.NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kWarps);
    }
    fence_mbar_init();
  }

  kv_follow();
  // ---- this CTA's units [u0, u1) and the item that u0 falls into; every warp on its own for up to 32 sequences,
  // so that nothing waits
  Cursor c;
  int64_t U = 0, G, u0, u1, at;
  const int64_t cta = blockIdx.x;
  auto share = [&](int items) {
    // Where there is little work, a whole number of CTAs an item (if the items are alike, none has shares of two), of
    // some kMinUnits each: joining costs as much as a few tiles.
    const int64_t mean = div_u64(U, max(items, 1));
    G = min((int64_t)gridDim.x, items * max((int64_t)1, div_u64(mean + kMinUnits / 2, kMinUnits)));
    const int64_t x = G > 0 ? div_u64((cta + (lane & 1)) * U, G) : 0;
    u0 = __shfl_sync(0xffffffffu, x, 0);
    u1 = __shfl_sync(0xffffffffu, x, 1);
  };
  if (p.a.n_seqs <= 32) {
    if (lane < p.a.n_seqs) c.s = kv_seq(p.v, p.a, lane, kTile);
    const int64_t own = lane < p.a.n_seqs ? seq_units(p, c.s) : 0, incl = scan_inclusive(own, lane);
    U = __shfl_sync(0xffffffffu, incl, 31);
    share(__popc(__ballot_sync(0xffffffffu, own > 0)) * p.v.n_kv_heads);
    c.b = __ffs(__ballot_sync(0xffffffffu, u0 < incl)) - 1;
    at = u0 - __shfl_sync(0xffffffffu, incl - own, c.b & 31);
    __syncthreads();  // the barriers are in place
    if (cta >= G) return;
  } else {
    int items = 0;
    for (int b = tid; b < p.a.n_seqs; b += kThreads) {
      const int64_t own = seq_units(p, kv_seq(p.v, p.a, b, kTile));
      U += own;
      items += own > 0;
    }
    items = __syncthreads_count(items) * p.v.n_kv_heads;  // at least, with more sequences than threads
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) U += __shfl_xor_sync(0xffffffffu, U, o);
    if (lane == 0) scan[warp] = U;
    __syncthreads();
    U = 0;
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) U += scan[w];
    share(items);
    if (cta >= G) return;
    int64_t before = 0;
    for (int b0 = 0;; b0 += 32) {
      const int b = b0 + lane;
      const int64_t own = b < p.a.n_seqs ? seq_units(p, kv_seq(p.v, p.a, b, kTile)) : 0;
      const int64_t incl = before + scan_inclusive(own, lane);
      before = __shfl_sync(0xffffffffu, incl, 31);
      if (u0 < before) {
        const int l = __ffs(__ballot_sync(0xffffffffu, u0 < incl)) - 1;
        c.b = b0 + l;
        at = u0 - __shfl_sync(0xffffffffu, incl - own, l);
        break;
      }
    }
  }
  c.u = u0;
  c.s = kv_seq(p.v, p.a, c.b, kTile);
  const unsigned item = kItemCost + c.s.tiles;
  c.h = (int)div_u64(at, item);
  c.off = (int)(at - (int64_t)c.h * item);
  Segment sg;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    int st = 0;
    unsigned phase = 0;
    bool bad = false;
    int issued = 0;
    while (!bad && next_segment(p, c, u1, sg)) {
      const int blocks = (c.s.L + 15) / 16, first = first_key(p.a, c.s.L - c.s.n) / 16;  // pages before may be gone
      for (int i = sg.t0; i < sg.t1; ++i) {
        const int blk = (c.s.lo + i) * kBlocksPerTile + lane;
        const uint8_t* src = nullptr;
        if (lane < kBlocksPerTile && blk >= first && blk < blocks) {
          const int pg = p.a.page_table[(int64_t)c.b * p.a.ld_pt + blk / p.v.bpp];
          if (pg >= 0 && pg < p.v.n_pages)
            src = p.v.pool + (((int64_t)pg * p.v.n_kv_heads + c.h) * p.v.bpp + blk % p.v.bpp) * BB;
          else
            atomicOr(p.v.status, kStatusBadIndex);
        }
        const unsigned copies = __popc(__ballot_sync(0xffffffffu, src != nullptr));
        if (issued >= p.NS && !mbar_wait_bounded(empty + st, phase ^ 1u, p.wait_ns)) bad = true;
        bad = __any_sync(0xffffffffu, bad);
        if (bad) {
          if (lane == 0) atomicOr(p.v.status, kStatusTimeoutPipe);
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(full + st, copies * BB);
        __syncwarp();
        if (src) bulk_g2s_shared_u32(stages_at + st * p.stage_bytes + lane * BB, src, BB, full + st);
        issued = min(issued + 1, p.NS);
        if (++st == p.NS) st = 0, phase ^= 1u;
      }
    }
    // the copies in flight land before the CTA's shared memory is given back
    for (int i = 0; i < issued; ++i) {
      if (st == 0) st = p.NS, phase ^= 1u;
      --st;
      mbar_wait_bounded(full + st, phase, p.wait_ns);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  const int kw = warp % kKeyWarps, row0 = warp / kKeyWarps * 8 * NT;  // this warp's keys and rows
  int st = 0;
  unsigned phase = 0;
  bool bad = false;

  while (next_segment(p, c, u1, sg)) {
    const int len = sg.t1 - sg.t0;
    const KvSeq& s = c.s;
    const int rows = s.n * p.v.group;

    // the rows as f16 B fragments, their sums and their scales
    uint32_t qf[NT][D / 16][2];
    float qs[NT][2], qi[NT][2];
    int hi[NT][2];  // last visible key of this lane's columns 2 t, 2 t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      uint4 w[KW];
#pragma unroll
      for (int i = 0; i < KW; ++i) w[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const __nv_bfloat16* src = p.a.q + (int64_t)(s.row + r / p.v.group) * p.a.ld_q +
                                   (int64_t)(c.h * p.v.group + r % p.v.group) * D + t * (D / 4);
#pragma unroll
        for (int i = 0; i < KW; ++i) w[i] = reinterpret_cast<const uint4*>(src)[i];
      }
      float x = 0.f, top = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t e[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float lo = __uint_as_float(e[k] << 16), up = __uint_as_float(e[k] & 0xFFFF0000u);
          x += lo + up;
          top = fmaxf(top, fmaxf(fabsf(lo), fabsf(up)));
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      // a power of two that brings the row's largest element to 2^14 .. 2^15 (less leaves more to qi, which is to stay finite:
      // it does for rows below 2^118 / scale)
      const uint32_t es = min(268u - (__float_as_uint(top) >> 23), 253u);
      const float up2 = __uint_as_float(es << 23), down = __uint_as_float((254u - es) << 23);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint32_t e[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        // elements (j, j + 4) and (j + 1, j + 5), j even, meet lo and lo + 16 hi: q0 lo + q1 hi = (q0 - q1 / 16) lo +
        // (q1 / 16) (lo + 16 hi), the difference taken with what f16 holds of q1 / 16
        auto pair = [&](int j) {
          const uint32_t a = e[j / 2], b = e[j / 2 + 2];
          const uint32_t odd = pack_f16x2(up2 * 0.0625f * __uint_as_float(a & 0xFFFF0000u),
                                          up2 * 0.0625f * __uint_as_float(b & 0xFFFF0000u));
          if (j & 1) return odd;
          const float2 o = __half22float2(*reinterpret_cast<const __half2*>(&odd));
          return pack_f16x2(fmaf(up2, __uint_as_float(a << 16), -o.x), fmaf(up2, __uint_as_float(b << 16), -o.y));
        };
        qf[nt][2 * i][0] = pair(0);
        qf[nt][2 * i][1] = pair(1);
        qf[nt][2 * i + 1][0] = pair(2);
        qf[nt][2 * i + 1][1] = pair(3);
      }
      // a row with an infinity is NaN, as its result is (minus infinity alone would look like a mask's)
      if (top == INFINITY) x = NAN;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qs[nt][k] = __shfl_sync(0xffffffffu, x, (2 * t + k) * 4) * p.a.scale_log2;
        // codes read as c 2^-24
        qi[nt][k] = __shfl_sync(0xffffffffu, down, (2 * t + k) * 4) * (16777216.f * p.a.scale_log2);
        hi[nt][k] = s.L - s.n + min((row0 + nt * 8 + 2 * t + k) / p.v.group, s.n - 1);
      }
    }
    float acc[D / 16][NT][4];
    float m[NT][2], l[NT][2], off[NT][2];
    uint32_t low_s = kNoScale;  // bits of the lowest value scale that f16 takes; none has been met yet
    float lazy = kLazy;         // kLazy + k
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][nt][e] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) m[nt][k] = -INFINITY, l[nt][k] = 0.f, off[nt][k] = 0.f;
    }

    for (int i = 0; i < len; ++i) {
      const int key0 = (s.lo + sg.t0 + i) * kTile + kw * 32;
      if (!bad && !mbar_wait_bounded(full + st, phase, p.wait_ns)) {
        bad = true;
        if (lane == 0) atomicOr(p.v.status, kStatusTimeoutPipe);
      }
      bad = __any_sync(0xffffffffu, bad);
      const uint32_t base = stages_at + st * p.stage_bytes + kw * 2 * BB;
      // this lane's row of the four 8 x 8 matrices of 16-bit words: key lane % 16 (its low 8 first), chunk lane / 8 % 2
      const uint32_t vrow = base + 8 * D + ((lane & 7) + (lane >> 4) * 8) * (D / 2) + ((lane >> 3) & 1) * 16;
      auto tile = [&](auto masked) {
        // the value scale of one key a lane, looked at below
        const uint32_t sv = lds32(base + (lane >> 4) * BB + 16 * D + 64 + 4 * (lane & 15));
        float sc[2][NT][4];
        // ---- scores
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t blk = base + mt * BB;
          uint32_t wa[KW], wb[KW];
          lds_words(blk + g * (D / 2) + t * (D / 8), wa);
          lds_words(blk + (8 + g) * (D / 2) + t * (D / 8), wb);
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            // bytes 0 and 2, or 1 and 3, of the word as lo + 16 hi, and lo
            const uint32_t x = j & 1 ? odd_bytes(wa[j / 2]) : wa[j / 2] & 0x00FF00FFu;
            const uint32_t y = j & 1 ? odd_bytes(wb[j / 2]) : wb[j / 2] & 0x00FF00FFu;
            const uint32_t a[4] = {x & 0x000F000Fu, y & 0x000F000Fu, x, y};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (j == 0)
                mma_f16_16816_first(sc[mt][nt], a, qf[nt][j][0], qf[nt][j][1]);
              else
                mma_f16_16816(sc[mt][nt], a, qf[nt][j][0], qf[nt][j][1]);
            }
          }
          const uint32_t pa = lds32(blk + 16 * D + 4 * g), pb = lds32(blk + 16 * D + 4 * (8 + g));
          const float s0 = __uint_as_float(pa << 16), o0 = __uint_as_float(pa & 0xFFFF0000u);
          const float s1 = __uint_as_float(pb << 16), o1 = __uint_as_float(pb & 0xFFFF0000u);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            sc[mt][nt][0] = fmaf(s0 * qi[nt][0], sc[mt][nt][0], o0 * qs[nt][0]);
            sc[mt][nt][1] = fmaf(s0 * qi[nt][1], sc[mt][nt][1], o0 * qs[nt][1]);
            sc[mt][nt][2] = fmaf(s1 * qi[nt][0], sc[mt][nt][2], o1 * qs[nt][0]);
            sc[mt][nt][3] = fmaf(s1 * qi[nt][1], sc[mt][nt][3], o1 * qs[nt][1]);
          }
        }
        bool see[2][NT][4];
        if constexpr (masked) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + mt * 16 + g + 8 * (e >> 1), last = hi[nt][e & 1];
                see[mt][nt][e] = key <= last && (p.a.window == 0 || key > last - p.a.window);
                if (!see[mt][nt][e]) sc[mt][nt][e] = -INFINITY;
              }
        }
        // ---- running maximum
        bool over = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            top[nt][k] = fmaxf(fmaxf(sc[0][nt][k], sc[0][nt][k + 2]), fmaxf(sc[1][nt][k], sc[1][nt][k + 2]));
            over |= top[nt][k] > m[nt][k] + lazy;
          }
        // Scales that f16 takes? (0, of a row of one value, it does not.) Of keys that some row sees: in other places may
        // stand what earlier work has left, and the results' bits must not follow it.
        const uint32_t scale = sv << 16;
        bool counts = true;
        if constexpr (masked) counts = key0 + lane < s.L && (p.a.window == 0 || key0 + lane > s.L - s.n - p.a.window);
        auto odd = [&] { return counts && scale - low_s > (kScaleBinades << 23 | 0x7FFFFF); };
        bool wide = false;
        if (__any_sync(0xffffffffu, over || odd())) {  // one vote in nearly all cases
          const float below = lazy - kLazy;  // m is so much below the maximum
          const uint32_t ex = scale >> 23 & 255u;
          const uint32_t most = __reduce_max_sync(
              0xffffffffu, counts && ex - 1u < 254u ? min(max(ex, kScaleMin), kScaleMax) : 0u);
          if (low_s == kNoScale ? most > 0 : most > (low_s >> 23) + kScaleBinades) {
            low_s = (most - kScaleBinades) << 23;
            lazy = kLazy + 133.f - (float)most;
          }
          wide = __any_sync(0xffffffffu, odd());
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float x = top[nt][k];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
              const float mn = fmaxf(m[nt][k] + below, x) - (lazy - kLazy);
              const float f = m[nt][k] == -INFINITY ? 0.f : ex2(m[nt][k] - mn);
              m[nt][k] = mn;
              l[nt][k] *= f;
              off[nt][k] *= f;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) acc[j][nt][k] *= f, acc[j][nt][k + 2] *= f;
            }
        }
        float mu[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) mu[nt][k] = m[nt][k] == -INFINITY ? 0.f : m[nt][k];
        // ---- weights, and the values
        auto values = [&](auto wide) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t blk = base + mt * BB;
          const uint32_t pa = lds32(blk + 16 * D + 64 + 4 * g), pb = lds32(blk + 16 * D + 64 + 4 * (8 + g));
          const float vs[2] = {__uint_as_float(pa << 16), __uint_as_float(pb << 16)};
          const float vo[2] = {fmaf(8.f, vs[0], __uint_as_float(pa & 0xFFFF0000u)),
                               fmaf(8.f, vs[1], __uint_as_float(pb & 0xFFFF0000u))};
          uint32_t bf[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = e & 1, y = e >> 1;
              const float pe = ex2(sc[mt][nt][e] - mu[nt][k]);
              l[nt][k] += pe;
              w[e] = pe * vs[y];
              float o = pe * vo[y];
              if constexpr (masked) {
                if (!see[mt][nt][e]) w[e] = 0.f, o = 0.f;  // 0 x NaN of a key that the row does not see
              }
              off[nt][k] += o;
            }
            bf[nt][0] = movmatrix(wide ? pack_bf16x2(w[0], w[1]) : pack_f16x2(w[0], w[1]));
            bf[nt][1] = movmatrix(wide ? pack_bf16x2(w[2], w[3]) : pack_f16x2(w[2], w[3]));
          }
#pragma unroll
          for (int i2 = 0; i2 < VW; ++i2) {
            // 8 keys x 32 channels each: keys 0..7 and 8..15 of two neighbouring 16-byte chunks; a register holds
            // four channels of keys 2 t and 2 t + 1
            uint32_t y[4];
            ldmatrix_x4_trans(y, vrow + mt * BB + i2 * 32);
            // even j: the low nibble of byte j / 2, (lo - 8) 2^-9; odd j: all of the byte, (lo + 16 hi - 136) 2^-9
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t a[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t byte = j < 2 ? y[x] & 0x00FF00FFu : odd_bytes(y[x]);
                const uint32_t c = j & 1 ? byte : byte & 0x000F000Fu;
                if constexpr (wide)
                  a[x] = bf16x2_fma(c, 0x7D807D80u /* 2^124 */, j & 1 ? 0xBE88BE88u : 0xBC80BC80u);
                else
                  a[x] = f16x2_fma(c, 0x78007800u /* 2^15 */, j & 1 ? 0xB440B440u : 0xA400A400u);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (wide)
                  mma_bf16_16816(acc[i2 * 4 + j][nt], a, bf[nt][0], bf[nt][1]);
                else
                  mma_f16_16816(acc[i2 * 4 + j][nt], a, bf[nt][0], bf[nt][1]);
              }
            }
          }
        }
        };
        if (wide)
          values(std::true_type{});
        else
          values(std::false_type{});
      };
      if (!bad && key0 < s.L) {
        // does some row not see all 32 keys?
        const bool masked = key0 + 31 > s.L - s.n || (p.a.window > 0 && key0 <= s.L - 1 - p.a.window);
        if (masked)
          tile(std::true_type{});
        else
          tile(std::false_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st);
      if (++st == p.NS) st = 0, phase ^= 1u;
    }

    // ---- join the four warps' states
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], o);
          off[nt][k] += __shfl_xor_sync(0xffffffffu, off[nt][k], o);
        }
        const int r = row0 + nt * 8 + 2 * t + k;
        if (g == 0) {
          ml[(kw * R + r) * 2] = m[nt][k];
          ml[(kw * R + r) * 2 + 1] = l[nt][k];
        }
        float* dst = om + (kw * R + r) * OS + g * 4;
#pragma unroll
        for (int i2 = 0; i2 < VW; ++i2)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float4 o4;
            const int e = k + 2 * y;
            const float a0 = acc[i2 * 4][nt][e], a2 = acc[i2 * 4 + 2][nt][e];
            o4.x = fmaf(a0, 512.f, off[nt][k]);
            o4.y = fmaf(acc[i2 * 4 + 1][nt][e] - a0, 32.f, off[nt][k]);  // (byte - lo) / 16
            o4.z = fmaf(a2, 512.f, off[nt][k]);
            o4.w = fmaf(acc[i2 * 4 + 3][nt][e] - a2, 32.f, off[nt][k]);
            *reinterpret_cast<float4*>(dst + i2 * 64 + y * 32) = o4;
          }
      }
    consumer_sync<32 * kWarps>();
    const bool whole = len == s.tiles;
    // a segment that starts its item in this CTA and one that goes on with an earlier CTA's have a slot each
    float* slot = p.part + (cta * 2 + (sg.t0 == 0 ? 1 : 0)) * kPart;
    auto write_row = [&](int r, const float (&o)[E], float inv) {
      if (r >= rows) return;
      __nv_bfloat16* dst = p.a.out + (int64_t)(s.row + r / p.v.group) * p.a.ld_out +
                           (int64_t)(c.h * p.v.group + r % p.v.group) * D + lane * E;
      uint32_t w[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) w[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
      if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(dst) = w[0];
    };
    for (int r = warp; r < min(R, rows); r += kWarps) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKeyWarps; ++w) M = fmaxf(M, ml[(w * R + r) * 2]);
      float L = 0.f, o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kKeyWarps; ++w) {
        const float mw = ml[(w * R + r) * 2];
        const float f = mw == -INFINITY ? (ml[(w * R + r) * 2 + 1] == 0.f ? 0.f : 1.f) : ex2(mw - M);
        L = fmaf(f, ml[(w * R + r) * 2 + 1], L);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(f, om[(w * R + r) * OS + lane * E + e], o[e]);
      }
      if (whole) {
        write_row(r, o, L == 0.f ? 0.f : 1.f / L);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) slot[r * D + lane * E + e] = o[e];
        if (lane == 0) slot[R * D + 2 * r] = M, slot[R * D + 2 * r + 1] = L;
      }
    }
    if (!whole) {
      // CTAs ca .. cb hold the item's units
      const int64_t unit0 = c.u - c.off + kItemCost;  // of tile 0
      const int64_t x0 = div_u64(((lane & 1) ? unit0 + s.tiles : unit0 + 1) * G - 1, U);
      const int ca = (int)__shfl_sync(0xffffffffu, x0, 0), parts = (int)__shfl_sync(0xffffffffu, x0, 1) - ca + 1;
      consumer_sync<32 * kWarps>();
      // release what the barrier above has collected from the four warps, acquire what the others released
      if (tid == 0) found[0] = add_acq_rel(p.counters + ca, 1u) == (unsigned)(parts - 1);
      consumer_sync<32 * kWarps>();
      if (found[0]) {
        if (tid == 0) p.counters[ca] = 0;
        auto part = [&](int x) { return p.part + ((int64_t)(ca + x) * 2 + (x == 0)) * kPart; };
        for (int r = warp; r < min(R, rows); r += 2 * kWarps) {  // two rows at a time, 16 loads in flight
          float M[2] = {-INFINITY, -INFINITY};
          for (int x = lane; x < parts; x += 32)
#pragma unroll
            for (int k = 0; k < 2; ++k) M[k] = fmaxf(M[k], __ldcg(part(x) + R * D + 2 * (r + k * kWarps)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) M[k] = fmaxf(M[k], __shfl_xor_sync(0xffffffffu, M[k], o));
          float L[2] = {0.f, 0.f}, o[2][E];
#pragma unroll
          for (int e = 0; e < E; ++e) o[0][e] = o[1][e] = 0.f;
          for (int x0 = 0; x0 < parts; x0 += 32) {
            float f[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};  // of part x0 + lane
            if (x0 + lane < parts) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float2 ml2 = __ldcg(reinterpret_cast<const float2*>(part(x0 + lane) + R * D) + r + k * kWarps);
                l[k] = ml2.y;
                f[k] = ml2.x == -INFINITY ? (l[k] == 0.f ? 0.f : 1.f) : ex2(ml2.x - M[k]);
              }
            }
            const int n = min(32, parts - x0);
            for (int y0 = 0; y0 < n; y0 += 8) {
              float v[8][2][E];
#pragma unroll
              for (int y = 0; y < 8; ++y)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  ldcg_row(part(x0 + min(y0 + y, n - 1)) + (r + k * kWarps) * D + lane * E, v[y][k]);
#pragma unroll
              for (int y = 0; y < 8; ++y)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float fy = __shfl_sync(0xffffffffu, f[k], (y0 + y) & 31);
                  const float ly = __shfl_sync(0xffffffffu, l[k], (y0 + y) & 31);
                  if (y0 + y < n) {
                    L[k] = fmaf(fy, ly, L[k]);
#pragma unroll
                    for (int e = 0; e < E; ++e) o[k][e] = fmaf(fy, v[y][k][e], o[k][e]);
                  }
                }
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) write_row(r + k * kWarps, o[k], L[k] == 0.f ? 0.f : 1.f / L[k]);
        }
      }
    }
    consumer_sync<32 * kWarps>();  // the joined results have been read
  }
}

template <int D, int NT, int RG>
spear_status_t launch(const spear_kv_s* h, DecodeParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  if (smem_limit_once(reinterpret_cast<const void*>(decode_kernel<D, NT, RG>), done) != cudaSuccess) return SPEAR_ERR_CUDA;
  constexpr int kPerSm = per_sm(D, NT, RG);
  constexpr uint32_t om = ((kKeyWarps * 8 * NT * RG * (2 + D + 4)) * 4 + 127) / 128 * 128;
  constexpr uint32_t stage = kBlocksPerTile * 16 * (D + 8);
  constexpr int kRoom = (227 * 1024 / kPerSm - 1024 - 512 - (int)om) / (int)stage;
  p.stage_bytes = stage;
  p.NS = kRoom < kMaxStages ? kRoom : kMaxStages;
  static_assert(kRoom >= 2, "two stages at least");
  const size_t smem = 512 + om + (size_t)p.NS * stage;
  return kv_launch(decode_kernel<D, NT, RG>, dim3(h->sm_count * kPerSm), 32 * (kKeyWarps * RG + 1), smem, stream, p);
}

}  // namespace
}  // namespace spear

using namespace spear;

size_t kv_decode_workspace(const spear_kv_s* h) {
  const int D = h->view.D;
  int rows = 0;  // of all CTAs of an SM
  for (int nt = 1; nt <= 2; ++nt) rows = std::max(rows, 8 * nt * per_sm(D, nt, 1));
  rows = std::max(rows, 32 * per_sm(D, 2, 2));
  return (size_t)h->sm_count * 2 * rows * (D + 2) * sizeof(float);
}

spear_status_t kv_launch_decode(const spear_kv_s* h, const KvAttnArgs& a, int nt, float* part, unsigned* counters,
                                cudaStream_t stream) {
  DecodeParams p;
  p.v = h->view;
  p.a = a;
  p.max_rows = 8 * nt;
  p.part = part;
  p.counters = counters;
  p.wait_ns = 100000000ull;
  const bool wide = h->view.D == 128;
  switch (nt) {
    case 1: return wide ? launch<128, 1, 1>(h, p, stream) : launch<64, 1, 1>(h, p, stream);
    case 2: return wide ? launch<128, 2, 1>(h, p, stream) : launch<64, 2, 1>(h, p, stream);
    default: return wide ? launch<128, 2, 2>(h, p, stream) : launch<64, 2, 2>(h, p, stream);
  }
}

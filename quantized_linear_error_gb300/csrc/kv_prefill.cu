// Attention of many query rows over the paged 4-bit cache (prefill chunks) on
// the tcgen05 tensor cores.
//
// For each (sequence, key/value head) the rows are the query tokens times the
// heads that share it, in tiles of 256 (two MMA tiles of 128); a row meets its
// visible keys in tiles of 128:
//   S = Q K^T (fp32, tensor memory), P = 2^(scale (S - m)) (16 bits, written
//   over S), O += P V (fp32, tensor memory), l += sum P;  out = O / l.
// Bound by the tensor cores, 4 D flops a (row, key) pair, with the smaller
// units close behind: per 256 x 128 block of D = 128 the MMAs take 2048 cycles
// of an SM, their operands in shared memory 1536 at 128 bytes a cycle, the
// dequantised tiles' stores 512; a block takes some 2800 here, the chain
// scores, weights, product of one half being longer than the other half's
// products that hide it. Measured, D = 128: a prompt of 8192 tokens, 32 heads
// over 8 (550 GFLOP), 387 us or 1.42 PFLOP/s in bursts, 72% of a library
// product's rate, and 403 to 411 us once the power limit lowers the clocks; 320
// tokens behind 7901 (42 GFLOP) 44.5 us, of which 5 are the start and 8 partial
// results and their join.
//
// A row tile with at most 128 rows leaves the other half idle, and a key tile
// then takes 2700 cycles, of which the dequantisers need 2200: both halves at
// every other tile of it were 5% slower (32 sequences x 12 drafts x 4 heads at
// 4000 keys).
//
//  - Operands are f16, whose 11 bits hold queries and codes' values with an
//    error far below that of the bf16 result (bf16 operands doubled it). Rows
//    of Q are scaled by a power of two each. 32 keys at a time may leave f16's
//    range: their K are scaled by a power of two each, which the softmax takes
//    back from their columns, and their V and P go through bf16.
//  - Dequantisers (8 warps, two threads a key) turn a tile's packed rows into
//    code * scale + offset, rounded once, in 128-byte-swizzled shared memory.
//    Both tiles are stored key by key: K is the K-major B operand of S, V the
//    MN-major B operand of O, so nothing is transposed. A code word's pairs come
//    out as elements (0, 4), (1, 5), (2, 6), (3, 7); Q's rows are permuted
//    alike, and O's columns are put back in the epilogue. Keys past the
//    sequence's end or before the window become zeros, and a key whose V is not
//    finite is moved to its K (V zero, K NaN): rows that see it get NaN, the mask
//    keeps it from the others (0 x NaN in O += P V would not).
//  - Two softmax warpgroups, one an MMA tile, one row a thread; P goes from
//    registers to tensor memory in two parts, so that the product with the
//    first 64 keys runs while the other weights are computed. m need not be the
//    maximum: it is taken from a segment's first tile, 8 binades below its
//    maximum, and again only when the weights of 64 keys sum to more than 2^15;
//    no other tile takes a maximum. In between all of f16's range serves: weights
//    keep 8 bits down to 2^-24 of the largest, and are lost below 2^-33 (with the
//    maximum itself for m 2^-16 and 2^-25: thousands of keys of weight 2^-22
//    behind one came out 14% off).
//  - Two warps issue the MMAs, one a half, in turns "product of the last tile,
//    scores of the next": an S overwrites its P only after the product that
//    reads it, which the same warp issued before it.
//  - One warp copies the packed tiles, a bulk copy a 16-token block; one lays
//    out the CTA's work and fetches the coming query rows into L2.
//
// Work: (sequence, head, row tile, key tile) units in this order are split
// evenly over the CTAs (one an SM), an item (row tile) counting as four units
// more than its key tiles. Items that several CTAs share leave partial results,
// which a second small kernel joins in CTA order on all SMs (the last CTA of an
// item to finish, on its own, took 12 us for it).
#include <algorithm>
#include <atomic>

#include "kv_device.cuh"
#include "tcgen05.cuh"

namespace spear {
namespace {

constexpr int kThreads = 640;         // 8 softmax, 8 dequantising, 2 MMA warps, copies, schedule
constexpr int kDeqWarps = 8;
constexpr int kTile = 128;            // keys of a unit
constexpr int kRows = 256;            // rows of an item
constexpr int kBlocksPerTile = kTile / 16;
constexpr int kItemCost = 4;          // units
constexpr int kHeader = 1024;         // barriers, segments
constexpr int kSegs = 4;              // segments in flight
constexpr int kSegReaders = 8 + kDeqWarps + 2 + 1;  // warps that read each segment
constexpr float kBig = 0x1p15f;   // weights up to here fit f16
constexpr float kFresh = 8.f;     // log2 of the largest weight when m is taken
constexpr uint32_t kHintNs = 100;
// setmaxnreg: 256 x 168 + 384 x 48 registers are the 640 x 96 of the launch
constexpr int kJoinRows = 32;

// An item that several CTAs share, written by the CTA that starts it.
struct Join {
  int parts;  // 0: none
  int rows, r0, h, row;
};

struct PrefillParams {
  KvView v;
  KvAttnArgs a;
  unsigned inv_group;  // floor(2^32 / group) + 1, 0 for a group of one
  int max_rows;   // sequences with at most this many rows of a key/value head belong to the other kernel
  float* part;    // [grid][2][2 halves][D + 2][128]
  Join* joins;    // [grid]
  uint64_t wait_ns;
};

// A CTA's share of an item: `len` key tiles from tile `tile0` on.
struct Segment {
  int len;          // 0: the end
  int b, h, L, tile0;
  int first;        // first key that any of the item's rows sees
  int row;          // first query row of the sequence
  int pos0;         // position of the sequence's first query row
  int r0, rows;     // the item's rows of the key/value head: [r0, r0 + rows)
  int whole;        // all of the item's tiles
  int slot;         // else, this share's partial result
};

struct Header {
  uint64_t raw_full[2], raw_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], p_full[2][2], pa_done[2], o_full[2], turn[2], done[2];  // p_full: [64 keys][half]
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Segment seg[kSegs];
  uint32_t tmem;
  // of the last four tiles: per 32 keys bit 0, their K is scaled by 2^-exponent each; bit 1, their V is in bf16
  uint8_t flags[4][4];
  int8_t exponent[4][kTile];
};
static_assert(sizeof(Header) <= kHeader, "");

// R / group for R < 2^27 (the launch checks T x group): the reciprocal's error, below 2^-32, times R stays below
// 1 / group.
SPEAR_DEVINL unsigned div_group(const PrefillParams& p, unsigned R) {
  return p.inv_group ? __umulhi(R, p.inv_group) : R;
}

// Row tile qt of a sequence: its key tiles.
struct Item {
  int first;  // key that a row sees
  int lo, tiles;
  int rows;  // rows of this tile, <= 256
};

SPEAR_DEVINL int row_tiles(const PrefillParams& p, const KvSeq& s) {
  const int rows = s.n * p.v.group;
  return rows > p.max_rows ? (rows + kRows - 1) / kRows : 0;
}

SPEAR_DEVINL Item item_of(const PrefillParams& p, const KvSeq& s, int qt) {
  Item it;
  const int r0 = qt * kRows;
  it.rows = min(kRows, s.n * p.v.group - r0);
  const int t0 = div_group(p, r0), t1 = div_group(p, r0 + it.rows - 1);
  const int last = s.L - s.n + t1;
  it.first = first_key(p.a, s.L - s.n + t0);
  it.lo = it.first / kTile;
  it.tiles = max(1, (last >= 0 ? last / kTile + 1 : 0) - it.lo);
  return it;
}

// Units of one head of a sequence, the whole warp at it.
SPEAR_DEVINL int64_t head_units(const PrefillParams& p, const KvSeq& s, int nqt, int lane) {
  int64_t x = 0;
  for (int qt = lane; qt < nqt; qt += 32) x += kItemCost + item_of(p, s, qt).tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

SPEAR_DEVINL void fail(const PrefillParams& p) { atomicOr(p.v.status, kStatusTimeoutPipe); }

SPEAR_DEVINL KvSeq shuffled(const KvSeq& s, int l) {
  KvSeq r;
  r.n = __shfl_sync(0xffffffffu, s.n, l);
  r.row = __shfl_sync(0xffffffffu, s.row, l);
  r.L = __shfl_sync(0xffffffffu, s.L, l);
  return r;  // lo and tiles are of no use here
}

// The warp that lays out a CTA's work. Every CTA counts all units, finds where
// its equal share begins and hands its segments to the other warps; it also
// fetches the coming items' query rows into L2.
template <int D>
SPEAR_DEVINL void schedule(const PrefillParams& p, Header& hd, int lane) {
  // units of 32 sequences, lane b's in lane b; the lane's sequence is left in `s`
  KvSeq s;
  auto units_of = [&](int b0) {
    const int b = b0 + lane;
    int nqt = 0;
    if (b < p.a.n_seqs) {
      s = kv_seq(p.v, p.a, b, kTile);
      nqt = row_tiles(p, s);
    }
    int64_t own = 0;
    // Many sequences: a lane counts its own's row tiles, beside the others. (One sequence after another, the warp at
    // each, 64 of one row tile took 12 us.) Few with many row tiles: the warp at each.
    const bool alone = nqt <= 2 * __popc(__ballot_sync(0xffffffffu, nqt > 0));
    if (alone) {
      int n = kItemCost * nqt;  // 64 row tiles of 2^23 key tiles at most
      for (int qt = 0; qt < nqt; ++qt) n += item_of(p, s, qt).tiles;
      own = (int64_t)n * p.v.n_kv_heads;
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, !alone); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      const int64_t x = head_units(p, shuffled(s, l), __shfl_sync(0xffffffffu, nqt, l), lane) * p.v.n_kv_heads;
      if (lane == l) own = x;
    }
    return own;
  };
  int64_t U = 0, own = 0, G = 0, u = 0, u1 = 0, before = 0;
  const int64_t cta = blockIdx.x;
  int b = 0, h = 0, qt = 0, off = 0, nqt = 0;
  bool counted = false;
  for (int b0 = 0;;) {  // once over all sequences for the sum, then to the one that u falls into (one copy of the code)
    if (!counted || p.a.n_seqs > 32) own = units_of(b0);
    if (!counted) {
      int64_t x = own;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      U += x;
      b0 += 32;
      if (b0 < p.a.n_seqs) continue;
      G = min((int64_t)gridDim.x, U);
      if (cta >= G) break;
      x = div_u64((cta + (lane & 1)) * U, G);
      u = __shfl_sync(0xffffffffu, x, 0);
      u1 = __shfl_sync(0xffffffffu, x, 1);
      counted = true;
      b0 = 0;
      continue;
    }
    int64_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, u < before + incl);
    if (past) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      const int64_t hu = div_u64(__shfl_sync(0xffffffffu, own, l), p.v.n_kv_heads);
      int64_t rest = u - before - (__shfl_sync(0xffffffffu, incl, l) - __shfl_sync(0xffffffffu, own, l));
      s = shuffled(s, l);
      nqt = row_tiles(p, s);
      h = (int)div_u64(rest, hu);
      rest -= h * hu;
      for (int q0 = 0; q0 < nqt; q0 += 32) {
        const int cost = q0 + lane < nqt ? kItemCost + item_of(p, s, q0 + lane).tiles : 0;
        int sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += x;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31);
        if (rest < all) {
          const int at = __ffs(__ballot_sync(0xffffffffu, rest < sum)) - 1;
          qt = q0 + at;
          off = (int)rest - (__shfl_sync(0xffffffffu, sum, at) - __shfl_sync(0xffffffffu, cost, at));
          break;
        }
        rest -= all;
      }
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
    b0 += 32;
  }
  Join join = {};
  unsigned n = 0;
  for (bool end = false; !end;) {
    Segment g = {};
    while (u < u1 && g.len == 0) {
      const Item it = item_of(p, s, qt);
      const int stop = (int)min((int64_t)kItemCost + it.tiles, off + (u1 - u));
      const int t0 = max(0, off - kItemCost), t1 = max(0, stop - kItemCost);
      if (t1 > t0) {
        g.len = t1 - t0;
        g.b = b;
        g.h = h;
        g.L = s.L;
        g.tile0 = it.lo + t0;
        g.first = it.first;
        g.row = s.row;
        g.pos0 = s.L - s.n;
        g.r0 = qt * kRows;
        g.rows = it.rows;
        g.whole = g.len == it.tiles;
        g.slot = (int)cta * 2 + (t0 == 0);  // one slot for the share that starts an item, one for a later share
        if (t0 == 0 && !g.whole) {
          const int64_t last = u - off + kItemCost + it.tiles - 1;  // the item's last unit
          join = {(int)(div_u64((last + 1) * G - 1, U) - cta) + 1, it.rows, g.r0, h, s.row};
        }
      }
      u += stop - off;
      off = 0;
      if (u < u1 && ++qt == nqt) {
        qt = 0;
        if (++h == p.v.n_kv_heads) {
          h = 0;
          do {
            ++b;
            s = kv_seq(p.v, p.a, b, kTile);
            nqt = row_tiles(p, s);
          } while (nqt == 0);
        }
      }
    }
    end = g.len == 0;
    const unsigned i = n % kSegs;
    if (n >= kSegs && !warp_wait(&hd.seg_empty[i], ((n / kSegs) & 1u) ^ 1u, p.wait_ns, 1000)) {
      if (lane == 0) {
        fail(p);
        p.joins[cta] = {};
      }
      return;
    }
    if (lane == 0) {
      hd.seg[i] = g;
      mbar_arrive(&hd.seg_full[i]);
    }
    __syncwarp();
    if (n > 0)
      for (int r = lane; r < g.rows; r += 32) {
        const unsigned R = g.r0 + r, tok = div_group(p, R);
        const __nv_bfloat16* q = p.a.q + (int64_t)(g.row + tok) * p.a.ld_q + (int64_t)(g.h * p.v.group + R - tok * p.v.group) * D;
#pragma unroll
        for (int x = 0; x < D; x += 64) prefetch_l2_line(q + x);
      }
    ++n;
  }
  if (lane == 0) p.joins[cta] = join;
}

// Eight codes of a word as four pairs, elements (0, 4), (1, 5), (2, 6), (3, 7): code * scale + offset, rounded once.
// f16: a nibble beneath the exponent of 1024 reads as 1024 + c, or + 16 c; c is taken out exactly.
SPEAR_DEVINL uint4 dequant8_f16(uint32_t w, uint32_t ss, uint32_t oo) {
  const uint32_t u = w >> 8;
  constexpr uint32_t k1024 = 0x64006400u, kNeg1024 = 0xE400E400u, kOne = 0x3C003C00u;
  constexpr uint32_t k16th = 0x2C002C00u, kNeg64 = 0xD400D400u;
  return make_uint4(f16x2_fma(f16x2_fma((w & 0x000F000Fu) | k1024, kOne, kNeg1024), ss, oo),
                    f16x2_fma(f16x2_fma((w & 0x00F000F0u) | k1024, k16th, kNeg64), ss, oo),
                    f16x2_fma(f16x2_fma((u & 0x000F000Fu) | k1024, kOne, kNeg1024), ss, oo),
                    f16x2_fma(f16x2_fma((u & 0x00F000F0u) | k1024, k16th, kNeg64), ss, oo));
}
// bf16: a masked nibble pair reads as tiny values (see decode_frag_unpack), which one exact multiplication brings to
// c 2^-7 or c 2^-3; s_lo = scale 2^7, s_hi = scale 2^3.
SPEAR_DEVINL uint4 dequant8_bf16(uint32_t w, uint32_t s_lo, uint32_t s_hi, uint32_t oo) {
  const uint32_t u = w >> 8;
  constexpr uint32_t k2p126 = 0x7E807E80u, k0 = 0x80008000u;  // x 2^126 - 0
  return make_uint4(bf16x2_fma(bf16x2_fma(w & 0x000F000Fu, k2p126, k0), s_lo, oo),
                    bf16x2_fma(bf16x2_fma(w & 0x00F000F0u, k2p126, k0), s_hi, oo),
                    bf16x2_fma(bf16x2_fma(u & 0x000F000Fu, k2p126, k0), s_lo, oo),
                    bf16x2_fma(bf16x2_fma(u & 0x00F000F0u, k2p126, k0), s_hi, oo));
}

SPEAR_DEVINL void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Half `half` of one key's row: codes (D / 2 bytes at `src`) to row `key` of a swizzled tile, `convert` turning a word
// into 16 bytes.
template <int D, class F>
SPEAR_DEVINL void dequant_row(uint32_t src, uint32_t tile, int key, int half, F convert) {
  constexpr int Q = D / 64;  // 16-byte quarters of the packed row a thread
  // D = 128: quarters in an order of the key's own, so that a quarter warp meets every bank once
  auto quarter = [&](int i) { return Q == 2 ? (i + 2 * half + (key >> 1)) & 3 : half; };
  uint4 w[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) w[i] = lds128(src + quarter(i) * 16);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int q = quarter(i);
    const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    const uint32_t row = tile + (q >> 1) * (kTile * 128) + key * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sts128(row + ((((q & 1) * 4 + j) ^ (key & 7)) * 16), convert(words[j]));
  }
}

// Whether a row with these parameters is safe in f16, 11 bits for its larger elements: scale in 2^-12 .. 2^10, offset
// below 2^14 (the bit patterns of bf16 numbers order like the numbers).
SPEAR_DEVINL bool fits_f16(uint32_t par) {
  return (uint16_t)(par - 0x3980u) < 0x0B00u && (par & 0x7FFF0000u) < 0x46800000u;
}

SPEAR_DEVINL bool finite_par(uint32_t par) {
  return (par & 0x7F80u) != 0x7F80u && (par & 0x7F800000u) != 0x7F800000u;
}

// Eight results in the order of Q's permuted elements, 0, 4, 1, 5, 2, 6, 3, 7, back in their places, as bf16.
SPEAR_DEVINL uint4 unpermute8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[4], x[6]), pack_bf16x2(x[1], x[3]), pack_bf16x2(x[5], x[7]));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ PrefillParams p) {
  constexpr int BB = 16 * (D + 8);
  constexpr uint32_t kTileBytes = kTile * D * 2;   // a K, V or 128-row Q tile
  constexpr uint32_t kRawBytes = kBlocksPerTile * BB;
  constexpr int kPart = (D + 2) * 128;
  extern __shared__ __align__(1024) uint8_t smem[];
  Header& hd = *reinterpret_cast<Header*>(smem);
  const uint32_t q_at = smem_u32(smem) + kHeader;
  const uint32_t k_at = q_at + 2 * kTileBytes, v_at = k_at + 2 * kTileBytes, raw_at = v_at + 2 * kTileBytes;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid & 31;

  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hd.raw_full[i], 1);
      mbar_init(&hd.raw_empty[i], kDeqWarps);
      mbar_init(&hd.k_full[i], kDeqWarps);
      mbar_init(&hd.k_empty[i], 2);
      mbar_init(&hd.v_full[i], kDeqWarps);
      mbar_init(&hd.v_empty[i], 2);
      mbar_init(&hd.q_full[i], 4);
      mbar_init(&hd.s_full[i], 1);
      mbar_init(&hd.p_full[0][i], 4);
      mbar_init(&hd.p_full[1][i], 4);
      mbar_init(&hd.o_full[i], 1);
      mbar_init(&hd.pa_done[i], 1);
      mbar_init(&hd.turn[i], 1);
      mbar_init(&hd.done[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&hd.seg_full[i], 1);
      mbar_init(&hd.seg_empty[i], kSegReaders);
    }
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(&hd.tmem, 512);
    tmem_relinquish();
  }
  __syncwarp();
  kv_follow();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(&hd.tmem), 0);

  // The n-th segment, read by a whole warp; false at the end (or if the wait gave up).
  auto read_segment = [&](unsigned n, Segment& g) {
    const unsigned i = n % kSegs;
    if (!warp_wait(&hd.seg_full[i], (n / kSegs) & 1u, p.wait_ns, kHintNs)) {
      if (lane == 0) fail(p);
      return false;
    }
    const volatile Segment& x = hd.seg[i];
    g.len = __shfl_sync(0xffffffffu, x.len, 0);
    g.b = x.b;
    g.h = x.h;
    g.L = x.L;
    g.tile0 = x.tile0;
    g.first = x.first;
    g.row = x.row;
    g.pos0 = x.pos0;
    g.r0 = x.r0;
    g.rows = __shfl_sync(0xffffffffu, x.rows, 0);
    g.whole = x.whole;
    g.slot = x.slot;
    __syncwarp();
    if (lane == 0) mbar_arrive(&hd.seg_empty[i]);
    return g.len > 0;
  };

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 19) {
      // -------------------------------------------------------------- the CTA's segments, in order
      schedule<D>(p, hd, lane);
    } else if (warp == 18) {
      // -------------------------------------------------------------- copies of the packed tiles
      int st = 0;
      unsigned ph = 0, issued = 0;
      bool ok = true;
      Segment g;
      for (unsigned n = 0; ok && read_segment(n, g); ++n) {
        const int blocks = (g.L + 15) / 16, first = g.first / 16;  // pages before may be gone
        for (int t = 0; t < g.len; ++t) {
          const int blk = (g.tile0 + t) * kBlocksPerTile + lane;
          const uint8_t* src = nullptr;
          if (lane < kBlocksPerTile && blk >= first && blk < blocks) {
            const int pg = p.a.page_table[(int64_t)g.b * p.a.ld_pt + blk / p.v.bpp];
            if (pg >= 0 && pg < p.v.n_pages)
              src = p.v.pool + (((int64_t)pg * p.v.n_kv_heads + g.h) * p.v.bpp + blk % p.v.bpp) * BB;
            else
              atomicOr(p.v.status, kStatusBadIndex);
          }
          const unsigned copies = __popc(__ballot_sync(0xffffffffu, src != nullptr));
          if (issued >= 2 && !warp_wait(&hd.raw_empty[st], ph ^ 1u, p.wait_ns, kHintNs)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&hd.raw_full[st], copies * BB);
          __syncwarp();
          if (src) bulk_g2s_shared_u32(raw_at + st * kRawBytes + lane * BB, src, BB, &hd.raw_full[st]);
          ++issued;
          if (++st == 2) st = 0, ph ^= 1u;
        }
      }
      if (!ok && lane == 0) fail(p);
      for (unsigned i = 0; i < min(issued, 2u); ++i) {  // copies in flight land before the CTA ends
        if (st == 0) st = 2, ph ^= 1u;
        --st;
        warp_wait(&hd.raw_full[st], ph, p.wait_ns, kHintNs);
      }
    } else {
      // -------------------------------------------------------------- MMA issue, one warp a half, uniform
      const int i = warp - 16;
      const uint32_t leader = elect_leader();
      const uint32_t idesc_s = idesc_f16_f32(128, kTile);
      const uint32_t idesc_o = idesc_f16_f32(128, D) | kIdescBMnMajor;
      constexpr uint32_t kHalfWide = (idesc_bf16_f32(128, D) - idesc_f16_f32(128, D)) / 2;
      // a descriptor's address field counts 16 bytes and holds any shared-memory address: steps are added to it
      const uint64_t q_desc = sw128_kmajor_desc(q_at + i * kTileBytes), k_desc = sw128_kmajor_desc(k_at);
      const uint64_t v_desc = sw128_mnmajor_desc(v_at, kTile * 128);
      const uint32_t s_d = tmem + 128 * i, o_d = tmem + 256 + 128 * i;
      unsigned kc = 0, q_ph = 0, p_ph = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, unsigned parity) {
        ok = warp_wait(bar, parity, p.wait_ns, kHintNs);
        return ok;
      };
      // The halves take turns, "product of the last tile, scores of the next" each, so that one half's softmax
      // runs beside the other's products; left alone they fall into step and wait for the tensor cores together.
      unsigned turn_ph = i == 0 ? 1u : 0u;  // half 0's first turn needs no one's leave
      auto take_turn = [&] {
        const bool got = wait(&hd.turn[i], turn_ph);
        turn_ph ^= 1u;
        return got;
      };
      Segment g;
      unsigned n = 0;
      bool more = read_segment(n++, g);
      if (more) take_turn() && wait(&hd.k_full[0], 0);
      while (more && ok) {
        const int len = g.len;
        const bool mine = g.rows > 128 * i;
        more = read_segment(n++, g);
        for (int k = 0; k < len; ++k, ++kc) {
          const unsigned st = kc & 1u, ph = (kc >> 1) & 1u;
          if (mine) {
            if (k == 0) {
              if (!wait(&hd.q_full[i], q_ph)) break;
              q_ph ^= 1u;
            }
            tc_fence_after_sync();
            const uint64_t kd = k_desc + st * (kTileBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              constexpr uint32_t kBlock = (128 * 128) >> 4;
              umma_bf16(leader, s_d, q_desc + (kk / 4) * kBlock + (kk % 4) * 2,
                        kd + (kk / 4) * kBlock + (kk % 4) * 2, idesc_s, kk != 0);
            }
            umma_commit(leader, &hd.s_full[i]);
            umma_commit(leader, &hd.k_empty[st]);
          } else if (leader) {
            mbar_arrive(&hd.k_empty[st]);
          }
          if (leader) mbar_arrive(&hd.turn[i ^ 1]);
          // (a reduction's result is uniform for the compiler, so that the descriptors below stay in uniform registers)
          const uint32_t flags =
              __reduce_or_sync(0xffffffffu, *reinterpret_cast<const volatile uint32_t*>(hd.flags[kc & 3]));
          // what the turn needs, before taking it: the next K tile (dequantised after this V tile) or this V tile
          if (more || k + 1 < len ? !wait(&hd.k_full[st ^ 1u], ((kc + 1) >> 1) & 1u) : !wait(&hd.v_full[st], ph)) break;
          if (!take_turn()) break;
          if (mine && !wait(&hd.p_full[0][i], p_ph)) break;
          if (mine) {
            const uint64_t vd = v_desc + st * (kTileBytes >> 4);
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // the first 64 keys' product runs while the others' weights are computed
              if (x && !wait(&hd.p_full[1][i], p_ph)) break;
              tc_fence_after_sync();
#pragma unroll
              for (int kk = 4 * x; kk < 4 * x + 4; ++kk)
                umma_ts_bf16(leader, o_d, s_d + 8 * kk, vd + kk * (2048 >> 4),
                             idesc_o + (flags >> (8 * (kk / 2)) & 2u) * kHalfWide, kk == 0 ? (k != 0) : 1u);
              if (x == 0) umma_commit(leader, &hd.pa_done[i]);
            }
            if (!ok) break;
            p_ph ^= 1u;
            if (k + 1 == len) umma_commit(leader, &hd.o_full[i]);
            umma_commit(leader, &hd.v_empty[st]);
          } else if (leader) {
            mbar_arrive(&hd.v_empty[st]);
          }
        }
      }
      if (!ok && leader) fail(p);
      if (leader) mbar_arrive(&hd.turn[i ^ 1]);
      // nothing of this CTA's is still running on the tensor cores when the others go on to the end
      umma_commit(leader, &hd.done[i]);
      if (!warp_wait(&hd.done[i], 0, p.wait_ns, 0) && leader) fail(p);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- dequantisers, two threads a key
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    const int key = (tid - 256) & 127, half = (tid - 256) >> 7;
    const uint32_t blk_at = raw_at + (key / 16) * BB;
    const int r = key & 15;
    bool ok = true;
    unsigned k = 0;
    Segment g;
    for (unsigned n = 0; ok && read_segment(n, g); ++n) {
      for (int t = 0; t < g.len; ++t, ++k) {
        const unsigned st = k & 1u, ph = (k >> 1) & 1u;
        const uint32_t blk = blk_at + st * kRawBytes;
        ok = warp_wait(&hd.raw_full[st], ph, p.wait_ns, kHintNs);
        if (!ok) break;
        uint32_t kp = 0, vp = 0;  // of a key past the end, or before all rows' windows: zeros
        if (const int at = (g.tile0 + t) * kTile + key; at >= g.first && at < g.L) {
          kp = lds32(blk + 16 * D + 4 * r);
          vp = lds32(blk + 16 * D + 64 + 4 * r);
        }
        ok = k < 2 || warp_wait(&hd.k_empty[st], ph ^ 1u, p.wait_ns, kHintNs);
        if (!ok) break;
        auto put_k = [&](float ks, float ko) {
          const uint32_t ks2 = pack_f16x2(ks, ks), ko2 = pack_f16x2(ko, ko);
          dequant_row<D>(blk + r * (D / 2), k_at + st * kTileBytes, key, half,
                         [&](uint32_t w) { return dequant8_f16(w, ks2, ko2); });
        };
        put_k(__uint_as_float(kp << 16), __uint_as_float(kp & 0xFFFF0000u));
        uint32_t odd = 0;
        if (__any_sync(0xffffffffu, !fits_f16(kp) || !fits_f16(vp))) {  // either end, or parameters out of f16's range
          if (!finite_par(vp)) vp = 0, kp = 0x7FC07FC0u;
          if (!finite_par(kp)) kp = 0x7FC07FC0u;
          const bool k_odd = kp != 0 && kp != 0x7FC07FC0u && !fits_f16(kp);
          odd = __any_sync(0xffffffffu, vp != 0 && !fits_f16(vp)) ? 2u : 0u;
          float ks = __uint_as_float(kp << 16), ko = __uint_as_float(kp & 0xFFFF0000u);
          int e = 0;
          if (k_odd) {  // the row's largest element goes to 1 .. 2
            const float top = fmaxf(fabsf(ko), fabsf(fmaf(15.f, ks, ko)));
            e = max((int)(__float_as_uint(top) >> 23), 1) - 127;
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
            ks *= f, ko *= f;
          }
          odd |= __any_sync(0xffffffffu, k_odd) ? 1u : 0u;
          if (half == 0 && (odd & 1u)) hd.exponent[k & 3][key] = (int8_t)e;
          put_k(ks, ko);
        }
        if (half == 0 && lane == 0) hd.flags[k & 3][key / 32] = (uint8_t)odd;
        const bool wide_v = odd & 2u;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&hd.k_full[st]);
        ok = k < 2 || warp_wait(&hd.v_empty[st], ph ^ 1u, p.wait_ns, kHintNs);
        if (!ok) break;
        const uint32_t v_src = blk + 8 * D + r * (D / 2), v_dst = v_at + st * kTileBytes;
        const float vs = __uint_as_float(vp << 16), vo = __uint_as_float(vp & 0xFFFF0000u);
        if (!wide_v) {
          const uint32_t vs2 = pack_f16x2(vs, vs), vo2 = pack_f16x2(vo, vo);
          dequant_row<D>(v_src, v_dst, key, half, [&](uint32_t w) { return dequant8_f16(w, vs2, vo2); });
        } else {
          const uint32_t s_lo = pack_bf16x2(vs * 128.f, vs * 128.f), s_hi = pack_bf16x2(vs * 8.f, vs * 8.f);
          const uint32_t vo2 = pack_bf16x2(vo, vo);
          dequant_row<D>(v_src, v_dst, key, half, [&](uint32_t w) { return dequant8_bf16(w, s_lo, s_hi, vo2); });
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&hd.v_full[st]);
          mbar_arrive(&hd.raw_empty[st]);
        }
      }
    }
    if (!ok && lane == 0) fail(p);
  } else {
    // ---------------------------------------------------------------- softmax, one row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int i = warp / 4, quarter = warp & 3;
    const int row = 32 * quarter + lane;  // of the half
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_t = tmem + lanes + 128 * i, o_t = tmem + lanes + 256 + 128 * i;
    const float scale = fabsf(p.a.scale_log2);
    const float sign = p.a.scale_log2 < 0.f ? -1.f : 1.f;
    float sl = 0.f, sl_next = 0.f;  // scale over the row's factor in the Q tile, not 0 (x infinity of a masked score)
    unsigned n_s = 0, n_o = 0, tiles = 0;  // tiles: of the CTA, as the dequantisers count them
    bool ok = true;

    // This warp's 32 rows of an item into the Q tile: D / 8 lanes a row, 16 bytes each, the loads of 16 rows in flight
    // (all 32 at once are twice the code, which comes from memory at a call's start: the mixed step took 128 us against
    // 124; a quarter at a time waits too often, 415 us for the prompt of 8192 tokens against 393). A row is
    // scaled by a power of two that brings its largest element to 2^7 .. 2^8, so that f16 holds its bf16 values.
    auto load_q = [&](const Segment& x) {
      constexpr int C = D / 8, RPI = 32 / C, N = C / 2;  // 32 / RPI loads a lane, N at a time
#pragma unroll 1
      for (int j0 = 0; j0 < C; j0 += N) {
        uint4 w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int in_item = 128 * i + 32 * quarter + (j0 + j) * RPI + lane / C;
          w[j] = make_uint4(0, 0, 0, 0);
          if (in_item < x.rows) {
            const unsigned R = x.r0 + in_item, tok = div_group(p, R);
            w[j] = *reinterpret_cast<const uint4*>(p.a.q + (int64_t)(x.row + tok) * p.a.ld_q +
                                                   (int64_t)(x.h * p.v.group + R - tok * p.v.group) * D + (lane % C) * 8);
          }
        }
        uint32_t top[N / 2];  // the rows' largest magnitudes as bf16, of loads j and j + N / 2
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          auto largest = [](const uint4& x) {
            constexpr uint32_t kAbs = 0x7FFF7FFFu;
            const uint32_t t = __vmaxu2(__vmaxu2(x.x & kAbs, x.y & kAbs), __vmaxu2(x.z & kAbs, x.w & kAbs));
            return max(t & 0xFFFFu, t >> 16);
          };
          top[j] = largest(w[j]) | (largest(w[j + N / 2]) << 16);
#pragma unroll
          for (int o = 1; o < C; o <<= 1) top[j] = __vmaxu2(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t eb = (j < N / 2 ? top[j % (N / 2)] & 0xFFFFu : top[j % (N / 2)] >> 16) >> 7;  // exponent
          const uint32_t es = eb == 255u ? 127u : min(261u - eb, 254u);
          // not finite: all of the row is NaN, as its result is (minus infinity alone would look like a mask's)
          const float f = eb == 255u ? NAN : sign * __uint_as_float(es << 23);
          const uint32_t mine = __shfl_sync(0xffffffffu, es, lane % RPI * C);
          if (lane / RPI == j0 + j) sl_next = fmaxf(scale * __uint_as_float((254u - mine) << 23), 1e-37f);
          const int rr = 32 * quarter + (j0 + j) * RPI + lane / C, ch = lane % C;
          auto pair = [&](uint32_t a, uint32_t b, bool up) {
            return up ? pack_f16x2(f * __uint_as_float(a & 0xFFFF0000u), f * __uint_as_float(b & 0xFFFF0000u))
                      : pack_f16x2(f * __uint_as_float(a << 16), f * __uint_as_float(b << 16));
          };
          const uint4 o = make_uint4(pair(w[j].x, w[j].z, false), pair(w[j].x, w[j].z, true), pair(w[j].y, w[j].w, false),
                                     pair(w[j].y, w[j].w, true));
          sts128(q_at + i * kTileBytes + (ch / 8) * (128 * 128) + rr * 128 + (((ch % 8) ^ (rr & 7)) * 16), o);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd.q_full[i]);
    };

    // One copy of the code that loads rows, met before every segment: the first time with nothing to compute. (The three
    // roles' loops share the instruction cache: three copies cost the prompt of 8192 tokens 5 us, the mixed step 4.)
    Segment g = {};
    bool mine = false;  // a short item has no second half
    for (unsigned n = 0;;) {
      const int in_item = min(128 * i + row, g.rows - 1);
      const unsigned R = g.r0 + in_item, tok = div_group(p, R);
      const int hi = g.pos0 + (int)tok;  // last key that this row sees
      // keys that every row of the half sees
      const int all_hi = g.pos0 + (int)div_group(p, g.r0 + 128 * i);
      const int all_lo = p.a.window > 0 ? g.pos0 + (int)div_group(p, g.r0 + min(128 * i + 127, g.rows - 1)) - p.a.window + 1 : 0;
      float m = -INFINITY, l = 0.f;
      sl = sl_next;
      if (!mine) tiles += g.len;
      for (int k = 0; mine && k < g.len; ++k) {
        const int key0 = (g.tile0 + k) * kTile;
        ok = warp_wait(&hd.s_full[i], n_s & 1u, p.wait_ns, kHintNs);
        if (!ok) break;
        ++n_s;
        tc_fence_after_sync();
        const uint32_t flags = *reinterpret_cast<const volatile uint32_t*>(hd.flags[tiles & 3]);
        const int8_t* exps = hd.exponent[tiles & 3];
        ++tiles;
        const bool masked = key0 + kTile - 1 > all_hi || key0 < all_lo;
        const int d = hi - key0, e = p.a.window > 0 ? d - p.a.window : -1;  // visible: e < column <= d
        auto mask = [&](int j, uint32_t (&x32)[32]) {
          const int a = d - 32 * j, b = e - 32 * j;
          const uint32_t see = (a >= 31 ? 0xffffffffu : a < 0 ? 0u : (2u << a) - 1u) &
                               ~(b >= 31 ? 0xffffffffu : b < 0 ? 0u : (2u << b) - 1u);
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (!(see & (1u << x))) x32[x] = 0xFF800000u;
        };
        auto below = [&](float mx) { return mx - __fdividef(kFresh, sl); };
        auto rescale = [&](float mx) {  // m becomes mx, what has been summed is scaled to it
          const float f = m == -INFINITY ? 0.f : ex2((m - mx) * sl);
          l *= f;
          m = mx;
#pragma unroll 1
          for (int j = 0; j < D; j += 16) {
            uint32_t o[16];
            tmem_ld_x16(o_t + j, o);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st_x16(o_t + j, o);
          }
        };
        auto hand_over = [&](int y) {
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&hd.p_full[y][i]);
        };
        bool done = false;
        if (flags == 0) {
          uint32_t v[4][32];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld_x32(s_t + 32 * j, v[j]);
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int j = 0; j < 4; ++j) mask(j, v[j]);
          }
          if (k == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int x = 0; x < 32; x += 2)
                m = fmaxf(m, fmaxf(__uint_as_float(v[j][x]), __uint_as_float(v[j][x + 1])));
            m = below(m);
          }
          uint32_t w[32];
          // weights of 64 keys by the present m, and their sum
          auto weights = [&](int y) {
            const float ms = -m * sl;
            const uint64_t sl2 = pack_f32x2(sl, sl), ms2 = pack_f32x2(ms, ms);
            uint64_t sum2[2];
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
              const uint32_t* q = &v[2 * y + x / 32][x % 32];
              float pa, pb;
              unpack_f32x2(fma_f32x2(pack_b32x2(q[0], q[1]), sl2, ms2), pa, pb);
              pa = ex2(pa);
              pb = ex2(pb);
              sum2[(x >> 1) & 1] = x < 4 ? pack_f32x2(pa, pb) : add_f32x2(sum2[(x >> 1) & 1], pack_f32x2(pa, pb));
              w[x / 2] = pack_f16x2(pa, pb);
            }
            float sa, sb;
            unpack_f32x2(add_f32x2(sum2[0], sum2[1]), sa, sb);
            return sa + sb;
          };
          // The weights' size shows whether m will do: no maximum is taken as long as their sum stays below kBig (and
          // m scale is small enough for the one rounding of weights())
          float sum = weights(0);
          if (!__any_sync(0xffffffffu, !(fabsf(m * sl) < 16777216.f) || sum > kBig)) {
            tmem_st_x32(s_t, w);
            hand_over(0);
            l += sum;
            sum = weights(1);
            if (__any_sync(0xffffffffu, sum > kBig)) {
              ok = warp_wait(&hd.pa_done[i], (n_s & 1u) ^ 1u, p.wait_ns, kHintNs);  // the product with the first weights
              if (!ok) break;
              tc_fence_after_sync();
              float mx = -INFINITY;
#pragma unroll
              for (int j = 2; j < 4; ++j) {
                tmem_ld_x32(s_t + 32 * j, v[j]);
                tmem_ld_wait();
                if (masked) mask(j, v[j]);
#pragma unroll
                for (int x = 0; x < 32; ++x) mx = fmaxf(mx, __uint_as_float(v[j][x]));
              }
              rescale(fmaxf(m, below(mx)));
              sum = 0.f;
#pragma unroll
              for (int x = 0; x < 64; x += 2) {
                const float pa = ex2((__uint_as_float(v[2 + x / 32][x % 32]) - m) * sl);
                const float pb = ex2((__uint_as_float(v[2 + x / 32][x % 32 + 1]) - m) * sl);
                sum += pa + pb;
                w[x / 2] = pack_f16x2(pa, pb);
              }
            }
            tmem_st_x32(s_t + 32, w);
            hand_over(1);
            l += sum;
            done = true;
          }
        }
        if (!done) {
          // A new maximum, rows that have seen nothing, keys or values out of f16's range: 32 keys at a time, twice. (The product
          // before has finished, s_full covers it; the next waits for this thread.)
          float mx = -INFINITY;
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint32_t x32[32];
            tmem_ld_x32(s_t + 32 * j, x32);
            tmem_ld_wait();
            if (flags >> (8 * j) & 1u) {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                x32[x] = __float_as_uint(__uint_as_float(x32[x]) * __uint_as_float((uint32_t)(exps[32 * j + x] + 127) << 23));
            }
            if (masked) mask(j, x32);
#pragma unroll
            for (int x = 0; x < 32; ++x) mx = fmaxf(mx, __uint_as_float(x32[x]));
            if (flags || masked) tmem_st_x32(s_t + 32 * j, x32);
          }
          tmem_st_wait();
          if (k > 0)
            rescale(fmaxf(m, below(mx)));
          else
            m = below(mx);
          const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            uint32_t x32[32], w[16];
            tmem_ld_x32(s_t + 32 * j, x32);
            tmem_ld_wait();
            const bool wide = flags >> (8 * j) & 2u;
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float pa = ex2((__uint_as_float(x32[x]) - mu) * sl);
              const float pb = ex2((__uint_as_float(x32[x + 1]) - mu) * sl);
              l += pa + pb;
              w[x / 2] = wide ? pack_bf16x2(pa, pb) : pack_f16x2(pa, pb);
            }
            tmem_st_x16(s_t + 16 * j, w);
            if (j & 1) hand_over(j >> 1);
          }
        }
      }
      if (!ok) break;
      // the half's scores are done with its Q tile: the next item's rows go in while the last product runs
      Segment nx;
      const bool more = read_segment(n++, nx), next = more && nx.rows > 128 * i;
      if (next) load_q(nx);
      if (mine) {
        // ---- the segment's result
        ok = warp_wait(&hd.o_full[i], n_o & 1u, p.wait_ns, kHintNs);
        if (!ok) break;
        ++n_o;
        tc_fence_after_sync();
        const bool real = 128 * i + row < g.rows;
        if (g.whole) {
          __nv_bfloat16* dst = p.a.out + (int64_t)(g.row + tok) * p.a.ld_out +
                               (int64_t)(g.h * p.v.group + R - tok * p.v.group) * D;
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
          for (int j = 0; j < D; j += 32) {
            uint32_t o[32];
            tmem_ld_x32(o_t + j, o);
            tmem_ld_wait();
            if (real) {
#pragma unroll
              for (int x = 0; x < 32; x += 8) {
                float f[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) f[y] = l == 0.f ? 0.f : __uint_as_float(o[x + y]) * inv;
                *reinterpret_cast<uint4*>(dst + j + x) = unpermute8(f);
              }
            }
          }
        } else {
          float* slot = p.part + (int64_t)(g.slot * 2 + i) * kPart + row;
#pragma unroll 1
          for (int j = 0; j < D; j += 32) {
            uint32_t o[32];
            tmem_ld_x32(o_t + j, o);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) __stcg(slot + (j + x) * 128, __uint_as_float(o[x]));
          }
          __stcg(slot + D * 128, m * sl);  // in units of log2: the row's factor is gone
          __stcg(slot + (D + 1) * 128, l);
        }
        tc_fence_before_sync();
      }
      if (!more) break;
      g = nx;
      mine = next;
    }
    if (!ok && lane == 0) fail(p);
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 16) tmem_dealloc(tmem, 512);
}

// Joins the partial results of an item that several CTAs share, in their
// order: block (CTA that starts the item, 32 rows), a row a lane, 8 columns a
// warp, four shares' loads in flight. Bound by the partial results' bytes,
// which come from L2.
template <int D>
__global__ void __launch_bounds__(4 * D) join_kernel(const __grid_constant__ PrefillParams p) {
  constexpr int kPart = (D + 2) * 128;
  constexpr int N = 8, U = 4;
  kv_follow();
  const int64_t first = blockIdx.x;
  const Join j = p.joins[first];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int in_item = blockIdx.y * kJoinRows + lane, half = in_item / 128;
  if (blockIdx.y * kJoinRows >= (j.parts ? j.rows : 0)) return;
  float M = -INFINITY, L = 0.f, o[N];
#pragma unroll
  for (int y = 0; y < N; ++y) o[y] = 0.f;
  for (int x0 = 0; x0 < j.parts; x0 += U) {
    float m[U], l[U], v[U][N];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int xx = x0 + x;
      m[x] = -INFINITY, l[x] = 0.f;
      if (xx < j.parts) {
        const float* q = p.part + (((first + xx) * 2 + (xx == 0)) * 2 + half) * kPart + in_item % 128;
        m[x] = __ldcg(q + D * 128);
        l[x] = __ldcg(q + (D + 1) * 128);
#pragma unroll
        for (int y = 0; y < N; ++y) v[x][y] = __ldcg(q + (warp * N + y) * 128);
      } else {
#pragma unroll
        for (int y = 0; y < N; ++y) v[x][y] = 0.f;
      }
    }
    const float top = fmaxf(fmaxf(M, fmaxf(m[0], m[1])), fmaxf(m[2], m[3]));
    const float f0 = M == -INFINITY ? 1.f : ex2(M - top);  // nothing, or a NaN, so far: as it is
    M = top;
    L *= f0;
#pragma unroll
    for (int y = 0; y < N; ++y) o[y] *= f0;
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const float f = m[x] == -INFINITY ? (l[x] == 0.f ? 0.f : 1.f) : ex2(m[x] - M);
      L = fmaf(f, l[x], L);
#pragma unroll
      for (int y = 0; y < N; ++y) o[y] = l[x] == 0.f ? o[y] : fmaf(f, v[x][y], o[y]);
    }
  }
  if (in_item >= j.rows) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const unsigned R = j.r0 + in_item, tok = div_group(p, R);
  __nv_bfloat16* dst = p.a.out + (int64_t)(j.row + tok) * p.a.ld_out +
                       (int64_t)(j.h * p.v.group + R - tok * p.v.group) * D + warp * N;
#pragma unroll
  for (int y = 0; y < N; ++y) o[y] *= inv;
  *reinterpret_cast<uint4*>(dst) = unpermute8(o);
}

template <int D>
spear_status_t launch(const spear_kv_s* h, PrefillParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  if (smem_limit_once(reinterpret_cast<const void*>(prefill_kernel<D>), done) != cudaSuccess) return SPEAR_ERR_CUDA;
  // at least half of an SM's shared memory, so that one CTA has its tensor memory for itself
  const size_t used = kHeader + 6 * (size_t)kTile * D * 2 + 2 * (size_t)kBlocksPerTile * 16 * (D + 8);
  const size_t smem = used > 116 * 1024 ? used : 116 * 1024;
  const spear_status_t st = kv_launch(prefill_kernel<D>, dim3(h->sm_count), kThreads, smem, stream, p);
  if (st != SPEAR_OK) return st;
  return kv_launch(join_kernel<D>, dim3(h->sm_count, kRows / kJoinRows), 4 * D, 0, stream, p);
}

}  // namespace
}  // namespace spear

using namespace spear;

static size_t part_bytes(const spear_kv_s* h) { return (size_t)h->sm_count * 4 * (h->view.D + 2) * 128 * sizeof(float); }

size_t kv_prefill_workspace(const spear_kv_s* h) { return part_bytes(h) + (size_t)h->sm_count * sizeof(Join); }

spear_status_t kv_launch_prefill(const spear_kv_s* h, const KvAttnArgs& a, int max_rows, void* ws, cudaStream_t stream) {
  PrefillParams p;
  p.v = h->view;
  p.a = a;
  p.max_rows = max_rows;
  p.inv_group = h->view.group > 1 ? (unsigned)((1ull << 32) / h->view.group) + 1u : 0u;
  p.part = static_cast<float*>(ws);
  p.joins = reinterpret_cast<Join*>(static_cast<char*>(ws) + part_bytes(h));
  // Most waits are for a tile, some for segments: the schedule's for the softmax to take the next one, and an idle half's
  // first for scores, while the other half works on as many as are in flight. A segment can be all the key tiles of an
  // item, 1.4 us each: twice that, so often, beside 100 ms. (100 ms alone ended a correct call beyond 9 million keys.)
  const int64_t keys = std::min((int64_t)a.ld_pt * h->view.page_size, (int64_t)kKvMaxTokens);
  p.wait_ns = 100000000ull + (uint64_t)(keys / kTile + 1) * (2 * 1400 * (kSegs + 1));
  return h->view.D == 128 ? launch<128>(h, p, stream) : launch<64>(h, p, stream);
}

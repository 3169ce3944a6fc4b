// Attention of many query rows over the paged 4-bit cache (prefill chunks) on
// the tcgen05 tensor cores.
//
// For each (sequence, key/value head) the rows are the query tokens times the
// heads that share it, in tiles of 256 (two MMA tiles of 128); a row meets its
// visible keys in tiles of 128:
//   S = Q K^T (fp32, tensor memory), P = 2^(scale (S - m)) (bf16, written over
//   S), O += P V (fp32, tensor memory), l += sum P;  out = O / l.
// Bound by the tensor cores, 4 D flops a (row, key) pair, with the smaller
// units close behind: per 256 x 128 block of D = 128 the MMAs take 2048 cycles
// of an SM, their operands in shared memory 1536 at 128 bytes a cycle, the
// dequantised tiles' stores 512.
//
//  - Dequantisers (4 warps, one key a thread) turn a tile's packed rows into
//    bf16 code * scale + offset, rounded once, in 128-byte-swizzled shared
//    memory. Both tiles are stored key by key: K is the K-major B operand of
//    S, V the MN-major B operand of O, so nothing is transposed. A code word's
//    pairs come out as elements (0, 4), (1, 5), (2, 6), (3, 7); Q's rows are
//    permuted alike, and O's columns are put back in the epilogue. Keys past
//    the sequence's end become zeros, and a key whose V is not finite is moved
//    to its K (V zero, K NaN): rows that see it get NaN, the mask keeps it from
//    the others (0 x NaN in O += P V would not).
//  - Two softmax warpgroups, one an MMA tile, one row a thread; P goes from
//    registers to tensor memory. While one works on S the other's products run.
//    The running maximum is lazy as in the other kernel: O is rescaled only
//    when a score passes m by 8 in log2.
//  - One thread issues the MMAs, in the order O0 S0 O1 S1 of successive tiles:
//    an S overwrites its P only after the product that reads it, which was
//    issued before it.
//  - One warp copies the packed tiles, a bulk copy a 16-token block.
//
// Work: (sequence, head, row tile, key tile) units in this order are split
// evenly over the CTAs (one an SM); items that several CTAs share are joined
// by the last of them to arrive, in CTA order, one 128-row half at a time.
#include <atomic>

#include "kv_device.cuh"
#include "tcgen05.cuh"

namespace spear {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 128;            // keys of a unit
constexpr int kRows = 256;            // rows of an item
constexpr int kBlocksPerTile = kTile / 16;
constexpr int kHeader = 1024;         // barriers and the start position
constexpr float kLazy = 8.f;
constexpr uint32_t kHintNs = 100;

struct PrefillParams {
  KvView v;
  KvAttnArgs a;
  int max_rows;        // sequences with at most this many rows of a key/value head belong to the other kernel
  float* part;         // [grid][2][2 halves][D + 2][128]
  unsigned* counters;  // [grid][2 halves]
  uint64_t wait_ns;
};

struct Header {
  uint64_t raw_full[2], raw_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], done;
  uint32_t tmem;
  int start_b, start_h, start_qt, start_tile;
  int last[2];
  int64_t units;
};
static_assert(sizeof(Header) <= kHeader, "");

// Row tile qt of a sequence: its key tiles.
struct Item {
  int lo, tiles;
  int rows;  // rows of this tile, <= 256
};

SPEAR_DEVINL int row_tiles(const PrefillParams& p, const KvSeq& s) {
  const int64_t rows = (int64_t)s.n * p.v.group;
  return rows > p.max_rows ? (int)((rows + kRows - 1) / kRows) : 0;
}

SPEAR_DEVINL Item item_of(const PrefillParams& p, const KvSeq& s, int qt) {
  Item it;
  const int64_t rows = (int64_t)s.n * p.v.group, r0 = (int64_t)qt * kRows;
  it.rows = (int)min((int64_t)kRows, rows - r0);
  const int t0 = (int)(r0 / p.v.group), t1 = (int)((r0 + it.rows - 1) / p.v.group);
  const int last = s.L - s.n + t1;
  const int64_t first = p.a.window > 0 ? (int64_t)s.L - s.n + t0 - p.a.window + 1 : 0;
  it.lo = first > 0 ? (int)(first / kTile) : 0;
  it.tiles = max(1, (last >= 0 ? last / kTile + 1 : 0) - it.lo);
  return it;
}

struct Cursor {
  int b, h, qt, nqt, tile;
  KvSeq s;
  Item it;
};

SPEAR_DEVINL void next_item(const PrefillParams& p, Cursor& c) {
  c.tile = 0;
  if (++c.qt == c.nqt) {
    c.qt = 0;
    if (++c.h == p.v.n_kv_heads) {
      c.h = 0;
      do {
        ++c.b;
        c.s = kv_seq(p.v, p.a, c.b, kTile);
        c.nqt = row_tiles(p, c.s);
      } while (c.nqt == 0);
    }
  }
  c.it = item_of(p, c.s, c.qt);
}

// Units of one head of a sequence, the whole warp at it.
SPEAR_DEVINL int64_t head_units(const PrefillParams& p, const KvSeq& s, int nqt, int lane) {
  int64_t x = 0;
  for (int qt = lane; qt < nqt; qt += 32) x += item_of(p, s, qt).tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Calls f(sequence, row tiles) for every sequence of this kernel, the warp
// together, until f returns true.
template <class F>
SPEAR_DEVINL void each_sequence(const PrefillParams& p, int lane, F f) {
  for (int b0 = 0; b0 < p.a.n_seqs; b0 += 32) {
    const int b = b0 + lane;
    const bool mine = b < p.a.n_seqs && row_tiles(p, kv_seq(p.v, p.a, b, kTile)) > 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, mine); todo; todo &= todo - 1) {
      const int bb = b0 + __ffs(todo) - 1;
      const KvSeq s = kv_seq(p.v, p.a, bb, kTile);
      if (f(bb, s, row_tiles(p, s))) return;
    }
  }
}

SPEAR_DEVINL void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// Eight codes of a word as four bf16 pairs, elements (0, 4), (1, 5), (2, 6), (3, 7).
SPEAR_DEVINL uint4 dequant8(uint32_t w, uint32_t ss, uint32_t oo) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = bf16x2_fma(bf16x2_sub(int4_pair_to_bf16x2_biased(w >> (4 * i)), 0x43004300u), ss, oo);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

SPEAR_DEVINL void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// One key's row: codes (D / 2 bytes at `src`) to row `key` of a swizzled tile.
template <int D>
SPEAR_DEVINL void dequant_row(uint32_t src, uint32_t tile, int key, uint32_t par) {
  const uint32_t ss = __byte_perm(par, par, 0x1010), oo = __byte_perm(par, par, 0x3232);
  constexpr int Q = D / 32;  // 16-byte quarters of the packed row
  uint4 w[Q];
  int q[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    // quarters in an order of the key's own: a quarter warp then meets every bank once
    q[i] = Q == 4 ? (i + (key >> 1)) & 3 : i;
    w[i] = lds128(src + q[i] * 16);
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    const uint32_t row = tile + (q[i] >> 1) * (kTile * 128) + key * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sts128(row + ((((q[i] & 1) * 4 + j) ^ (key & 7)) * 16), dequant8(words[j], ss, oo));
  }
}

SPEAR_DEVINL bool finite_par(uint32_t par) {
  return (par & 0x7F80u) != 0x7F80u && (par & 0x7F800000u) != 0x7F800000u;
}

SPEAR_DEVINL void fail(const PrefillParams& p) { atomicOr(p.v.status, kStatusTimeoutPipe); }

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
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;

  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&hd.raw_full[i], 1);
      mbar_init(&hd.raw_empty[i], 4);
      mbar_init(&hd.k_full[i], 4);
      mbar_init(&hd.k_empty[i], 1);
      mbar_init(&hd.v_full[i], 4);
      mbar_init(&hd.v_empty[i], 1);
      mbar_init(&hd.q_full[i], 4);
      mbar_init(&hd.s_full[i], 1);
      mbar_init(&hd.p_full[i], 4);
      mbar_init(&hd.o_full[i], 1);
    }
    mbar_init(&hd.done, 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(&hd.tmem, 512);
    tmem_relinquish();
  }
  // ---- this CTA's units [u0, u1) and the position of u0
  if (warp == 0) {
    int64_t U = 0;
    each_sequence(p, lane, [&](int, const KvSeq& s, int nqt) {
      U += head_units(p, s, nqt, lane) * p.v.n_kv_heads;
      return false;
    });
    const int64_t G = min((int64_t)gridDim.x, U), u0 = blockIdx.x * U / max(G, (int64_t)1);
    int64_t before = 0;
    if ((int64_t)blockIdx.x < G)
      each_sequence(p, lane, [&](int b, const KvSeq& s, int nqt) {
        const int64_t hu = head_units(p, s, nqt, lane);
        if (u0 >= before + hu * p.v.n_kv_heads) {
          before += hu * p.v.n_kv_heads;
          return false;
        }
        const int h = (int)((u0 - before) / hu);
        int64_t rest = u0 - before - h * hu;
        for (int q0 = 0; q0 < nqt; q0 += 32) {
          const int qt = q0 + lane;
          const int own = qt < nqt ? item_of(p, s, qt).tiles : 0;
          int incl = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
          }
          if (own > 0 && rest >= incl - own && rest < incl) {
            hd.start_b = b;
            hd.start_h = h;
            hd.start_qt = qt;
            hd.start_tile = (int)(rest - (incl - own));
          }
          const int sum = __shfl_sync(0xffffffffu, incl, 31);
          if (rest < sum) break;
          rest -= sum;
        }
        return true;
      });
    if (lane == 0) hd.units = U;
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const int64_t U = hd.units, G = min((int64_t)gridDim.x, U), cta = blockIdx.x;
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&hd.tmem);
  const int64_t u0 = cta < G ? cta * U / G : 0, u1 = cta < G ? (cta + 1) * U / G : 0;
  Cursor c{};
  if (u0 < u1) {
    c.b = hd.start_b;
    c.h = hd.start_h;
    c.qt = hd.start_qt;
    c.tile = hd.start_tile;
    c.s = kv_seq(p.v, p.a, c.b, kTile);
    c.nqt = row_tiles(p, c.s);
    c.it = item_of(p, c.s, c.qt);
  }

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 13) {
      // -------------------------------------------------------------- copies of the packed tiles
      int st = 0;
      unsigned ph = 0;
      int64_t issued = 0;
      for (int64_t u = u0; u < u1; ++u) {
        const int blk = (c.it.lo + c.tile) * kBlocksPerTile + lane;
        const uint8_t* src = nullptr;
        if (lane < kBlocksPerTile && blk < (c.s.L + 15) / 16) {
          const int pg = p.a.page_table[(int64_t)c.b * p.a.ld_pt + blk / p.v.bpp];
          if (pg >= 0 && pg < p.v.n_pages)
            src = p.v.pool + (((int64_t)pg * p.v.n_kv_heads + c.h) * p.v.bpp + blk % p.v.bpp) * BB;
          else
            atomicOr(p.v.status, kStatusBadIndex);
        }
        const unsigned copies = __popc(__ballot_sync(0xffffffffu, src != nullptr));
        if (issued >= 2 && !warp_wait(&hd.raw_empty[st], ph ^ 1u, p.wait_ns, kHintNs)) {
          if (lane == 0) fail(p);
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&hd.raw_full[st], copies * BB);
        __syncwarp();
        if (src) bulk_g2s_shared_u32(raw_at + st * kRawBytes + lane * BB, src, BB, &hd.raw_full[st]);
        ++issued;
        if (++st == 2) st = 0, ph ^= 1u;
        if (++c.tile == c.it.tiles && u + 1 < u1) next_item(p, c);
      }
      for (int i = 0; i < (int)min(issued, (int64_t)2); ++i) {  // copies in flight land before the CTA ends
        if (st == 0) st = 2, ph ^= 1u;
        --st;
        warp_wait(&hd.raw_full[st], ph, p.wait_ns, kHintNs);
      }
    } else if (warp == 12 && lane == 0) {
      // -------------------------------------------------------------- MMA issue
      const uint32_t idesc_s = idesc_bf16_f32(128, kTile);
      const uint32_t idesc_o = idesc_bf16_f32(128, D) | kIdescBMnMajor;
      unsigned n_q[2] = {0, 0}, n_p[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, unsigned parity) {
        if (ok && !mbar_wait_bounded_hint(bar, parity, p.wait_ns, kHintNs)) {
          ok = false;
          fail(p);
        }
        return ok;
      };
      auto scores = [&](int i, int64_t k, bool first) {  // S_i = Q_i K^T of the CTA's k-th tile
        const int st = (int)(k & 1);
        if (!wait(&hd.k_full[st], (unsigned)(k >> 1) & 1u)) return;
        if (first && !wait(&hd.q_full[i], n_q[i]++ & 1u)) return;
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk / 4) * (128 * 128) + (kk % 4) * 32;
          umma_bf16(tmem + 128 * i, sw128_kmajor_desc(q_at + i * kTileBytes + at),
                    sw128_kmajor_desc(k_at + st * kTileBytes + at), idesc_s, kk != 0);
        }
        umma_commit(&hd.s_full[i]);
      };
      int64_t k = 0;
      int halves = c.it.rows > 128 ? 2 : 1;
      for (int i = 0; i < halves && u0 < u1; ++i) scores(i, 0, true);
      if (u0 < u1 && ok) umma_commit(&hd.k_empty[0]);
      for (int64_t u = u0; u < u1 && ok; ++u, ++k) {
        const bool first = u == u0 || c.tile == 0;
        const bool last = c.tile + 1 == c.it.tiles || u + 1 == u1;
        const int st = (int)(k & 1);
        int next_halves = halves;
        bool next_first = false;
        if (u + 1 < u1 && ++c.tile == c.it.tiles) {
          next_item(p, c);
          next_halves = c.it.rows > 128 ? 2 : 1;
          next_first = true;
        }
        for (int i = 0; i < 2 && ok; ++i) {
          if (i < halves) {
            if (!wait(&hd.p_full[i], n_p[i]++ & 1u)) break;
            if (i == 0 && !wait(&hd.v_full[st], (unsigned)(k >> 1) & 1u)) break;
            tc_fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_ts_bf16(tmem + 256 + 128 * i, tmem + 128 * i + 8 * kk,
                           sw128_mnmajor_desc(v_at + st * kTileBytes + kk * 2048, kTile * 128), idesc_o,
                           !(first && kk == 0));
            if (last) umma_commit(&hd.o_full[i]);
            if (i == halves - 1) umma_commit(&hd.v_empty[st]);
          }
          if (u + 1 < u1 && i < next_halves) {
            scores(i, k + 1, next_first);
            if (ok && i == next_halves - 1) umma_commit(&hd.k_empty[st ^ 1]);
          }
        }
        halves = next_halves;
      }
      // nothing of this CTA's is still running on the tensor cores when the others go on to the end
      umma_commit(&hd.done);
      if (!mbar_wait_bounded(&hd.done, 0, p.wait_ns)) fail(p);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- dequantisers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int key = tid - 256;
    const uint32_t blk_at = raw_at + (key / 16) * BB;
    const int r = key & 15;
    bool ok = true;
    int64_t k = 0;
    for (int64_t u = u0; u < u1; ++u, ++k) {
      const int st = (int)(k & 1);
      const unsigned ph = (unsigned)(k >> 1) & 1u;
      const uint32_t blk = blk_at + st * kRawBytes;
      ok = ok && warp_wait(&hd.raw_full[st], ph, p.wait_ns, kHintNs);
      const bool live = (c.it.lo + c.tile) * kTile + key < c.s.L;
      uint32_t kp = 0, vp = 0;
      if (live) {
        kp = lds32(blk + 16 * D + 4 * r);
        vp = lds32(blk + 16 * D + 64 + 4 * r);
        if (!finite_par(vp)) vp = 0, kp = 0x7FC07FC0u;
      }
      ok = ok && (k < 2 || warp_wait(&hd.k_empty[st], ph ^ 1u, p.wait_ns, kHintNs));
      if (ok) dequant_row<D>(blk + r * (D / 2), k_at + st * kTileBytes, key, kp);
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&hd.k_full[st]);
      ok = ok && (k < 2 || warp_wait(&hd.v_empty[st], ph ^ 1u, p.wait_ns, kHintNs));
      if (ok) dequant_row<D>(blk + 8 * D + r * (D / 2), v_at + st * kTileBytes, key, vp);
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) {
        mbar_arrive(&hd.v_full[st]);
        mbar_arrive(&hd.raw_empty[st]);
      }
      if (++c.tile == c.it.tiles && u + 1 < u1) next_item(p, c);
    }
    if (!ok && lane == 0) fail(p);
  } else {
    // ---------------------------------------------------------------- softmax, one row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int i = warp / 4, quarter = warp & 3;
    const int row = 32 * quarter + lane;  // of the half
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t s_t = tmem + lanes + 128 * i, o_t = tmem + lanes + 256 + 128 * i;
    const float sl = fabsf(p.a.scale_log2);
    const uint32_t flip = p.a.scale_log2 < 0.f ? 0x80008000u : 0u;
    unsigned n_s = 0, n_o = 0;
    bool ok = true;

    // this warp's 32 rows of an item into the Q tile: D / 8 lanes a row, 16 bytes each
    auto load_q = [&](const Cursor& x) {
      constexpr int C = D / 8, RPI = 32 / C;
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += RPI) {
        const int rr = 32 * quarter + r0 + lane / C, ch = lane % C;
        const int in_item = 128 * i + rr;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (in_item < x.it.rows) {
          const int64_t R = (int64_t)x.qt * kRows + in_item;
          w = *reinterpret_cast<const uint4*>(p.a.q + (x.s.row + R / p.v.group) * p.a.ld_q +
                                              (int64_t)(x.h * p.v.group + (int)(R % p.v.group)) * D + ch * 8);
        }
        uint4 o;
        o.x = __byte_perm(w.x, w.z, 0x5410) ^ flip;
        o.y = __byte_perm(w.x, w.z, 0x7632) ^ flip;
        o.z = __byte_perm(w.y, w.w, 0x5410) ^ flip;
        o.w = __byte_perm(w.y, w.w, 0x7632) ^ flip;
        sts128(q_at + i * kTileBytes + (ch / 8) * (128 * 128) + rr * 128 + (((ch % 8) ^ (rr & 7)) * 16), o);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&hd.q_full[i]);
    };

    bool loaded = false;  // the item's Q rows are already in place
    for (int64_t u = u0; u < u1;) {
      const int64_t len = min((int64_t)(c.it.tiles - c.tile), u1 - u);
      const bool mine = c.it.rows > 128 * i;  // a short item has no second half
      Cursor nx;
      if (mine) {
        if (!loaded && ok) load_q(c);
        loaded = false;
        const int64_t R = (int64_t)c.qt * kRows + min(128 * i + row, c.it.rows - 1);
        const int hi = c.s.L - c.s.n + (int)(R / p.v.group);  // last key that this row sees
        // keys that every row of the half sees
        const int64_t ra = (int64_t)c.qt * kRows + 128 * i, rb = (int64_t)c.qt * kRows + min(128 * i + 127, c.it.rows - 1);
        const int all_hi = c.s.L - c.s.n + (int)(ra / p.v.group);
        const int all_lo = p.a.window > 0 ? c.s.L - c.s.n + (int)(rb / p.v.group) - p.a.window + 1 : 0;
        float m = -INFINITY, l = 0.f;
        for (int64_t k = 0; k < len; ++k) {
          const int key0 = (c.it.lo + c.tile + (int)k) * kTile;
          ok = ok && warp_wait(&hd.s_full[i], n_s & 1u, p.wait_ns, kHintNs);
          ++n_s;
          if (!ok) continue;
          tc_fence_after_sync();
          uint32_t s[4][32];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld_x32(s_t + 32 * j, s[j]);
          tmem_ld_wait();
          const bool masked = key0 + kTile - 1 > all_hi || key0 < all_lo;
          if (masked) {
            const int d = hi - key0, e = p.a.window > 0 ? d - p.a.window : -1;
#pragma unroll
            for (int j = 0; j < 128; ++j)
              if (j > d || j <= e) s[j / 32][j % 32] = 0xFF800000u;
          }
          float top[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            top[j] = __uint_as_float(s[j][0]);
#pragma unroll
            for (int x = 1; x < 32; ++x) top[j] = fmaxf(top[j], __uint_as_float(s[j][x]));
          }
          const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          if (k == 0) {
            m = mx;
          } else if (__any_sync(0xffffffffu, m == -INFINITY ? mx > m : (mx - m) * sl > kLazy)) {
            // the previous product has finished (s_full covers it), the next waits for this thread
            const float mn = fmaxf(m, mx);
            const float f = m == -INFINITY ? 0.f : ex2((m - mn) * sl);
            m = mn;
            l *= f;
            for (int j = 0; j < D; j += 16) {
              uint32_t o[16];
              tmem_ld_x16(o_t + j, o);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
              tmem_st_x16(o_t + j, o);
            }
          }
          const float ms = m == -INFINITY ? 0.f : -m * sl;
          float sum[2] = {0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
              const float a = __uint_as_float(s[2 * j + x / 32][x % 32]), b = __uint_as_float(s[2 * j + x / 32][x % 32 + 1]);
              float pa = ex2(fmaf(a, sl, ms)), pb = ex2(fmaf(b, sl, ms));
              if (masked) {  // scale 0 makes 0 x infinity of a masked score
                pa = a == -INFINITY ? 0.f : pa;
                pb = b == -INFINITY ? 0.f : pb;
              }
              sum[0] += pa;
              sum[1] += pb;
              w[x / 2] = pack_bf16x2(pa, pb);
            }
            tmem_st_x32(s_t + 32 * j, w);
          }
          l += sum[0] + sum[1];
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&hd.p_full[i]);
        }
        nx = c;
        if (u + len < u1) next_item(p, nx);
        // the half's scores are done with its Q tile: the next item's rows go in while the last product runs
        if (u + len < u1 && nx.it.rows > 128 * i && ok) {
          load_q(nx);
          loaded = true;
        }
        // ---- the segment's result
        ok = ok && warp_wait(&hd.o_full[i], n_o & 1u, p.wait_ns, kHintNs);
        ++n_o;
        tc_fence_after_sync();
        const bool whole = c.tile == 0 && len == c.it.tiles;
        const bool real = 128 * i + row < c.it.rows;
        __nv_bfloat16* dst = p.a.out + (c.s.row + R / p.v.group) * p.a.ld_out +
                             (int64_t)(c.h * p.v.group + (int)(R % p.v.group)) * D;
        auto write32 = [&](int col, const float (&v)[32], float inv) {
#pragma unroll
          for (int g8 = 0; g8 < 4; ++g8) {
            const float* x = v + 8 * g8;  // elements 0, 4, 1, 5, 2, 6, 3, 7
            uint4 w;
            w.x = pack_bf16x2(x[0] * inv, x[2] * inv);
            w.y = pack_bf16x2(x[4] * inv, x[6] * inv);
            w.z = pack_bf16x2(x[1] * inv, x[3] * inv);
            w.w = pack_bf16x2(x[5] * inv, x[7] * inv);
            *reinterpret_cast<uint4*>(dst + col + 8 * g8) = w;
          }
        };
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
          for (int j = 0; j < D; j += 32) {
            uint32_t o[32];
            tmem_ld_x32(o_t + j, o);
            tmem_ld_wait();
            float v[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = l == 0.f ? 0.f : __uint_as_float(o[x]);
            if (real && ok) write32(j, v, inv);
          }
        } else {
          const int64_t first_unit = u - c.tile;
          const int64_t ca = ((first_unit + 1) * G - 1) / U, cb = ((first_unit + c.it.tiles) * G - 1) / U;
          float* slot = p.part + ((cta * 2 + (c.tile == 0 ? 1 : 0)) * 2 + i) * kPart + row;
#pragma unroll
          for (int j = 0; j < D; j += 32) {
            uint32_t o[32];
            tmem_ld_x32(o_t + j, o);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 32; ++x) __stcg(slot + (j + x) * 128, __uint_as_float(o[x]));
          }
          __stcg(slot + D * 128, m);
          __stcg(slot + (D + 1) * 128, l);
          __threadfence();
          wg_sync(1 + i);
          if (row == 0) hd.last[i] = atomicAdd(p.counters + ca * 2 + i, 1u) == (unsigned)(cb - ca);
          wg_sync(1 + i);
          if (*reinterpret_cast<volatile int*>(&hd.last[i])) {
            __threadfence();
            if (row == 0) p.counters[ca * 2 + i] = 0;
            float M = -INFINITY, Ls = 0.f;
            for (int64_t x = ca; x <= cb; ++x)
              M = fmaxf(M, __ldcg(p.part + ((x * 2 + (x == ca)) * 2 + i) * kPart + D * 128 + row));
            for (int64_t x = ca; x <= cb; ++x) {
              const float* q = p.part + ((x * 2 + (x == ca)) * 2 + i) * kPart + D * 128 + row;
              const float mx = __ldcg(q), lx = __ldcg(q + 128);
              Ls += mx == -INFINITY ? lx : lx * ex2((mx - M) * sl);
            }
            const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
              float v[32];
#pragma unroll
              for (int x = 0; x < 32; ++x) v[x] = 0.f;
              for (int64_t x = ca; x <= cb; ++x) {
                const float* q = p.part + ((x * 2 + (x == ca)) * 2 + i) * kPart + row;
                const float mx = __ldcg(q + D * 128), lx = __ldcg(q + (D + 1) * 128);
                const float f = mx == -INFINITY ? (lx == 0.f ? 0.f : 1.f) : ex2((mx - M) * sl);
                if (f != 0.f || lx != 0.f) {
#pragma unroll
                  for (int y = 0; y < 32; ++y) v[y] = fmaf(f, __ldcg(q + (j + y) * 128), v[y]);
                }
              }
              if (real && ok) write32(j, v, inv);
            }
          }
        }
        tc_fence_before_sync();
      } else {
        nx = c;
        if (u + len < u1) next_item(p, nx);
      }
      u += len;
      c = nx;
    }
    if (!ok && lane == 0) fail(p);
  }

  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
spear_status_t launch(const spear_kv_s* h, PrefillParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> done{0};
  if (smem_limit_once(reinterpret_cast<const void*>(prefill_kernel<D>), done) != cudaSuccess) return SPEAR_ERR_CUDA;
  // at least half of an SM's shared memory, so that one CTA has its tensor memory for itself
  const size_t used = kHeader + 6 * (size_t)kTile * D * 2 + 2 * (size_t)kBlocksPerTile * 16 * (D + 8);
  const size_t smem = used > 116 * 1024 ? used : 116 * 1024;
  prefill_kernel<D><<<h->sm_count, kThreads, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPEAR_OK : SPEAR_ERR_CUDA;
}

}  // namespace
}  // namespace spear

using namespace spear;

size_t kv_prefill_workspace(const spear_kv_s* h) {
  return (size_t)h->sm_count * 4 * (h->view.D + 2) * 128 * sizeof(float);
}

spear_status_t kv_launch_prefill(const spear_kv_s* h, const KvAttnArgs& a, int max_rows, float* part,
                                 unsigned* counters, cudaStream_t stream) {
  PrefillParams p;
  p.v = h->view;
  p.a = a;
  p.max_rows = max_rows;
  p.part = part;
  p.counters = counters;
  p.wait_ns = 100000000ull;
  return h->view.D == 128 ? launch<128>(h, p, stream) : launch<64>(h, p, stream);
}

// The paged 4-bit key/value cache: handle lifetime, argument checks, the
// append kernel (rotation, quantisation and the write into the pages, one
// launch) and the read-back kernel.
#include <math.h>

#include <new>

#include "kv.h"

namespace spear {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendChunk = 8, kAppendBlocks = 4;

SPEAR_DEVINL uint2 ldg_stream(const void* p) {  // read once: keep it out of L1
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

SPEAR_DEVINL void unpack4(const uint2& w, float* x) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

SPEAR_DEVINL float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
SPEAR_DEVINL float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The 16-token block of head 0 that holds a slot (in range); page_size is a multiple of 16.
SPEAR_DEVINL uint8_t* slot_block(const KvView& v, int64_t slot) {
  const int64_t blk = slot / 16;  // a 64-bit division by bpp takes ten times a 32-bit one
  const int page = blk <= 0xFFFFFFFFll ? (int)((uint32_t)blk / (uint32_t)v.bpp) : (int)(blk / v.bpp);
  return v.pool + ((int64_t)page * v.n_kv_heads * v.bpp + (blk - (int64_t)page * v.bpp)) * v.block_bytes;
}

struct AppendParams {
  KvView v;
  const __nv_bfloat16 *q, *k, *val;
  int64_t ld_q, ld_k, ld_v, ld_q_out;
  const int64_t *positions, *slots;
  int T;
  __nv_bfloat16* q_out;
  int rope_dim, n_positions;
  const float* table;
  int q_rows;  // rotated query rows a token (0: none)
  int rows;    // q_rows + 2 n_kv_heads
  int chunk;   // rows of one token that a group of lanes takes
};

// One row of D values is 8 elements a lane, LPR = D / 8 lanes: four from `a`
// on and four from `b` on, which for rotated halves are the four partners, so
// that a lane has both elements of its pairs and needs four cosines and sines.
// A group of LPR lanes takes `chunk` rows of one token (a token's cosines and
// sines are as many bytes as two rows), four rows' loads in flight. Products
// and sums are rounded one by one (no contraction), so that the codes are
// defined bit for bit. Bound by memory: a token reads and writes (2 n_heads +
// 2 n_kv_heads) D bf16 and writes 2 n_kv_heads (D / 2 + 4) bytes. Measured:
// 12289 tokens of 64 + 2 x 8 heads of 128 (470 MB) in 88 us, 5.3 TB/s, 79% of
// a plain copy; 1088 tokens of 32 + 2 x 32 heads (40 MB) in 14.5 us, 2.8 TB/s: there the
// launch, the slot and the first row's latency are a third of the time. (16
// bytes a lane of one row, partners exchanged by shuffles: 12289 tokens with
// the read-back took 265 us, against 102.)
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 8, U = 4;
  kv_follow();
  const int sub = threadIdx.x % LPR, lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
  if (t >= p.T) return;  // whole groups leave: the shuffles below are within a group
  const uint32_t mask = (uint32_t)((1ull << LPR) - 1) << (lane / LPR * LPR);
  const int r0 = blockIdx.y * p.chunk;
  const int r1 = min(r0 + p.chunk, p.rows);

  const int half = p.rope_dim / 2;
  const bool rotated = kInterleaved ? 8 * sub < p.rope_dim : 4 * sub < half;
  int a = 8 * sub, b = 8 * sub + 4;  // the lane's elements
  if (!kInterleaved && p.rope_dim > 0) {
    a = rotated ? 4 * sub : p.rope_dim + 8 * (sub - half / 4);
    b = rotated ? a + half : a + 4;
  }

  // row r of the token, as q rows, k rows, v rows
  const __nv_bfloat16* qs = p.q + t * p.ld_q;
  const __nv_bfloat16* ks = p.k + t * p.ld_k;
  const __nv_bfloat16* vs = p.val + t * p.ld_v;
  const int k_end = p.q_rows + p.v.n_kv_heads;
  auto source = [&](int r) {
    return r < p.q_rows ? qs + r * D : r < k_end ? ks + (r - p.q_rows) * D : vs + (r - k_end) * D;
  };
  uint2 wa[U], wb[U];
  auto load = [&](int r) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const __nv_bfloat16* src = source(min(r + u, r1 - 1));
      wa[u] = ldg_stream(src + a);
      wb[u] = ldg_stream(src + b);
    }
  };
  load(r0);

  const int64_t slot = p.slots[t];
  const int64_t n_slots = (int64_t)p.v.n_pages * p.v.page_size;
  bool bad = slot < -1 || slot >= n_slots;
  uint8_t* block = nullptr;
  if (slot >= 0 && slot < n_slots) {
    block = slot_block(p.v, slot) + slot % 16 * 4;  // of the parameters
  }
  const int codes_at = (int)(slot % 16) * (D / 2 - 4);  // page_size is a multiple of 16

  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.rope_dim > 0) {
    const int64_t pos = p.positions[t];
    const bool ok = pos >= 0 && pos < p.n_positions;
    bad |= !ok;
    if (ok && rotated) {
      const float* row = p.table + pos * p.rope_dim + 4 * sub;
      *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(row);
      *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(row + half);
    }
  }
  if (bad) {
    if (sub == 0) atomicOr(p.v.status, kStatusBadIndex);
    return;
  }

  for (int r = r0; r < r1; r += U) {
    if (r > r0) load(r);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ru = r + u;
      if (ru >= r1) break;
      float x[8];
      unpack4(wa[u], x);
      unpack4(wb[u], x + 4);
      if (ru < k_end && rotated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          constexpr int f = kInterleaved ? 2 : 1, d = kInterleaved ? 1 : 4;
          const float x1 = x[f * i], x2 = x[f * i + d];
          x[f * i] = __fsub_rn(__fmul_rn(x1, c[i]), __fmul_rn(x2, s[i]));
          x[f * i + d] = __fadd_rn(__fmul_rn(x2, c[i]), __fmul_rn(x1, s[i]));
        }
      }
      if (ru < p.q_rows) {
        __nv_bfloat16* dst = p.q_out + t * p.ld_q_out + ru * D;
        *reinterpret_cast<uint2*>(dst + a) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        *reinterpret_cast<uint2*>(dst + b) = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        continue;
      }
      float lo = x[0], hi = x[0];  // a NaN stays one; infinities show in the range
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) {
        lo = min_nan(lo, __shfl_xor_sync(mask, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(mask, hi, o));
      }
      const float range = __fsub_rn(hi, lo);
      __nv_bfloat16 sb = __float2bfloat16_rn(__fmul_rn(range, 1.0f / 15.0f));
      const __nv_bfloat16 ob = __float2bfloat16_rn(lo);
      if (__bfloat162float(sb) < 1.17549435e-38f) sb = __float2bfloat16_rn(0.f);
      const float sf = __bfloat162float(sb), of = __bfloat162float(ob);
      const float inv = sf > 0.f ? __fdiv_rn(1.f, sf) : 0.f;
      // Adding and taking away 2^23 rounds to an integer (half to even); four codes are one number below 2^16, whose
      // bits stand in the sum with 2^23.
      uint32_t codes[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[i] = __fsub_rn(__fadd_rn(fminf(fmaxf(__fmul_rn(__fsub_rn(x[4 * y + i], of), inv), 0.f), 15.f), 8388608.f),
                           8388608.f);
        codes[y] = __float_as_uint(fmaf(fmaf(fmaf(f[3], 16.f, f[2]), 16.f, f[1]), 16.f, f[0]) + 8388608.f);
      }
      uint32_t par = (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(ob) << 16);
      if (!(range <= 0x1p120f)) par = 0x7FC07FC0u;
      if (block) {
        const int is_v = ru >= k_end;
        uint8_t* row = block + (int64_t)(is_v ? ru - k_end : ru - p.q_rows) * p.v.bpp * p.v.block_bytes;
        uint8_t* cd = row + codes_at + is_v * 8 * D;
        *reinterpret_cast<uint16_t*>(cd + a / 2) = (uint16_t)codes[0];
        *reinterpret_cast<uint16_t*>(cd + b / 2) = (uint16_t)codes[1];
        if (sub == 0) *reinterpret_cast<uint32_t*>(row + 16 * D + is_v * 64) = par;
      }
    }
  }
}

// A group of D / 8 lanes hands back `chunk` of a token's 2 n_kv_heads rows (8
// elements a lane), four rows' loads in flight. Bound by memory: 12289 tokens
// of 2 x 8 heads of 128 (64 MB, most of it written) take 13.4 us, 4.8 TB/s.
template <int D>
__global__ void __launch_bounds__(kAppendThreads)
    read_kernel(const KvView v, const int64_t* __restrict__ slots, int T, int chunk, __nv_bfloat16* k_out,
                __nv_bfloat16* v_out) {
  constexpr int LPR = D / 8, U = 4;
  kv_follow();
  const int sub = threadIdx.x % LPR;
  const int t = blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
  if (t >= T) return;
  const int r0 = blockIdx.y * chunk, r1 = min(r0 + chunk, 2 * v.n_kv_heads);
  const int64_t slot = slots[t];
  const bool held = slot >= 0 && slot < (int64_t)v.n_pages * v.page_size;
  if (!held && slot != -1 && sub == 0) atomicOr(v.status, kStatusBadIndex);
  const uint8_t* b = held ? slot_block(v, slot) : v.pool;
  const int at = (int)(slot & 15);
  for (int r = r0; r < r1; r += U) {
    uint32_t codes[U], par[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ru = min(r + u, r1 - 1), is_v = ru >= v.n_kv_heads;
      const uint8_t* row = b + (int64_t)(is_v ? ru - v.n_kv_heads : ru) * v.bpp * v.block_bytes;
      codes[u] = held ? *reinterpret_cast<const uint32_t*>(row + is_v * 8 * D + at * (D / 2) + sub * 4) : 0u;
      par[u] = held ? *reinterpret_cast<const uint32_t*>(row + 16 * D + is_v * 64 + at * 4) : 0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ru = r + u, is_v = ru >= v.n_kv_heads;
      if (ru >= r1) break;
      const float s = __uint_as_float(par[u] << 16), o = __uint_as_float(par[u] & 0xFFFF0000u);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(fmaf((float)((codes[u] >> (8 * i)) & 15u), s, o),
                           fmaf((float)((codes[u] >> (8 * i + 4)) & 15u), s, o));
      __nv_bfloat16* dst = (is_v ? v_out : k_out) + ((int64_t)t * v.n_kv_heads + (is_v ? ru - v.n_kv_heads : ru)) * D;
      *reinterpret_cast<uint4*>(dst + sub * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Rows of a token that a group takes: up to kAppendChunk, as long as the device stays filled.
int rows_per_group(const spear_kv_s* h, int T, int rows, int64_t groups_per_block) {
  int chunk = kAppendChunk;
  while (chunk > 1 && (int64_t)T * rows < chunk * groups_per_block * kAppendBlocks * h->sm_count) chunk /= 2;
  return chunk;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool row_ok(const void* p, int64_t ld, int64_t len) { return p && aligned16(p) && ld % 8 == 0 && ld >= len; }

// T rows of `len` elements, `ld` from one to the next.
struct Rows {
  const void* p;
  int64_t ld, len;
};

// Whether no element of one is the other's: ranges that do not meet, or columns of the same rows that do not.
bool apart(const Rows& a, const Rows& b, int64_t T) {
  const auto pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const Rows &lo = pa <= pb ? a : b, &up = pa <= pb ? b : a;
  const int64_t off = (int64_t)((pa <= pb ? pb - pa : pa - pb) / 2);  // elements; both are aligned
  if (off >= (T - 1) * lo.ld + lo.len) return true;
  return T > 1 && a.ld == b.ld && off % a.ld >= lo.len && off % a.ld + up.len <= a.ld;
}
bool same(const Rows& a, const Rows& b, int64_t T) { return a.p == b.p && (a.ld == b.ld || T == 1); }

}  // namespace
}  // namespace spear

using namespace spear;

extern "C" {

spear_status_t spear_kv_create(const spear_kv_desc_t* d, cudaStream_t stream, spear_kv_t* out) {
  if (!out) return SPEAR_ERR_INVALID_ARG;
  *out = nullptr;
  if (!d || !d->pool || !aligned16(d->pool)) return SPEAR_ERR_INVALID_ARG;
  if (d->n_kv_heads < 1 || d->n_heads < d->n_kv_heads || d->n_heads % d->n_kv_heads != 0 ||
      d->n_heads / d->n_kv_heads > 32 || d->n_heads > 4096)
    return SPEAR_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return SPEAR_ERR_INVALID_ARG;
  if (d->page_size < 16 || d->page_size % 16 != 0 || d->page_size > 65536 || d->n_pages < 1)
    return SPEAR_ERR_INVALID_ARG;
  if (d->rope_dim < 0 || d->rope_dim % 16 != 0 || d->rope_dim > d->head_dim) return SPEAR_ERR_INVALID_ARG;
  if (d->rope_dim > 0 && (d->n_positions < 1 || !d->rope_table || !aligned16(d->rope_table)))
    return SPEAR_ERR_INVALID_ARG;
  spear_kv_s* h = new (std::nothrow) spear_kv_s();
  if (!h) return SPEAR_ERR_OOM;
  h->view.pool = static_cast<uint8_t*>(d->pool);
  h->view.n_heads = d->n_heads;
  h->view.n_kv_heads = d->n_kv_heads;
  h->view.group = d->n_heads / d->n_kv_heads;
  h->view.D = d->head_dim;
  h->view.page_size = d->page_size;
  h->view.bpp = d->page_size / 16;
  h->view.n_pages = d->n_pages;
  h->view.block_bytes = 16 * (d->head_dim + 8);
  h->rope_dim = d->rope_dim;
  h->rope_interleaved = d->rope_interleaved != 0;
  h->n_positions = d->n_positions;
  h->rope_table = d->rope_table;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device);
  if (e == cudaSuccess) {
    h->ws_bytes = kv_attention_workspace(h);
    e = cudaMalloc(&h->ws, h->ws_bytes);
  }
  if (e == cudaSuccess) e = cudaMemsetAsync(h->ws, 0, kKvControlBytes, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);  // the first call may be on another stream
  if (e != cudaSuccess) {
    cudaGetLastError();
    if (h->ws) cudaFree(h->ws);
    delete h;
    return e == cudaErrorMemoryAllocation ? SPEAR_ERR_OOM : SPEAR_ERR_CUDA;
  }
  h->view.status = static_cast<unsigned*>(h->ws);
  *out = h;
  return SPEAR_OK;
}

spear_status_t spear_kv_append(spear_kv_t h, const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                               int64_t ld_v, const int64_t* positions, const int64_t* slots, int32_t T, void* q_out,
                               int64_t ld_q_out, cudaStream_t stream) {
  if (!h || T < 0) return SPEAR_ERR_INVALID_ARG;
  if (T == 0) return SPEAR_OK;
  const int64_t D = h->view.D, qn = h->view.n_heads * D, kn = h->view.n_kv_heads * D;
  if (!row_ok(k, ld_k, kn) || !row_ok(v, ld_v, kn) || !slots || (h->rope_dim > 0 && !positions))
    return SPEAR_ERR_INVALID_ARG;
  if (q) {
    if (!row_ok(q, ld_q, qn) || !row_ok(q_out, ld_q_out, qn)) return SPEAR_ERR_INVALID_ARG;
    const Rows qr{q, ld_q, qn}, outr{q_out, ld_q_out, qn};
    if ((!same(qr, outr, T) && !apart(qr, outr, T)) || !apart({k, ld_k, kn}, outr, T) || !apart({v, ld_v, kn}, outr, T))
      return SPEAR_ERR_INVALID_ARG;
  }
  AppendParams p;
  p.v = h->view;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.val = static_cast<const __nv_bfloat16*>(v);
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_v = ld_v;
  p.ld_q_out = ld_q_out;
  p.positions = positions;
  p.slots = slots;
  p.T = T;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.rope_dim = h->rope_dim;
  p.n_positions = h->n_positions;
  p.table = h->rope_table;
  p.q_rows = q ? h->view.n_heads : 0;
  p.rows = p.q_rows + 2 * h->view.n_kv_heads;
  const int64_t per_block = kAppendThreads / (D / 8);
  p.chunk = rows_per_group(h, T, p.rows, per_block);
  const dim3 blocks((unsigned)((T + per_block - 1) / per_block), (p.rows + p.chunk - 1) / p.chunk);
  auto* kernel = D == 128 ? (h->rope_interleaved ? append_kernel<128, true> : append_kernel<128, false>)
                          : (h->rope_interleaved ? append_kernel<64, true> : append_kernel<64, false>);
  return kv_launch(kernel, blocks, kAppendThreads, 0, stream, p);
}

spear_status_t spear_kv_read(spear_kv_t h, const int64_t* slots, int32_t T, void* k_out, void* v_out,
                             cudaStream_t stream) {
  if (!h || T < 0) return SPEAR_ERR_INVALID_ARG;
  if (T == 0) return SPEAR_OK;
  if (!slots || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return SPEAR_ERR_INVALID_ARG;
  const int D = h->view.D, kn = h->view.n_kv_heads * D;
  if (!apart({k_out, kn, kn}, {v_out, kn, kn}, T)) return SPEAR_ERR_INVALID_ARG;
  const int64_t per_block = kAppendThreads / (D / 8);
  const int rows = 2 * h->view.n_kv_heads, chunk = rows_per_group(h, T, rows, per_block);
  const dim3 blocks((unsigned)((T + per_block - 1) / per_block), (rows + chunk - 1) / chunk);
  auto* kernel = D == 128 ? read_kernel<128> : read_kernel<64>;
  return kv_launch(kernel, blocks, kAppendThreads, 0, stream, h->view, slots, T, chunk,
                   static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out));
}

spear_status_t spear_kv_attention(spear_kv_t h, const void* q, int64_t ld_q, void* out, int64_t ld_out,
                                  const int32_t* page_table, int32_t ld_pt, const int32_t* kv_lens,
                                  const int32_t* q_starts, int32_t n_seqs, int32_t T, int32_t max_q, float scale,
                                  int32_t window, cudaStream_t stream) {
  if (!h || n_seqs < 0 || T < 0) return SPEAR_ERR_INVALID_ARG;
  if (n_seqs == 0 || T == 0) return SPEAR_OK;
  const int64_t qn = (int64_t)h->view.n_heads * h->view.D;
  if (!row_ok(q, ld_q, qn) || !row_ok(out, ld_out, qn) || !page_table || ld_pt < 1 || !kv_lens || !q_starts ||
      max_q < 1 || window < 0 || !isfinite(scale) ||
      (int64_t)T * h->view.group >= (1 << 27))
    return SPEAR_ERR_INVALID_ARG;
  const Rows qr{q, ld_q, qn}, outr{out, ld_out, qn};
  if (!same(qr, outr, T) && !apart(qr, outr, T)) return SPEAR_ERR_INVALID_ARG;
  KvAttnArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.ld_q = ld_q;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.ld_out = ld_out;
  a.page_table = page_table;
  a.ld_pt = ld_pt;
  a.kv_lens = kv_lens;
  a.q_starts = q_starts;
  a.n_seqs = n_seqs;
  a.T = T;
  a.max_q = max_q;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.window = window > kKvMaxTokens ? 0 : window;  // no sequence is longer
  return kv_launch_attention(h, a, stream);
}

spear_status_t spear_kv_check(spear_kv_t h, cudaStream_t stream) {
  if (!h) return SPEAR_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return SPEAR_ERR_CUDA;
  unsigned status = 0;
  if (cudaMemcpy(&status, h->view.status, sizeof status, cudaMemcpyDeviceToHost) != cudaSuccess)
    return SPEAR_ERR_CUDA;
  if (status == 0) return SPEAR_OK;
  if (cudaMemset(h->ws, 0, kKvControlBytes) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess)
    return SPEAR_ERR_CUDA;
  return (status & kStatusTimeoutPipe) ? SPEAR_ERR_TIMEOUT : SPEAR_ERR_INVALID_ARG;
}

spear_status_t spear_kv_destroy(spear_kv_t h) {
  if (!h) return SPEAR_OK;
  if (h->ws) cudaFree(h->ws);
  delete h;
  return SPEAR_OK;
}

}  // extern "C"

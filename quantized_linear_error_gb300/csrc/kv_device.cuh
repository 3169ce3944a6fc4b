// Device helpers shared by the attention kernels over the paged 4-bit cache.
#pragma once
#include <math.h>

#include "kv.h"

namespace spear {

SPEAR_DEVINL float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

SPEAR_DEVINL uint32_t f16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

SPEAR_DEVINL uint32_t pack_f16x2(float lo, float up) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(up), "f"(lo));
  return r;
}

// Two fp32 operations in one instruction, on register pairs.
SPEAR_DEVINL uint64_t pack_b32x2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
SPEAR_DEVINL uint64_t pack_f32x2(float a, float b) { return pack_b32x2(__float_as_uint(a), __float_as_uint(b)); }
SPEAR_DEVINL void unpack_f32x2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
SPEAR_DEVINL uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SPEAR_DEVINL uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// a / b for a, b >= 0: most are small, and a 64-bit division takes several times a 32-bit one.
SPEAR_DEVINL int64_t div_u64(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : (int64_t)((uint64_t)a / (uint64_t)b);
}

// The first key that a row at position `pos` sees.
SPEAR_DEVINL int first_key(const KvAttnArgs& a, int pos) { return a.window > 0 ? max(0, pos - a.window + 1) : 0; }

// Sequence b of a call as a kernel works on it, every index checked.
struct KvSeq {
  int n;         // query rows (0: nothing to do)
  int row;       // first query row
  int L;         // cached tokens
  int lo;        // first tile that any row sees
  int tiles;     // tiles of `tile` keys from there (at least one, which a sequence without keys masks out)
};

SPEAR_DEVINL KvSeq kv_seq(const KvView& v, const KvAttnArgs& a, int b, int tile) {
  KvSeq s;
  s.row = a.q_starts[b];
  const int end = a.q_starts[b + 1];
  const int len = a.kv_lens[b];
  const int64_t room = min((int64_t)a.ld_pt * v.page_size, (int64_t)kKvMaxTokens);
  const bool rows_ok = s.row >= 0 && end >= s.row && end <= a.T && end - s.row <= a.max_q;
  const bool len_ok = len >= 0 && len <= room;
  if (!rows_ok || !len_ok) atomicOr(v.status, kStatusBadIndex);
  s.n = rows_ok ? end - s.row : 0;
  s.L = len_ok ? len : (len < 0 ? 0 : (int)room);
  s.lo = first_key(a, s.L - s.n) / tile;
  s.tiles = max(1, (s.L + tile - 1) / tile - s.lo);
  return s;
}

}  // namespace spear

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
  const int64_t first = a.window > 0 ? (int64_t)s.L - s.n - a.window + 1 : 0;  // first key that row 0 sees
  s.lo = first > 0 ? (int)(first / tile) : 0;
  s.tiles = max(1, (s.L + tile - 1) / tile - s.lo);
  return s;
}

}  // namespace spear

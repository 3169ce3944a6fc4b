// Attention over the paged 4-bit cache: which kernel takes which sequences.
#include <algorithm>

#include "kv.h"

size_t kv_attention_workspace(const spear_kv_s* h) {
  return kKvControlBytes + std::max(kv_decode_workspace(h), kv_prefill_workspace(h));
}

spear_status_t kv_launch_attention(spear_kv_s* h, const KvAttnArgs& a, cudaStream_t stream) {
  char* ws = static_cast<char*>(h->ws);
  auto* counters = reinterpret_cast<unsigned*>(ws + 128);
  auto* part = reinterpret_cast<float*>(ws + kKvControlBytes);
  // Up to kKvDecodeRows rows a key/value head the few-row kernel is the faster, or within 2%: 32 sequences x 8 key/value
  // heads x 4000 keys with 16 / 24 / 32 rows take 60 / 100 / 102 us against 99 / 100 / 100 of the chunk kernel, whose time
  // is the same from 9 to 128 rows (D = 64: 40 / 76 / 76 against 78 / 78 / 79); 64 sequences of 500 keys with 20 rows 48
  // against 50 (D = 64: 30 against 37); 4 of 4000 keys with 32 rows 24 against 26 (D = 64: 18 against 21).
  // Beside a chunk the few-row kernel takes the variant of single tokens: a larger one costs them more than drafts gain.
  // 32 sequences of 2000 to 4000 keys and a chunk of 512, 4 heads a key/value head, with the variant of 8 / 16 / 32 rows:
  // single tokens 70 / 87 / 116 us, 2 drafts 72 / 89 / 119, 8 drafts 104 / 104 / 126 (8 sequences: 49 / 54 / 61, 49 / 54
  // / 63, 50 / 49 / 67). 4 drafts, which are 16 rows, lose with 32 sequences, 104 / 92 / 119, not with 8, 50 / 57 / 62.
  // Both kernels read the lengths on the device and leave the other's sequences
  // out; they follow each other on the stream, so they share the workspace.
  const int64_t most = (int64_t)a.max_q * h->view.group;
  const bool chunks = most > kKvDecodeRows;
  const int64_t few = chunks ? h->view.group : most;
  const int nt = few <= 8 ? 1 : (few <= 16 ? 2 : 4);
  if (!chunks) return kv_launch_decode(h, a, nt, part, counters, stream);
  if (a.n_seqs == 1) return kv_launch_prefill(h, a, 0, part, stream);
  const spear_status_t st = kv_launch_decode(h, a, nt, part, counters, stream);
  return st != SPEAR_OK ? st : kv_launch_prefill(h, a, 8 * nt, part, stream);
}

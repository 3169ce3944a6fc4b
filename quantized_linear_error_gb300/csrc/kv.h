// The key/value cache handle and the device-side view of its pool, shared by
// the append/read kernels and the attention kernels.
#pragma once
#include "internal.h"

struct KvView {
  uint8_t* pool;
  int n_heads, n_kv_heads, group;  // group = n_heads / n_kv_heads
  int D;
  int page_size, bpp;              // bpp = 16-token blocks per page
  int n_pages;
  int block_bytes;                 // 16 * (D + 8)
  unsigned* status;
};

struct spear_kv_s {
  KvView view;
  int rope_dim, rope_interleaved, n_positions;
  const float* rope_table;
  int device, sm_count;
  void* ws;
  size_t ws_bytes;
};

// Launches a kernel that begins with kv_follow(): it is set up on the SMs while
// the kernel before it on the stream ends.
template <class... P, class... A>
inline spear_status_t kv_launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                const A&... args) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? SPEAR_OK : SPEAR_ERR_CUDA;
}

#ifdef __CUDACC__
// Lets the next kernel be set up, and waits until the work before this one on
// the stream has ended and is visible. Nothing outside the SM is touched before.
SPEAR_DEVINL void kv_follow() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
#endif

// Arguments of one attention call.
struct KvAttnArgs {
  const __nv_bfloat16* q;
  int64_t ld_q;
  __nv_bfloat16* out;
  int64_t ld_out;
  const int32_t* page_table;
  int ld_pt;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int n_seqs, T, max_q;
  float scale_log2;  // scale * log2(e): scores are kept in units of log2
  int window;
};

// The workspace starts with the status word and one arrival counter per CTA of
// the kernels that split a sequence (cleared at create), then partial results.
constexpr size_t kKvControlBytes = 16384;
constexpr int kKvMaxTokens = 1 << 30;  // longest sequence: key numbers and their sums with a tile fit 32 bits
constexpr int kKvDecodeRows = 32;      // most rows of a key/value head that the cache-streaming kernel takes
// The kernel that streams the cache for sequences of at most 8 nt rows a
// key/value head (nt 1, 2 or 4); others are left out.
spear_status_t kv_launch_decode(const spear_kv_s* h, const KvAttnArgs& a, int nt, float* part, unsigned* counters,
                                cudaStream_t stream);
size_t kv_decode_workspace(const spear_kv_s* h);
// The tensor-core kernel for the sequences with more than max_rows rows a key/value head.
spear_status_t kv_launch_prefill(const spear_kv_s* h, const KvAttnArgs& a, int max_rows, void* ws,
                                 cudaStream_t stream);
size_t kv_prefill_workspace(const spear_kv_s* h);
size_t kv_attention_workspace(const spear_kv_s* h);
spear_status_t kv_launch_attention(spear_kv_s* h, const KvAttnArgs& a, cudaStream_t stream);

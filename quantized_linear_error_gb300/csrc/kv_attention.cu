// Attention over the paged 4-bit cache: launch.
#include "kv.h"

namespace spear {
namespace {

constexpr int kThreads = 128;

// One warp per (query row, head): every visible key in turn, softmax with a
// running maximum and sum, D / 32 elements a lane.
template <int D>
__global__ void __launch_bounds__(kThreads) simple_kernel(KvView v, KvAttnArgs a, int max_rows) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (unit >= (int64_t)a.T * v.n_heads) return;
  const int t = (int)(unit / v.n_heads), head = (int)(unit % v.n_heads), kvh = head / v.group;
  int b = -1;
  for (int i = lane; i < a.n_seqs; i += 32)
    if (t >= a.q_starts[i] && t < a.q_starts[i + 1]) b = i;
  b = __reduce_max_sync(0xffffffffu, b);
  if (b < 0) return;
  const int n = a.q_starts[b + 1] - a.q_starts[b];
  if (n * v.group <= max_rows) return;
  const int64_t room = (int64_t)a.ld_pt * v.page_size;
  int64_t L = a.kv_lens[b];
  if (L < 0 || L > room) {
    if (lane == 0) atomicOr(v.status, kStatusBadIndex);
    L = L < 0 ? 0 : room;
  }
  const int64_t pos = L - n + (t - a.q_starts[b]);
  const int64_t j0 = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
  float q[E], o[E];
  const __nv_bfloat16* qr = a.q + t * a.ld_q + (int64_t)head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(qr[e]), o[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = j0; j <= pos; ++j) {
    const int page = a.page_table[(int64_t)b * a.ld_pt + j / v.page_size];
    if (page < 0 || page >= v.n_pages) {
      if (lane == 0) atomicOr(v.status, kStatusBadIndex);
      continue;
    }
    const int at = (int)(j % v.page_size), r = at % 16;
    const uint8_t* blk = v.pool + (((int64_t)page * v.n_kv_heads + kvh) * v.bpp + at / 16) * v.block_bytes;
    const uint32_t kp = *reinterpret_cast<const uint32_t*>(blk + 16 * D + r * 4);
    const uint32_t vp = *reinterpret_cast<const uint32_t*>(blk + 16 * D + 64 + r * 4);
    float dot = 0.f, val[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane * E + e;
      const int kc = blk[r * (D / 2) + i / 2] >> (4 * (i & 1)) & 15;
      const int vc = blk[8 * D + r * (D / 2) + i / 2] >> (4 * (i & 1)) & 15;
      dot = fmaf(q[e], fmaf((float)kc, __uint_as_float(kp << 16), __uint_as_float(kp & 0xFFFF0000u)), dot);
      val[e] = fmaf((float)vc, __uint_as_float(vp << 16), __uint_as_float(vp & 0xFFFF0000u));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
    const float s = dot * a.scale_log2;
    const float mn = fmaxf(m, s), alpha = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + p * val[e];
  }
  __nv_bfloat16* dst = a.out + t * a.ld_out + (int64_t)head * D + lane * E;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16_rn(o[e] * inv);
}

}  // namespace
}  // namespace spear

using namespace spear;

size_t kv_attention_workspace(const spear_kv_s* h) { return kKvControlBytes + kv_decode_workspace(h); }

spear_status_t kv_launch_attention(spear_kv_s* h, const KvAttnArgs& a, cudaStream_t stream) {
  char* ws = static_cast<char*>(h->ws);
  auto* counters = reinterpret_cast<unsigned*>(ws + 128);
  auto* part = reinterpret_cast<float*>(ws + kKvControlBytes);
  const int64_t most = (int64_t)a.max_q * h->view.group;
  const bool chunks = most > kKvDecodeRows;
  const int64_t few = chunks ? h->view.group : most;
  const int nt = few <= 8 ? 1 : (few <= 16 ? 2 : 4);
  int max_rows = 0;
  if (!chunks || a.n_seqs > 1) {
    max_rows = 8 * nt;
    const spear_status_t st = kv_launch_decode(h, a, nt, part, counters, stream);
    if (st != SPEAR_OK || !chunks) return st;
  }
  const int64_t blocks = ((int64_t)a.T * h->view.n_heads + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7FFFFFFF) return SPEAR_ERR_INVALID_ARG;
  if (h->view.D == 128)
    simple_kernel<128><<<(unsigned)blocks, kThreads, 0, stream>>>(h->view, a, max_rows);
  else
    simple_kernel<64><<<(unsigned)blocks, kThreads, 0, stream>>>(h->view, a, max_rows);
  return cudaGetLastError() == cudaSuccess ? SPEAR_OK : SPEAR_ERR_CUDA;
}

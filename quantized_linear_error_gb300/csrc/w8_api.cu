// Linears of 8-bit integers: handle lifetime, argument checks, the weight
// layout kernel and the dispatch by token count.
#include <algorithm>
#include <new>

#include "w8_device.cuh"

namespace spear {
namespace {

// One thread a 16-byte chunk of the layout (see w8.h).
__global__ void __launch_bounds__(256) layout_kernel(const int8_t* __restrict__ q0, const int8_t* __restrict__ q1, int N,
                                                     int K, int kb, int64_t chunks, uint8_t* __restrict__ w) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const int64_t block = i >> 6;
  const int r = (int)(i >> 2) & 15, t = (int)i & 3;
  const int64_t at = block / 2, pair = at / kb, strip = pair * 2 + block % 2;
  const int k = (int)(at - pair * kb) * kW8K + t * 16;
  const int8_t* src = q0;
  int64_t n = strip * 16 + r;
  if (q1) {
    src = r < 8 ? q0 : q1;
    n = strip * 8 + (r & 7);
  }
  uint4 v = make_uint4(0, 0, 0, 0);
  if (n < N && k < K) v = *reinterpret_cast<const uint4*>(src + n * K + k);
  v.x ^= kW8Bias, v.y ^= kW8Bias, v.z ^= kW8Bias, v.w ^= kW8Bias;
  *reinterpret_cast<uint4*>(w + block * kW8Block + w8_place(r, t) * 16) = v;
}

__global__ void __launch_bounds__(256) scales_kernel(const float* __restrict__ s0, const float* __restrict__ s1, int N,
                                                     int rows, float* __restrict__ out) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= rows) return;
  const float* src = s1 && (i & 8) ? s1 : s0;
  const int n = s1 ? (i >> 4) * 8 + (i & 7) : i;
  out[i] = n < N ? src[n] : 0.f;
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace spear

using namespace spear;

namespace {

// The sizes that a descriptor asks for, or why not.
spear_status_t set_up(const spear_w8_desc_t* d, spear_w8_s* h) {
  if (!d || !d->qweight || !d->scales || !aligned(d->qweight, 16) || !aligned(d->scales, 4)) return SPEAR_ERR_INVALID_ARG;
  if (d->K < 16 || d->K % 16 != 0 || d->N < 1 || d->max_tokens < 1) return SPEAR_ERR_INVALID_ARG;
  h->gated = d->qweight_up != nullptr;
  if (h->gated) {
    if (!aligned(d->qweight_up, 16) || !d->scales_up || !aligned(d->scales_up, 4)) return SPEAR_ERR_INVALID_ARG;
    if (d->activation != SPEAR_ACT_SILU && d->activation != SPEAR_ACT_GELU) return SPEAR_ERR_INVALID_ARG;
  } else if (d->scales_up) {
    return SPEAR_ERR_INVALID_ARG;
  }
  if (d->workspace && (!aligned(d->workspace, 128) || d->workspace_bytes < 0)) return SPEAR_ERR_INVALID_ARG;
  if (d->K > (1 << 20) || d->N > (1 << 22) || d->max_tokens > (1 << 20)) return SPEAR_ERR_UNSUPPORTED;
  h->K = d->K, h->N = d->N, h->act = d->activation, h->max_tokens = d->max_tokens;
  h->kb = (d->K + 2 * kW8K - 1) / (2 * kW8K) * 2;
  h->strips = h->gated ? (d->N + 7) / 8 : (d->N + 15) / 16;
  h->strips = (h->strips + kW8Tile - 1) / kW8Tile * kW8Tile;
  if ((int64_t)h->strips * h->kb > 1 << 30) return SPEAR_ERR_UNSUPPORTED;  // block numbers are 32-bit
  return SPEAR_OK;
}

spear_status_t look_at_device(spear_w8_s* h) {
  return cudaGetDevice(&h->device) == cudaSuccess &&
                 cudaDeviceGetAttribute(&h->sm_count, cudaDevAttrMultiProcessorCount, h->device) == cudaSuccess
             ? SPEAR_OK
             : SPEAR_ERR_CUDA;
}

// [part][sums][x16]: the first two at the same place whatever the layer, so that handles that share a workspace leave
// each other's zeros alone.
size_t workspace_bytes(const spear_w8_s* h) {
  return w8_decode_workspace(h) + w8_prefill_sums(h) + w8_prefill_workspace(h);
}

}  // namespace

extern "C" spear_status_t spear_w8_workspace(const spear_w8_desc_t* d, int64_t* bytes) {
  if (!bytes) return SPEAR_ERR_INVALID_ARG;
  spear_w8_s h = {};
  spear_status_t st = set_up(d, &h);
  if (st == SPEAR_OK) st = look_at_device(&h);
  if (st == SPEAR_OK) *bytes = (int64_t)workspace_bytes(&h);
  return st;
}

extern "C" spear_status_t spear_w8_create(const spear_w8_desc_t* d, cudaStream_t stream, spear_w8_t* out) {
  if (!out) return SPEAR_ERR_INVALID_ARG;
  *out = nullptr;
  spear_w8_s* h = new (std::nothrow) spear_w8_s();
  if (!h) return SPEAR_ERR_OOM;
  spear_status_t st = set_up(d, h);
  if (st == SPEAR_OK) st = look_at_device(h);
  if (st == SPEAR_OK && d->workspace && (size_t)d->workspace_bytes < workspace_bytes(h)) st = SPEAR_ERR_INVALID_ARG;
  if (st != SPEAR_OK) {
    delete h;
    return st;
  }
  const int64_t blocks = (int64_t)h->strips * h->kb;
  h->control_bytes = (32 + h->strips + w8_prefill_counters(h)) * 4;
  h->sums_bytes = w8_prefill_sums(h);
  h->wait_ns = kW8WaitNs;
  cudaError_t e = cudaMalloc(&h->w, (size_t)blocks * kW8Block);
  if (e == cudaSuccess) e = cudaMalloc(&h->w_scales, (size_t)h->strips * 16 * 4);
  if (e == cudaSuccess) e = cudaMalloc(&h->control, h->control_bytes);
  h->ws = d->workspace;
  if (e == cudaSuccess && !h->ws) {
    e = cudaMalloc(&h->ws, workspace_bytes(h));
    h->ws_owned = 1;
  }
  if (e == cudaSuccess) {
    h->status = static_cast<unsigned*>(h->control);
    h->counters = h->status + 32;
    h->gemm_counters = h->counters + h->strips;
    char* ws = static_cast<char*>(h->ws);
    h->part = reinterpret_cast<float*>(ws);
    ws += w8_decode_workspace(h);
    h->spoilt = reinterpret_cast<unsigned*>(ws);
    h->sums = reinterpret_cast<int*>(ws + kW8SumsAt);
    h->x16 = reinterpret_cast<uint8_t*>(ws + h->sums_bytes);
    e = cudaMemsetAsync(h->control, 0, h->control_bytes, stream);
  }
  if (e == cudaSuccess && h->sums_bytes) e = cudaMemsetAsync(h->spoilt, 0, h->sums_bytes, stream);
  if (e == cudaSuccess) {
    const int64_t chunks = blocks * 64;
    layout_kernel<<<(unsigned)((chunks + 255) / 256), 256, 0, stream>>>(d->qweight, d->qweight_up, d->N, d->K, h->kb, chunks,
                                                                        h->w);
    scales_kernel<<<(h->strips * 16 + 255) / 256, 256, 0, stream>>>(d->scales, d->scales_up, d->N, h->strips * 16,
                                                                    h->w_scales);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);  // the caller may reuse its buffers
  if (e != cudaSuccess) {
    cudaGetLastError();
    spear_w8_destroy(h);
    return e == cudaErrorMemoryAllocation ? SPEAR_ERR_OOM : SPEAR_ERR_CUDA;
  }
  *out = h;
  return SPEAR_OK;
}

extern "C" spear_status_t spear_w8_destroy(spear_w8_t h) {
  if (!h) return SPEAR_OK;
  cudaError_t e = cudaSuccess;
  for (void* p : {static_cast<void*>(h->w), static_cast<void*>(h->w_scales), h->control, h->ws_owned ? h->ws : nullptr}) {
    const cudaError_t f = p ? cudaFree(p) : cudaSuccess;
    if (f != cudaSuccess) e = f;
  }
  delete h;
  return e == cudaSuccess ? SPEAR_OK : SPEAR_ERR_CUDA;
}

extern "C" spear_status_t spear_w8_forward(spear_w8_t h, const int8_t* x, int64_t ld_x, const float* x_scales, void* y,
                                           int64_t ld_y, spear_dtype_t type, int32_t M, cudaStream_t stream) {
  if (!h || M < 0 || M > h->max_tokens) return SPEAR_ERR_INVALID_ARG;
  if (type != SPEAR_BF16 && type != SPEAR_F16 && type != SPEAR_F32) return SPEAR_ERR_INVALID_ARG;
  if (M == 0) return SPEAR_OK;
  if (M == 1) ld_x = h->K, ld_y = h->N;  // of no account
  const unsigned size = type == SPEAR_F32 ? 4 : 2;
  if (!x || !x_scales || !y || !aligned(x, 16) || !aligned(x_scales, 4) || !aligned(y, size)) return SPEAR_ERR_INVALID_ARG;
  if (ld_x < h->K || ld_x % 16 != 0 || ld_y < h->N) return SPEAR_ERR_INVALID_ARG;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y), s0 = reinterpret_cast<uintptr_t>(x_scales);
  const uintptr_t x1 = x0 + (uintptr_t)(M - 1) * ld_x + h->K, y1 = y0 + ((uintptr_t)(M - 1) * ld_y + h->N) * size;
  if ((x0 < y1 && y0 < x1) || (s0 < y1 && y0 < s0 + (uintptr_t)M * 4)) return SPEAR_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEAR_ERR_CUDA;
  if (dev != h->device) return SPEAR_ERR_INVALID_ARG;
  const W8Call c = {x, ld_x, x_scales, y, ld_y, (int)type, M};
  return w8_many(h, M) ? w8_launch_prefill(h, c, stream) : w8_launch_decode(h, c, stream);
}

extern "C" spear_status_t spear_w8_forward_args(const spear_w8_forward_args_t* a) {
  if (!a) return SPEAR_ERR_INVALID_ARG;
  return spear_w8_forward(a->h, a->x, a->ld_x, a->x_scales, a->y, a->ld_y, (spear_dtype_t)a->type, a->M, a->stream);
}

extern "C" spear_status_t spear_w8_debug_set(spear_w8_t h, int64_t wait_ns, int32_t skip_arrive) {
  if (!h || wait_ns < 0) return SPEAR_ERR_INVALID_ARG;
  h->wait_ns = wait_ns ? (uint64_t)wait_ns : kW8WaitNs;
  h->skip_arrive = skip_arrive != 0;
  return SPEAR_OK;
}

extern "C" spear_status_t spear_w8_check(spear_w8_t h, cudaStream_t stream) {
  if (!h) return SPEAR_ERR_INVALID_ARG;
  unsigned status = 0;
  if (cudaMemcpyAsync(&status, h->status, sizeof(status), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return SPEAR_ERR_CUDA;
  if (status == 0) return SPEAR_OK;
  if (cudaMemsetAsync(h->control, 0, h->control_bytes, stream) != cudaSuccess ||
      (h->sums_bytes && cudaMemsetAsync(h->spoilt, 0, h->sums_bytes, stream) != cudaSuccess) ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return SPEAR_ERR_CUDA;
  return SPEAR_ERR_TIMEOUT;
}

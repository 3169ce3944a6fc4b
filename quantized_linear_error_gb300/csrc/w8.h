// Linears of 8-bit integer weights and activations: handle, kernel-side weight
// layout and launches (not part of the public ABI).
#pragma once
#include "internal.h"

// Kernel-side weights, built once by spear_w8_create and read by both kernels.
// Rows are grouped in strips of 16, pairs of strips, and tiles of 8 strips, zero
// rows past N. A strip and 64 input channels make a block of 1 KB; blocks are
// ordered [pair][k block][strip of the pair], so that few rows are one long run
// (8 strips of a k block side by side instead: 14.6 us against 12 for a token
// through 14336 x 4096) and 128 channels of a tile are four runs of 4 KB. A
// block is 64 chunks of 16 channels of one row: the chunk of row r
// and channels 16 t .. 16 t + 15 (t = 0 .. 3), with g = r % 8, stands at
// 16-byte place
//   (r / 8) * 32 + t * 8 + (g ^ 2 t),
// so that 8 lanes in a row hit all banks both when a warp reads as MMA
// fragments are laid out (lane 4 g + t takes rows g and g + 8) and when lanes
// are rows. Codes are kept with their top bit turned (code + 128 as a byte).
// A gated handle's strip holds 8 rows of the first weight, then the same 8 of
// the second, so that one lane (or lanes 8 apart) has both of an output.
constexpr int kW8Strip = 16, kW8K = 64, kW8Block = kW8Strip * kW8K, kW8Tile = 8;

__host__ __device__ inline int w8_place(int r, int t) { return (r >> 3) * 32 + t * 8 + ((r & 7) ^ (2 * t)); }
__host__ __device__ inline int64_t w8_block(int strip, int k, int kb) {
  return (((int64_t)(strip / 2) * kb + k) * 2 + strip % 2) * kW8Block;
}

struct spear_w8_s {
  int device, sm_count;
  int K, N;            // N outputs
  int gated, act;      // act: spear_act_t
  int strips, kb;      // strips of 16 weight rows (whole tiles), blocks of 64 channels (an even number)
  int max_tokens;
  uint8_t* w;          // strips * kb blocks
  float* w_scales;     // [strips * 16], in the strips' row order
  void* control;            // status and counters
  unsigned* status;
  unsigned* counters;       // [strips], of the few-token kernel's shared rows; zero between calls
  unsigned* gemm_counters;  // of the tensor-core kernel's shared tiles; zero between calls
  size_t control_bytes;
  uint64_t wait_ns;         // limit of the device-side waits
  int skip_arrive;          // one of them runs out (see spear_w8_debug_set)
  // The workspace: the caller's, which several handles may use in turn, or the handle's own.
  void* ws;
  int ws_owned;
  float* part;              // sums of the few-token kernel's shared rows
  unsigned* spoilt;         // set by a call that gave up and may have left sums that are not zero
  int* sums;                // of the tensor-core kernel's shared tiles, behind it; zero between calls
  size_t sums_bytes;        // of both
  uint8_t* x16;             // tokens in f16
};

struct W8Call {
  const int8_t* x;
  int64_t ld_x;
  const float* x_scales;
  void* y;
  int64_t ld_y;
  int type;  // spear_dtype_t of y
  int M;
};

// Whether M tokens go to the tensor-core kernel: more than 32, or more than 16 through many weights. From 17 tokens on
// the streaming kernel is at some 2.7 TB/s at best; the other one starts later and is faster then, whatever the count up
// to 32. 17 / 24 / 32 tokens, streaming against tensor cores, in us: 17 MB (4096 x 4096) 8.8 / 8.9 / 9.0 against
// 13.6 / 13.8 / 13.9, 25 MB (6144 x 4096) 13.9 / 14.0 / 14.4 against 13.6 / 13.5 / 13.6, 34 MB (4096 x 8192) 13.1 / 13.1 /
// 13.3 against 15.2 / 15.3 / 15.3, 45 MB (11008 x 4096) 20.4 / 20.5 / 21.4 against 17.2 / 16.9 / 17.0, 59 MB (14336 x 4096)
// 21.6 / 21.8 / 22.2 against 16.2 / 16.2 / 16.3.
inline bool w8_many(const spear_w8_s* h, int M) { return M > 32 || (M > 16 && (int64_t)h->strips * h->kb > 36 * 1024); }

constexpr uint64_t kW8WaitNs = 100000000ull;  // limit of a device-side wait, unless set otherwise

constexpr size_t kW8SumsAt = 128;               // bytes from `spoilt` to the sums

constexpr int kRowsMaxWidth = 32768;       // 1024 threads x 32 elements in registers

namespace spear {
spear_status_t sm_count_of_current(int* sms);
size_t w8_decode_workspace(const spear_w8_s* h);
size_t w8_prefill_workspace(const spear_w8_s* h);
size_t w8_prefill_counters(const spear_w8_s* h);
size_t w8_prefill_sums(const spear_w8_s* h);
spear_status_t w8_launch_prefill(const spear_w8_s* h, const W8Call& c, cudaStream_t stream);
spear_status_t w8_launch_decode(const spear_w8_s* h, const W8Call& c, cudaStream_t stream);
}

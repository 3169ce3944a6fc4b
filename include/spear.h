/*
 * spear.h -- C ABI of the GB300 (sm_103a) W4 + input-adaptive error-compensator
 * linear layer.
 *
 * The layer ("SPEAR: A System for Post-Quantization Error-Adaptive Recovery",
 * section 2.1A, Input-Adaptive Error Compensators, "Mechanism") applies to each
 * token x the effective weight
 *
 *     W_q + alpha * B * diag(gamma(A x)) * A,
 *
 * i.e. y = W_q x + alpha * B (gamma(z) (.) z) with z = A x. W_q is a 4-bit
 * weight with bf16 scales and integer zero points per group of 128 input
 * channels or per output channel (section 1 and section 3.1 use 4-bit weights,
 * per-channel being the hard case); A is rank x K, B is N x rank, gamma is the
 * elementwise sigmoid, the constant one (which gives the static low-rank
 * correction W_q + alpha B A that section 1 contrasts with), or the
 * bottleneck MLP that section 2.1A names for gamma. Phase-aware
 * dispatch (section 2.2A) is exposed as two entry points: a fused single-kernel
 * decode path for M <= 32 tokens and a tensor-core prefill path for larger M.
 *
 * Conventions for every call:
 *  - Device pointers are plain CUDA device addresses on the current device;
 *    host pointers are ordinary (preferably pinned) host memory. No call takes
 *    ownership of a caller's buffer.
 *  - bf16 tensors are row-major and contiguous; x, y and every weight buffer
 *    must be 16-byte aligned.
 *  - Argument errors are reported synchronously and leave nothing enqueued.
 *  - Forward calls only enqueue work on `stream` (no allocation, no
 *    synchronisation). Errors detected on the device (a bounded wait that
 *    timed out) are latched in the handle and reported by spear_linear_check.
 *  - A handle is not safe for concurrent forwards (its workspace is shared);
 *    distinct handles are independent.
 */
#ifndef SPEAR_H_
#define SPEAR_H_

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct spear_linear_s* spear_linear_t;

typedef enum {
  SPEAR_OK = 0,
  SPEAR_ERR_INVALID_ARG = 1,   /* null pointer, bad shape, M outside the entry point's range */
  SPEAR_ERR_UNSUPPORTED = 2,   /* valid but outside what the kernels implement (see create) */
  SPEAR_ERR_OOM = 3,           /* device allocation failed in create */
  SPEAR_ERR_CUDA = 4,          /* a CUDA runtime call or kernel launch failed */
  SPEAR_ERR_TIMEOUT = 5        /* a bounded device-side wait gave up (reported by check) */
} spear_status_t;

typedef enum {
  SPEAR_GATE_SIGMOID = 0,      /* gamma(z) = 1 / (1 + exp(-z)), so gamma(z) * z = SiLU(z) */
  SPEAR_GATE_ONE = 1,          /* gamma = 1: static correction W_q + alpha B A */
  SPEAR_GATE_MLP = 2           /* bottleneck MLP ("SPEAR", section 2.1A, "Mechanism"), per token:
                                  gamma(z) = sigmoid(W2 relu(W1 z)), W1 (h x rank), W2 (rank x h);
                                  relu as the hidden activation is this library's reading */
} spear_gate_t;

typedef struct {
  int32_t K;                   /* input features; multiple of 128 */
  int32_t N;                   /* output features; multiple of 8 */
  int32_t group_size;          /* 128, or 0 for one group per output channel (G = K) */
  const uint8_t* qweight;      /* device, uint8 [N][K/2]: byte j of row n holds k = 2j in its
                                  low nibble and k = 2j + 1 in its high nibble, codes 0..15 */
  const void* scales;          /* device, bf16 [N][K/G] */
  const uint8_t* zeros;        /* device, uint8 [N][K/G], values 0..15; NULL means z = 8 */
  int32_t rank;                /* EC rank r: 0 (no compensator) or a multiple of 16, <= 256 */
  const void* A;               /* device, bf16 [rank][K] (ignored when rank == 0) */
  const void* B;               /* device, bf16 [N][rank] (ignored when rank == 0) */
  float alpha;                 /* compensator strength */
  spear_gate_t gate;
  int32_t max_tokens;          /* largest M any forward on this handle will use (>= 1) */
  /* SPEAR_GATE_MLP only (ignored otherwise; zero them for the other gates): */
  int32_t gate_hidden;         /* h, 1 <= h <= 64 */
  const void* gate_w1;         /* device, bf16 [h][rank], 16-byte aligned */
  const void* gate_w2;         /* device, bf16 [rank][h], 16-byte aligned */
} spear_linear_desc_t;

/* Build a handle from user-layout weights ("SPEAR", section 2.1A: the W_q of the
 * effective weight and the compensator's A, B, alpha, gamma).
 * Copies and re-lays-out every weight into handle-owned device memory on
 * `stream`, then synchronises `stream`, so the caller may free or reuse its
 * buffers as soon as this returns. On success *out holds the handle.
 * Errors: INVALID_ARG (null desc/out/pointers, K % 128, N % 8, bad group size,
 * rank not a multiple of 16 or > 256, max_tokens < 1; for SPEAR_GATE_MLP:
 * rank == 0, gate_hidden outside 1..64, null or unaligned gate weights),
 * UNSUPPORTED (shape outside the kernels' limits: N > 16 * 16 * SM count for
 * the decode path, or a decode grid that cannot be resident on the device all
 * at once, which its grid-wide compensator dependency needs), OOM, CUDA. On
 * error *out is left NULL and nothing is leaked.
 * Co-residency: the decode kernel runs at most one CTA per SM and its CTAs
 * wait for each other (bounded). Kernels of other streams or processes that
 * hold SMs while a decode call starts can delay some of its CTAs; if that
 * outlasts the wait limit, the call leaves the compensator out and latches
 * TIMEOUT, which spear_linear_check reports. */
spear_status_t spear_linear_create(const spear_linear_desc_t* desc, cudaStream_t stream,
                                   spear_linear_t* out);

/* Build ONE handle for several linears that read the same input x, such as
 * the q, k and v projections of an attention block or the gate and up
 * projections of an MLP (the paper has no counterpart; this is how serving
 * engines fuse such projections). Each member keeps its own weights, zero
 * points, compensator (A_i, B_i, alpha_i) and result:
 *   y[:, row_i : row_i + N_i] = W_i x + alpha_i B_i (gamma(A_i x) (.) A_i x),
 * row_i = N_0 + ... + N_{i-1}, so y is bf16 [M][N_0 + ... + N_{n-1}] and
 * every forward of the handle computes all members in one call (one launch
 * on the decode path: the stacked projection [A_0; ...; A_{n-1}] x and its
 * gate run once for all members, each output tile then applies its own
 * member's B_i and alpha_i).
 *   descs: n descriptors, 1 <= n <= 8 (n == 1 is spear_linear_create). All
 *   members must have the same K, group_size, rank and gate, N_i a multiple
 *   of 16, and n * rank <= 256; SPEAR_GATE_MLP is not supported here
 *   (UNSUPPORTED). max_tokens of the handle is the largest of the members'.
 * The members' buffers are copied (through temporary device buffers that
 * create frees before returning); errors as for spear_linear_create. */
spear_status_t spear_linear_create_grouped(const spear_linear_desc_t* descs, int32_t n, cudaStream_t stream,
                                           spear_linear_t* out);

/* Decode-phase forward ("SPEAR", section 2.2A: memory-bound, small M; the whole
 * layer, compensator included, runs as one kernel).
 *   x: device bf16 [M][K]; y: device bf16 [M][N] (must not overlap x).
 * 1 <= M <= min(32, max_tokens); M == 0 is a no-op returning OK.
 * y = bf16_RNE(W_q x + alpha B (gamma(Ax) (.) Ax)) with fp32 accumulation. */
spear_status_t spear_linear_forward_decode(spear_linear_t h, const void* x, void* y, int32_t M,
                                           cudaStream_t stream);

/* Prefill-phase forward ("SPEAR", section 2.2A: compute-bound, M > 1): the
 * main contraction runs on tcgen05 tensor cores with in-kernel INT4
 * dequantisation; the compensator's down-projection and gate run in a small
 * pre-kernel and its up-projection is folded into the same accumulator.
 *   x: device bf16 [M][K]; y: device bf16 [M][N]; 1 <= M <= max_tokens
 * (M == 0 is a no-op). Correct for every M; tuned for M >= 256. */
spear_status_t spear_linear_forward_prefill(spear_linear_t h, const void* x, void* y, int32_t M,
                                            cudaStream_t stream);

/* Prefill with the compensator on a concurrent stream ("SPEAR", section 2.2A:
 * in the prefill phase the compensator runs as a separate kernel overlapped
 * with the low-bit GEMM). The same y as spear_linear_forward_prefill, computed
 * as three launches: the compensator pre-kernel (u' = bf16(alpha gamma(Ax) (.)
 * Ax)) on ec_stream, forked from `stream` by an event; the main contraction
 * W x on `stream` into an fp32 buffer of the handle; after an event join, a
 * K-tail launch that adds alpha B u' to it and rounds to bf16 once. Both
 * streams are left joined (ec_stream's work precedes `stream`'s later work),
 * so the call can be captured into one CUDA graph. Requires
 * spear_linear_enable_concurrent_ec on handles with a compensator (a handle
 * without one takes the plain prefill path); ec_stream != stream.
 * Errors: INVALID_ARG, CUDA. */
spear_status_t spear_linear_forward_prefill_concurrent(spear_linear_t h, const void* x, void* y, int32_t M,
                                                       cudaStream_t stream, cudaStream_t ec_stream);

/* Allocates what spear_linear_forward_prefill_concurrent needs: an fp32
 * buffer of max_tokens x N and two events (once; later calls return OK). This
 * is the only allocation outside create. Errors: INVALID_ARG, OOM, CUDA. */
spear_status_t spear_linear_enable_concurrent_ec(spear_linear_t h);

/* Phase dispatch ("SPEAR", section 2.2A): decode path for M <= 32, prefill otherwise. */
spear_status_t spear_linear_forward(spear_linear_t h, const void* x, void* y, int32_t M,
                                    cudaStream_t stream);

/* End-to-end forward on HOST buffers: copies x_host (bf16 [M][K]) to a
 * handle-owned device buffer, runs spear_linear_forward, copies the result
 * into y_host (bf16 [M][N]) and synchronises `stream`. Pinned host memory gives
 * asynchronous copies. 1 <= M <= max_tokens. */
spear_status_t spear_linear_forward_host(spear_linear_t h, const void* x_host, void* y_host,
                                         int32_t M, cudaStream_t stream);

/* End-to-end forward of a batch of calls on HOST buffers with one
 * synchronisation: call i copies x_host[i] (bf16 [Ms[i]][K of hs[i]]) into
 * hs[i]'s staging buffer, runs spear_linear_forward on it and copies the
 * result into y_host[i] (bf16 [Ms[i]][N of hs[i]]); the call returns once
 * every result is in host memory. The forwards run in order on `stream`.
 * The copies run on two copy streams of hs[0], after the work already on
 * `stream`, and overlap the forwards: a call's input copy waits only for the
 * previous forward on the same handle (which has read its staging buffer),
 * its forward for that copy and for the previous result of the handle to be
 * copied out. A handle may appear several times. The copy streams and a
 * handle's four events are made on its first batch and destroyed with it.
 * Every argument is checked before anything is enqueued: INVALID_ARG for a
 * null array or handle, Ms[i] outside 0 .. max_tokens of hs[i], or null
 * buffers with Ms[i] > 0; CUDA if a stream or event cannot be made. Pinned
 * host memory gives asynchronous copies. */
spear_status_t spear_linear_forward_host_batch(const spear_linear_t* hs, const void* const* x_host,
                                               void* const* y_host, const int32_t* Ms, int32_t n,
                                               cudaStream_t stream);

/* Free every device allocation of the handle. cudaFree, which this calls,
 * waits for work already queued on the device, so forwards still in flight
 * finish first; the handle must not be used (or enqueued) afterwards. NULL is
 * accepted. */
spear_status_t spear_linear_destroy(spear_linear_t h);

/* Test surface: write the dequantised weight bf16_RNE((q - z) * s) as bf16
 * [N][K] (device) by unpacking the kernel-side layout of `path`
 * (0 = decode layout, 1 = prefill layout) with the kernels' own unpack code. */
spear_status_t spear_linear_dequantize(spear_linear_t h, int32_t path, void* w_out,
                                       cudaStream_t stream);

/* Synchronise `stream` and report the handle's device status word: OK, or
 * TIMEOUT if a bounded device-side wait gave up since the last check. A
 * TIMEOUT clears the status and resets the handle's workspace so it is usable
 * again. */
spear_status_t spear_linear_check(spear_linear_t h, cudaStream_t stream);

/* Test surface for the bounded waits: wait_ns sets the device-side wait limit
 * (0 restores the default of 100 ms); skip_arrive != 0 makes CTAs skip the
 * arrival another CTA waits for, so that the wait must run out:
 *  - decode: the "compensator projection done" arrival (the kernel then leaves
 *    the compensator out of y and latches TIMEOUT);
 *  - prefill, when the main kernel's stream-K schedule splits a tile over
 *    several CTAs (a handle sized for more than 32 tokens): the "partial tile
 *    stored" flag of the CTAs that run a tile's later K blocks (the tile's
 *    owner then gives up, writes nothing for its tile and latches TIMEOUT).
 * The prefill pre-kernel -> main kernel dependency is a stream (programmatic
 * launch) dependency that the hardware resolves; it has no arrival to skip. */
spear_status_t spear_linear_debug_set(spear_linear_t h, int64_t wait_ns, int32_t skip_arrive);

/* Test surface: the launch plan spear_linear_forward_decode uses for a handle
 * of this shape ("SPEAR", section 2.2A: the decode phase as one fused kernel),
 * computed by the same host code as the launch, with no device work.
 *   N, K: output and input width (as spear_linear_create accepts them);
 *   rank_b, n_members: each member's compensator rank and the member count
 *     (1 for spear_linear_create, 2..8 for a grouped handle with N split
 *     evenly); group_size: 128 or 0 (per output channel);
 *   gate_hidden: the MLP gate's hidden width (16, 32, 48 or 64), else 0;
 *   1 <= M <= 32; sm_count: SMs of the device.
 * info (13 int32 entries, caller-owned): grid, P (16-row tiles per CTA), NW
 * (consumer warps), T (tiles per warp), MT (8-token tiles), KW (warps along
 * K), KC (channels per stage), NS (stages), stage_bytes, smem (dynamic
 * shared memory), n_stages (stages over K), threads, bytes_x (x box bytes).
 * Errors: INVALID_ARG (bad shape or null info), UNSUPPORTED (as create or the
 * launch would report it). */
spear_status_t spear_decode_schedule(int32_t N, int32_t K, int32_t rank_b, int32_t n_members, int32_t group_size,
                                     int32_t gate_hidden, int32_t M, int32_t sm_count, int32_t* info);

/* Test surface: the launch plan spear_linear_forward_prefill uses for a layer
 * of this shape ("SPEAR", section 3.3: the compensator's projection fused
 * ahead of the weight contraction, its output GEMM as the K-tail), computed
 * by the same host code as the launch, with no device work and no GPU.
 *   N, K, rank: the layer (K a multiple of 64, 0 <= rank <= 256);
 *   gate_hidden: the hidden width of SPEAR_GATE_MLP (16, 32, 48 or 64), 0 for
 *     the elementwise gates; M >= 1 tokens;
 *   sm_count: SMs of the device the handle lives on;
 *   with_workspace: nonzero when the handle was created with max_tokens > 32
 *     (it then holds the stream-K partial-tile workspace).
 * info (14 int32 entries, caller-owned): mode (0: the projection runs in
 * the main kernel's prologue or rank = 0; 3: a split-K pre-kernel first),
 * G (main-kernel CTAs), TN (tokens per tile), kpt (units per tile), tail
 * (K-tail units per tile, ceil(rank / 64)), units (tiles x kpt), pro_items
 * (prologue items, one per 128 tokens; 0 in mode 3), pro_d (units each item
 * weighs in the split), NS (pipeline stages), stage_bytes, smem (dynamic
 * shared memory per CTA), pre_ctas (the pre-kernel's CTAs, mode 3),
 * tmem_a (first TMEM column of the dequantised-W slots), max_contrib (the
 * most partial tiles any owner adds).
 * starts (optional, caller-owned, starts_cap >= G + 1 entries): CTA c runs
 * units [starts[c], starts[c + 1]); starts[G] = units.
 * Errors: INVALID_ARG (bad shape, null info, starts_cap too small),
 * UNSUPPORTED (more than 2^31 units). */
spear_status_t spear_prefill_schedule(int32_t N, int32_t K, int32_t rank, int32_t gate_hidden, int32_t M,
                                      int32_t sm_count, int32_t with_workspace, int32_t* info, uint32_t* starts,
                                      int32_t starts_cap);

/* Decode forward that allocates nothing (the paper has no counterpart; this is
 * a deployment convenience). For callers that cannot call cudaMalloc at all,
 * for instance a process whose device memory is entirely reserved up front by
 * another allocator, or a serving loop in which a device allocation (which may
 * synchronise the device) is not allowed: such callers cannot create a handle,
 * so this call takes everything from the caller.
 *   desc: the same descriptor spear_linear_create takes (device pointers to
 *         the user-layout q, scales, zeros, A, B; max_tokens is ignored);
 *         qweight and A 16-byte aligned;
 *   x: device bf16 [M][K], 16-byte aligned; y: device bf16 [M][N];
 *   1 <= M <= 32 (0 is a no-op).
 * Result: y = bf16_RNE(W_q x + alpha B (gamma(Ax) (.) Ax)), fp32 accumulation,
 * as spear_linear_forward_decode computes (summation order differs).
 * SPEAR_GATE_MLP is not supported here (SPEAR_ERR_UNSUPPORTED).
 * Scratch: the compensator projection z lives in one static device array of
 * the library (32,768 bytes, held on every GPU that loads the library until
 * the process exits); it bounds rank <= 256 and M <= 32, and larger values
 * return SPEAR_ERR_INVALID_ARG. The first call on a device looks the array's
 * address up (cudaGetSymbolAddress, with that device current) and caches it;
 * make that first call before any stream capture. Each call enqueues two
 * kernels on `stream` (z = A x into the array, then the output rows), ordered
 * by the stream alone: no wait across blocks, no allocation, no
 * synchronisation. Every z entry a call reads was written by the same call,
 * so nothing needs clearing between calls. All calls share the array, so
 * calls that overlap on the GPU (different streams, or several host threads)
 * race with each other: serialise them. Slower than the handle-based decode
 * path (it reads the unpacked user layout on CUDA cores). */
spear_status_t spear_linear_forward_decode_noalloc(const spear_linear_desc_t* desc, const void* x, void* y,
                                                   int32_t M, cudaStream_t stream);

/* Round-to-nearest 4-bit quantiser (offline; the "RTN" backend of "SPEAR",
 * section 3.1, which the paper does not spell out: the usual asymmetric
 * min/max form). Per group of G input channels (G = 128, or K for
 * group_size 0) of each output row:
 *   lo = min(0, min w), hi = max(0, max w), range = max(hi - lo, 1e-8),
 *   s = bf16_RNE(range / 15), z = clamp(rint(-lo / s), 0, 15),
 *   q = clamp(rint(w / s) + z, 0, 15),
 * all in fp32 with IEEE division and round half to even.
 *   w: device fp32 [N][K], 16-byte aligned; outputs in the layout
 *   spear_linear_desc_t takes: qweight device uint8 [N][K/2] (2-byte
 *   aligned), scales device bf16 [N][K/G], zeros device uint8 [N][K/G].
 * K must be a multiple of 128. Enqueues one kernel on `stream`.
 * Errors: INVALID_ARG (null or misaligned pointers, bad shape or group size),
 * UNSUPPORTED (grid too large), CUDA. */
spear_status_t spear_quantize_rtn(const float* w, int32_t N, int32_t K, int32_t group_size, uint8_t* qweight,
                                  void* scales, uint8_t* zeros, cudaStream_t stream);

/* SLO-constrained, compensator-aware chunk scheduler ("SPEAR", section 2.2C:
 * a latency-aware scheduler driven by precomputed kernel-latency lookup tables
 * picks the largest prefill chunk that meets an inter-token-latency target,
 * adapting to the compensator density). Host only; no device work.
 * The table holds measured times of one whole serving step: ms[i * n_m + j]
 * for density densities[i] (share of layers with a compensator, strictly
 * ascending in [0, 1]) and tokens[j] tokens in the step (strictly ascending,
 * >= 1). Prediction is piecewise linear in the token count (extrapolated
 * linearly past the table's ends) and linear in the density between rows
 * (clamped to the first and last rows). */
typedef struct spear_sched_s* spear_sched_t;

/* Copies the table. Errors: INVALID_ARG (null pointers, empty or unsorted
 * axes, densities outside [0, 1], negative or NaN times), OOM. */
spear_status_t spear_sched_create(const double* densities, int32_t n_d, const int32_t* tokens, int32_t n_m,
                                  const double* ms, spear_sched_t* out);

/* Predicted step time (ms) for M tokens at the given density; -1 for a null
 * handle or M < 0. */
double spear_sched_predict(spear_sched_t s, int32_t M, double density);

/* *chunk_out = the largest candidate chunk c (candidates in any order, >= 0)
 * with predict(n_decode + c, density) <= itl_ms, or 0 if none fits. */
spear_status_t spear_sched_pick_chunk(spear_sched_t s, int32_t n_decode, double density, double itl_ms,
                                      const int32_t* candidates, int32_t n_c, int32_t* chunk_out);

/* Frees the scheduler; NULL is accepted. */
spear_status_t spear_sched_destroy(spear_sched_t s);

/* ------------------------------------------------------------------------
 * Key/value cache in 4 bits and the attention that reads it: what stands
 * between the q/k/v linears and the o linear of a decoder block (the paper's
 * serving engine has them as given; the formats and kernels are this
 * library's).
 *
 * Pool: device uint8 [n_pages][n_kv_heads][page_size / 16][16 * (D + 8)],
 * 16-byte aligned, owned by the caller. A block of 16 tokens of one head holds
 * K codes [16][D / 2], V codes [16][D / 2], K parameters [16][2] and V
 * parameters [16][2]; byte j of a row of codes holds element 2j in its low
 * nibble and 2j + 1 in its high one, a parameter pair is bf16 (scale, offset),
 * and an element stands for code * scale + offset. Slot number
 * page * page_size + i names token i of a page.
 *
 * A row x of D fp32 values is quantised with one scale and offset:
 *   scale = bf16_RNE((max x - min x) * fl32(1/15)), 0 if that is below 2^-126,
 *   offset = bf16_RNE(min x),  inv = scale > 0 ? fl32(1 / scale) : 0,
 *   code = clamp(rint((x - offset) * inv), 0, 15),
 * each operation in fp32, round to nearest even. A row with an element that
 * is not finite, or whose range is above 2^120, is held with scale = offset =
 * NaN.
 *
 * Rotation (rope_dim R > 0): element pairs (i, i + R / 2), or (2i, 2i + 1) if
 * rope_interleaved, i < R / 2, of the row at position p become
 *   x1 * c - x2 * s  and  x2 * c + x1 * s,  c = table[p][i], s = table[p][R / 2 + i],
 * products and sums each rounded to fp32; elements from R on stay as they are.
 *
 * Slots, positions, page numbers and lengths are device data that the host
 * cannot check. The kernels check them: what is out of range is neither read
 * nor written, and latches INVALID_ARG for spear_kv_check (an append skips the
 * token; an attention call leaves that sequence's results unspecified).
 * A handle's calls share its workspace: order them on one stream, or by
 * events; distinct handles are independent and may share a pool.
 * ---------------------------------------------------------------------- */
typedef struct spear_kv_s* spear_kv_t;

typedef struct {
  int32_t n_heads;             /* query heads (<= 4096), a multiple of n_kv_heads; head h reads
                                  key/value head h / (n_heads / n_kv_heads) */
  int32_t n_kv_heads;          /* n_heads / n_kv_heads <= 32 */
  int32_t head_dim;            /* D: 64 or 128 */
  int32_t page_size;           /* tokens per page, a multiple of 16, <= 65536 */
  int32_t n_pages;             /* pages in the pool (>= 1) */
  void* pool;
  int32_t rope_dim;            /* R: 0 (no rotation) or a multiple of 16, <= D */
  int32_t rope_interleaved;
  int32_t n_positions;         /* rows of rope_table (ignored when rope_dim == 0) */
  const float* rope_table;     /* device, fp32 [n_positions][R], 16-byte aligned, kept by the
                                  caller while the handle lives: R / 2 cosines, R / 2 sines */
} spear_kv_desc_t;

/* Build a handle over the caller's pool. Allocates the attention's workspace
 * (partial results of work split over a long cache; its size depends on the
 * device and the head counts only, not on lengths), clears it on `stream` and
 * synchronises `stream`, so that calls may follow on any; the pool is not
 * touched. Errors: INVALID_ARG (null or misaligned pointers, values outside the
 * ranges above), OOM, CUDA; *out is NULL then. */
spear_status_t spear_kv_create(const spear_kv_desc_t* desc, cudaStream_t stream, spear_kv_t* out);

/* Rotate the queries and keys of T tokens and put their keys and values into
 * the cache, in one launch.
 *   q: device bf16 [T][n_heads][D], or NULL (no queries to rotate);
 *   k, v: device bf16 [T][n_kv_heads][D];
 *   ld_q, ld_k, ld_v, ld_q_out: elements from one token to the next, so that
 *     slices of a fused projection's output can be passed as they are; heads
 *     are contiguous. Multiples of 8, at least the row's length;
 *   positions: device int64 [T] (ignored when rope_dim == 0);
 *   slots: device int64 [T]; -1 leaves the token's key and value uncached;
 *   q_out: device bf16 [T][n_heads][D], rotated queries: q itself, or it shares
 *     no element with q, k and v (memory of its own, or, with the same ld, other
 *     columns of the same rows).
 * Two tokens of one call must not have the same slot. T == 0 is a no-op.
 * Errors: INVALID_ARG, CUDA. */
spear_status_t spear_kv_append(spear_kv_t h, const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                               int64_t ld_v, const int64_t* positions, const int64_t* slots, int32_t T, void* q_out,
                               int64_t ld_q_out, cudaStream_t stream);

/* The values that T slots hold, bf16_RNE(code * scale + offset), into k_out
 * and v_out: device bf16 [T][n_kv_heads][D], contiguous, apart from each other.
 * Slot -1 gives zeros.
 * Errors: INVALID_ARG, CUDA. */
spear_status_t spear_kv_read(spear_kv_t h, const int64_t* slots, int32_t T, void* k_out, void* v_out,
                             cudaStream_t stream);

/* Causal attention of n_seqs sequences over the cache. Sequence b has the
 * query rows q_starts[b] <= t < q_starts[b + 1] and L = kv_lens[b] cached
 * tokens, its new ones included (append them first): key j is token
 * j % page_size of page page_table[b][j / page_size]. Row i of its n rows
 * stands at P = L - n + i and sees the keys j <= P, j >= 0, with window > 0
 * only j > P - window:
 *   out = bf16_RNE(sum_j softmax_j(scale * q . k_j) v_j),
 * zeros for a row that sees no key, NaN for a row of q that is not finite.
 * Scores, softmax statistics and sums are fp32. The weights are rounded to f16
 * (11 bits, 8 at 2^-22 of the largest; below 2^-31 they count in the sum alone),
 * or bf16 for 32 keys at a time whose values' scales lie far apart. For chunks
 * so are the cached keys and values, code * scale + offset; for few rows
 * differences of neighbours in q are rounded to f16. Where q . k * scale and the
 * result are ordinary fp32 numbers, elements of q up to 2^118 / max(1, scale) and
 * cached elements up to 2^60 in size are served; larger ones may give infinities
 * or NaN.
 *   q, out: device bf16 [T][n_heads][D], ld_q, ld_out as for spear_kv_append;
 *     out is q itself or shares no element with it: memory of its own, or (with
 *     the same ld) other columns of the same rows;
 *   page_table: device int32 [n_seqs][ld_pt]; entries of pages that no row sees,
 *     past a sequence's end or wholly before its window, may be anything;
 *   kv_lens: device int32 [n_seqs], at most 2^30;
 *   q_starts: device int32 [n_seqs + 1], ascending, within 0..T;
 *   max_q: the largest number of query rows of a sequence (>= 1);
 *   T * (n_heads / n_kv_heads) < 2^27; a window above 2^30 hides nothing.
 * Sequences whose rows of one key/value head, (n_heads / n_kv_heads) x query
 * rows, fit a few warp-MMA tiles run in a kernel that streams the cache once
 * (single tokens, drafts to verify), longer ones in a tensor-core kernel. A call
 * with longer ones runs both, and drafts then count as long unless they fit the
 * tiles of single tokens (8, 16 or 32 rows). The call only enqueues, so it can be
 * captured in a graph; lengths are read on the device when it runs.
 * Errors: INVALID_ARG, CUDA. */
spear_status_t spear_kv_attention(spear_kv_t h, const void* q, int64_t ld_q, void* out, int64_t ld_out,
                                  const int32_t* page_table, int32_t ld_pt, const int32_t* kv_lens,
                                  const int32_t* q_starts, int32_t n_seqs, int32_t T, int32_t max_q, float scale,
                                  int32_t window, cudaStream_t stream);

/* Synchronise `stream` and report the handle's device status: OK, or
 * INVALID_ARG if a call since the last check met an index out of range, or
 * TIMEOUT if a bounded device-side wait gave up. A status other than OK is
 * cleared and the workspace reset. */
spear_status_t spear_kv_check(spear_kv_t h, cudaStream_t stream);

/* Free the handle's device memory (waits for queued work, as
 * spear_linear_destroy does); the pool stays the caller's. NULL is accepted. */
spear_status_t spear_kv_destroy(spear_kv_t h);

/* ------------------------------------------------------------------------
 * 8-bit integers: rows in 8 bits, the norm that writes them, and linears of
 * 8-bit weights and activations, beside the 4-bit ones (the paper compares
 * with such layers; the forms and kernels here are this library's).
 *
 * A row v of fp32 values in 8 bits is K codes (int8) and one scale (fp32):
 *   a = max |v|,  scale = fl32(a / 127),
 *   code = clamp(rint(v * fl32(127 / a)), -127, 127),
 * each operation in fp32, round to nearest even; an element stands for
 * code * scale. A row with a below 2^-100 is held as zeros (scale 0); one with
 * an element that is not finite has scale NaN and codes 0, so that it reads as
 * NaN.
 *
 * Matrices are rows of K (or N) contiguous elements, ld elements from one row
 * to the next (ld >= K; of no account for a single row), aligned to their
 * elements. Rows whose base and ld are multiples of 16 bytes (8 for codes) are
 * moved in wide accesses. Where rows that the norm or the quantiser reads start
 * or end elsewhere, it reads the whole aligned 16-byte words that hold them: up
 * to 15 bytes before and behind a row, which are in the same words as the row's
 * own and which nothing depends on. M == 0 is a no-op. Calls only enqueue on
 * `stream`.
 * ---------------------------------------------------------------------- */
typedef enum { SPEAR_BF16 = 0, SPEAR_F16 = 1, SPEAR_F32 = 2 } spear_dtype_t;

/* Root-mean-square norm of M rows, with the residual's addition before it and
 * 8-bit rows as its result, in one launch:
 *   h = x + residual (fp32; x alone if residual is NULL), residual_out = round(h),
 *   v = h / sqrt(mean(h^2) + eps) * weight,
 *   y = round(v) (x's type), and / or q, scales = v in 8 bits.
 * Statistics and sums are fp32, of the unrounded h. The codes are taken from
 * h * weight, whose row v is up to a positive factor, which goes into the scale
 * alone; where max |h * weight| is below 2^-110 the row counts as zeros. h * weight
 * is formed in fp32, of rows with a sum of squares beyond 2^120 after h has been
 * scaled by 2^-96: elements of the weight beyond 2^66 in size, or of such rows
 * below 2^-60, may leave its range.
 *   x: device, `type`, [M][ld_x]; weight: device [K], `type` or fp32;
 *   residual, residual_out: device, `type` or fp32 (residual_type), both or
 *     neither; the same rows (residual_out == residual) or apart;
 *   y: or NULL; q: int8 [M][ld_q], with scales fp32 [M], or NULL; one of both.
 * y and residual_out may be x's own rows if the element types are the same;
 * else results share no element with each other or with what is read. K up to
 * 32768 (as for the quantiser: rows for wider linears are the caller's to
 * quantise). eps >= 0, finite; with eps 0 a row of zeros gives NaN.
 * Rows with an element that is not finite give NaN (in residual_out only there).
 * Errors: INVALID_ARG, UNSUPPORTED (K), CUDA. */
spear_status_t spear_rms_norm(const void* x, int64_t ld_x, spear_dtype_t type, const void* residual,
                              int64_t ld_residual, void* residual_out, int64_t ld_residual_out,
                              spear_dtype_t residual_type, const void* weight, spear_dtype_t weight_type, float eps,
                              int32_t M, int32_t K, void* y, int64_t ld_y, int8_t* q, int64_t ld_q, float* scales,
                              cudaStream_t stream);

/* M rows in 8 bits, bit for bit as defined above: activations each step (a scale
 * a token), weights once (a scale an output channel). K up to 32768.
 *   x: device, `type`; q: int8 [M][ld_q]; scales: fp32 [M]; all apart.
 * Errors: INVALID_ARG, UNSUPPORTED (K), CUDA. */
spear_status_t spear_quantize_rows(const void* x, int64_t ld_x, spear_dtype_t type, int32_t M, int32_t K, int8_t* q,
                                   int64_t ld_q, float* scales, cudaStream_t stream);

/* What rows in 8 bits stand for: out = round(code * scale) as `type`.
 * Errors: INVALID_ARG, UNSUPPORTED (more than 2^40 groups of 16 elements, the
 * last of a row with fewer), CUDA. */
spear_status_t spear_dequantize_rows(const int8_t* q, int64_t ld_q, const float* scales, int32_t M, int32_t K, void* out,
                                     int64_t ld_out, spear_dtype_t type, cudaStream_t stream);

typedef struct spear_w8_s* spear_w8_t;

typedef enum {
  SPEAR_ACT_SILU = 0,          /* act(g) = g / (1 + exp(-g)) */
  SPEAR_ACT_GELU = 1           /* act(g) = g / (1 + exp(-2 z)), z = sqrt(2 / pi) (g + 0.044715 g^3): the tanh form */
} spear_act_t;

typedef struct {
  int32_t K;                   /* input features, a multiple of 16 */
  int32_t N;                   /* output features, >= 1 */
  const int8_t* qweight;       /* device, int8 [N][K], 16-byte aligned */
  const float* scales;         /* device, fp32 [N]: one scale an output channel */
  const int8_t* qweight_up;    /* second projection of a gated pair, or NULL; as qweight */
  const float* scales_up;      /* its scales, or NULL */
  spear_act_t activation;      /* of a gated pair (ignored otherwise) */
  int32_t max_tokens;          /* largest M a forward on this handle will use (>= 1) */
  void* workspace;             /* device, 128-byte aligned, or NULL: the handle allocates its own. A workspace serves any
                                  number of handles whose calls follow one another (a model's layers), is the library's
                                  alone while they live, and is larger than the weights of small layers: 1.2 MB, or where
                                  calls may go to the tensor cores (more than 32 tokens, 17 through more than 36 MB of
                                  weights) 16.2 MB + K (512 + 2.25 max_tokens) bytes, K rounded up to 128 */
  int64_t workspace_bytes;     /* at least what spear_w8_workspace says (ignored without a workspace) */
} spear_w8_desc_t;

/* Bytes of the workspace that a handle of this descriptor needs on the current device (its workspace fields are of no
 * account). Errors: as for spear_w8_create. */
spear_status_t spear_w8_workspace(const spear_w8_desc_t* desc, int64_t* bytes);

/* Build a handle from 8-bit weights: the weights are copied and laid out once,
 * in one layout that serves every number of tokens, part of the workspace is
 * cleared, and `stream` is synchronised, so that the caller may free its
 * buffers. No call that uses the same workspace may be running meanwhile.
 * Errors: INVALID_ARG (null or misaligned pointers, values outside the ranges
 * above), UNSUPPORTED (K > 2^20, N > 2^22, max_tokens > 2^20), OOM, CUDA; *out
 * is NULL then. */
spear_status_t spear_w8_create(const spear_w8_desc_t* desc, cudaStream_t stream, spear_w8_t* out);

/* Product of 8-bit integers with scales for each token and channel:
 *   p[m][n] = x_scales[m] * scales[n] * sum_k x[m][k] qweight[n][k],
 *   y[m][n] = round(p[m][n]), or round(act(p[m][n]) * p_up[m][n]) of a gated handle
 * (both projections, the activation and the product in one kernel).
 * The integers are exact, and so are sums below 2^24 in size (in fp32); larger
 * ones are rounded to fp32, in an order that depends on the shape and M. The
 * codes may be -128 .. 127.
 *   x: device int8 [M][ld_x], 16-byte aligned, ld_x a multiple of 16 (M > 1);
 *   x_scales: device fp32 [M]; y: device, `type`, [M][ld_y], apart from x.
 * Up to 32 tokens run in a kernel that streams the weights once, more on the
 * tensor cores, as do 17 on through more than 36 MB of weights. A handle's calls
 * share its workspace: order them on one stream, or by events, as those of other
 * handles with the same workspace; else handles are independent. The handle
 * belongs to the device that was current at create, which has to be current here.
 * Errors: INVALID_ARG, CUDA. */
spear_status_t spear_w8_forward(spear_w8_t h, const int8_t* x, int64_t ld_x, const float* x_scales, void* y, int64_t ld_y,
                                spear_dtype_t type, int32_t M, cudaStream_t stream);

/* The calls of a step with their arguments in one struct, the same otherwise: for bindings, where a call costs by the
 * argument (from Python 20 of them take 1.6 us, a struct 0.4). Errors: as theirs, INVALID_ARG also for NULL. */
typedef struct {
  const void* x;
  int64_t ld_x;
  const void* residual;
  int64_t ld_residual;
  void* residual_out;
  int64_t ld_residual_out;
  const void* weight;
  void* y;
  int64_t ld_y;
  int8_t* q;
  int64_t ld_q;
  float* scales;
  cudaStream_t stream;
  int32_t type, residual_type, weight_type; /* spear_dtype_t */
  int32_t M, K;
  float eps;
} spear_rms_norm_args_t;
spear_status_t spear_rms_norm_args(const spear_rms_norm_args_t* args);

typedef struct {
  const void* x;
  int64_t ld_x;
  int8_t* q;
  int64_t ld_q;
  float* scales;
  cudaStream_t stream;
  int32_t type, M, K;
} spear_quantize_rows_args_t;
spear_status_t spear_quantize_rows_args(const spear_quantize_rows_args_t* args);

typedef struct {
  const int8_t* q;
  int64_t ld_q;
  const float* scales;
  void* out;
  int64_t ld_out;
  cudaStream_t stream;
  int32_t type, M, K;
} spear_dequantize_rows_args_t;
spear_status_t spear_dequantize_rows_args(const spear_dequantize_rows_args_t* args);

typedef struct {
  spear_w8_t h;
  const int8_t* x;
  int64_t ld_x;
  const float* x_scales;
  void* y;
  int64_t ld_y;
  cudaStream_t stream;
  int32_t type, M;
} spear_w8_forward_args_t;
spear_status_t spear_w8_forward_args(const spear_w8_forward_args_t* args);

/* Synchronise `stream` and report the handle's device status: OK, or TIMEOUT if
 * a bounded device-side wait gave up since the last check; the status is then
 * cleared and the workspace reset. Handles that share the workspace: a call that
 * gave up may leave it so that later ones of more than 32 tokens (17 through many
 * weights) are wrong, until one of the handles that took part is checked; a handle
 * that made such a call reports TIMEOUT too. So check all of them, with no call on
 * the workspace running, before their results are used. */
spear_status_t spear_w8_check(spear_w8_t h, cudaStream_t stream);

/* Test surface for the bounded waits, as spear_linear_debug_set: wait_ns sets the device-side wait limit of this handle's
 * calls (0 restores the default of 100 ms); skip_arrive != 0 leaves out an arrival, so that a wait must run out:
 *  - up to 32 tokens: the first copy of weights (the call then gives up copying, writes wrong values and latches TIMEOUT);
 *  - more: the dequantising warps' first one in one pair of CTAs (which then gives up: its tiles are not written, tiles
 *    that it shares with others are not completed, and TIMEOUT is latched).
 * Errors: INVALID_ARG (NULL, wait_ns < 0). */
spear_status_t spear_w8_debug_set(spear_w8_t h, int64_t wait_ns, int32_t skip_arrive);

/* Free the handle's device memory (waits for queued work). NULL is accepted. */
spear_status_t spear_w8_destroy(spear_w8_t h);

/* Human-readable name of a status code (static storage). */
const char* spear_status_string(spear_status_t s);

#ifdef __cplusplus
}
#endif
#endif /* SPEAR_H_ */

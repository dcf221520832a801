/*
 * ocq.h -- C ABI of the quantized speculative-verify MLP block for AMD
 * MI355X (gfx950).
 *
 * What one call computes (the post "OCRia 推理栈：单卡 B200 提速近 10 倍"):
 *   x [M, hidden] bf16                            (M = requests x (1 + drafts),
 *                                                   section "Generate more tokens
 *                                                   per target pass")
 *   xq, sx = per-token E4M3 quantization of x     (sx = amax/448)
 *   G = (xq Wg^T) sx sw_g ;  U = (xq Wu^T) sx sw_u (weights FP8 or NVFP4, section
 *                                                   "Reducing the data moved:
 *                                                   workload-aware quantization")
 *   h = SiLU(G) * U, quantized per token to E4M3  (German page "Wie es
 *                                                   funktioniert": SiLU fused with
 *                                                   the quantization, kept in
 *                                                   registers)
 *   y = bf16( h Wd^T )                            (down projection in the
 *                                                   precision chosen for the
 *                                                   layer: FP8, BF16 or NVFP4)
 * Formats: E4M3 = OCP FP8 E4M3FN (max 448); E2M1 = OCP MX FP4; NVFP4 = E2M1
 * elements with one E4M3 scale per 16 inputs and one fp32 per-tensor scale.
 * Rounding: nearest, ties to even, saturating.  Scales: fl32(amax / 448) for
 * E4M3 rows, fl32(amax / 2688) per NVFP4 tensor, fl32(block amax / (6 S)) per
 * NVFP4 block before its own E4M3 rounding.  A zero row gets scale 0 and codes 0.
 *
 * Conventions for every entry point
 *   - Pointers named *_dev are device pointers (hipMalloc / torch CUDA
 *     tensors); *_host are host pointers.  The caller owns all memory and
 *     the stream; the library allocates nothing and frees nothing.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *   - A negative ocq_status is returned on failure, before anything is
 *     launched; ocq_last_error() then gives a message (thread-local, valid
 *     until the next call on the same thread).  Argument checks are
 *     synchronous; faults inside a kernel surface at the caller's next
 *     synchronization, as with any stream API.
 *   - Shapes: hidden and inter must be multiples of 128, 128 <= each <= 65536;
 *     1 <= M <= 8192.  Device pointers must be 16-byte aligned.
 */
#ifndef OCQ_H
#define OCQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  OCQ_OK = 0,
  OCQ_ERR_INVALID_ARG = -1,      /* null / misaligned pointer, bad M, bad enum   */
  OCQ_ERR_UNSUPPORTED = -2,      /* shape outside the supported set              */
  OCQ_ERR_DEVICE = -3,           /* HIP runtime error (no device, launch failure) */
  OCQ_ERR_BUFFER_TOO_SMALL = -4, /* packed blob or workspace smaller than needed  */
  OCQ_ERR_BAD_BLOB = -5          /* blob header does not match the call          */
} ocq_status;

typedef enum {
  OCQ_PREC_FP8 = 0,           /* gate/up FP8 E4M3, down FP8 E4M3                */
  OCQ_PREC_FP8_DOWN_BF16 = 1, /* gate/up FP8 E4M3, down BF16 (sensitive layer)  */
  OCQ_PREC_FP4 = 2            /* gate/up/down NVFP4                              */
} ocq_prec_mode;

/* Library version (major * 10000 + minor * 100 + patch). */
int ocq_version(void);

/* Bytes of the packed weight blob for one block; 0 if the shape or mode is
 * invalid.  The blob holds a 256-byte header followed by the quantized
 * gate/up and down weights in the kernels' fragment order and their scales. */
size_t ocq_packed_bytes(int hidden, int inter, int prec_mode);

/* Quantize and pack one block's weights into a HOST buffer (no GPU used).
 * w_gate_host, w_up_host: fp32 [inter, hidden] row-major ([out, in]).
 * w_down_host: fp32 [hidden, inter] row-major.  Weights must be finite.
 * FP8: one fp32 scale per output row, codes E4M3(fl32(w / scale)).
 * BF16 (down in OCQ_PREC_FP8_DOWN_BF16): round to nearest even.
 * NVFP4: per-tensor S, per-16-input E4M3 block scale, E2M1 codes.
 * packed_host must hold ocq_packed_bytes() bytes.  Thread-safe. */
ocq_status ocq_pack_weights_host(const float* w_gate_host, const float* w_up_host,
                                 const float* w_down_host, int hidden, int inter,
                                 int prec_mode, void* packed_host, size_t packed_bytes);

/* Same, then copy the blob to device memory with hipMemcpyAsync on `stream`
 * and wait for that copy (the staging buffer is freed before returning). */
ocq_status ocq_pack_weights(const float* w_gate_host, const float* w_up_host,
                            const float* w_down_host, int hidden, int inter, int prec_mode,
                            void* packed_dev, size_t packed_bytes, void* stream);

/* Activation-aware smoothing (optional).  The per-token E4M3 scale of x is
 * set by its largest channel, so a few outlier input channels cost every
 * other channel precision.  Per-input-channel factors s[k] move that range
 * into the gate/up weights: the blob holds the codes of fl32(W[n][k] s[k]),
 * and the block multiplies x by fl32(1 / s[k]) before quantizing it, which
 * leaves x W^T unchanged in exact arithmetic.  (The pages' precision is
 * chosen and calibrated per workload: "OCRia 推理栈：单卡 B200 提速近 10 倍",
 * section "Reducing the data moved: workload-aware quantization"; the rule
 * for s below is the published SmoothQuant one.)
 *
 * ocq_calibrate_smoothing_host: s[k] = amax_x[k]^alpha / amax_w[k]^(1-alpha)
 * in double, rounded once to float, where amax_x[k] is max |x[t][k]| over the
 * `rows` calibration rows (bf16 bits [rows, hidden], host) and amax_w[k] is
 * max |W[n][k]| over the rows of both W_gate and W_up (host fp32 [inter,
 * hidden]); s[k] = 1 where either is 0; clamped to [2^-20, 2^20].
 * alpha in [0, 1].  s_out: host float [hidden].
 *
 * ocq_pack_weights_smoothed_host / ocq_pack_weights_smoothed: as the plain
 * packers, with smooth_host = s (host float [hidden], every s[k] finite and
 * > 0; NULL = no smoothing, the same blob as the plain packers).  The down
 * projection is not smoothed.  Blobs are used by ocq_mlp_forward unchanged. */
ocq_status ocq_calibrate_smoothing_host(const void* x_calib_bf16_host, int rows, int hidden,
                                        const float* w_gate_host, const float* w_up_host, int inter,
                                        float alpha, float* s_out);
ocq_status ocq_pack_weights_smoothed_host(const float* w_gate_host, const float* w_up_host,
                                          const float* w_down_host, const float* smooth_host,
                                          int hidden, int inter, int prec_mode, void* packed_host,
                                          size_t packed_bytes);
ocq_status ocq_pack_weights_smoothed(const float* w_gate_host, const float* w_up_host,
                                     const float* w_down_host, const float* smooth_host, int hidden,
                                     int inter, int prec_mode, void* packed_dev, size_t packed_bytes,
                                     void* stream);

/* Inverse of the packing layout, for inspection and tests: from a HOST copy
 * of a blob, write one projection in plain row-major form.
 *   which = 0 gate, 1 up, 2 down, 3 the x multiplier (float [hidden] into
 *   scales_out; codes_out unused).
 *   codes_out: uint8 [rows, cols] (E4M3 or E2M1 code per byte) or uint16
 *              bf16 bits [rows, cols] for a BF16 projection.
 *   scales_out: FP8 -> float [rows]; NVFP4 -> uint8 E4M3 [rows, cols/16];
 *               BF16 -> unused (may be NULL).
 *   tensor_scale_out: NVFP4 -> S; others -> 0 (may be NULL). */
ocq_status ocq_unpack_weights_host(const void* packed_host, size_t packed_bytes, int which,
                                   void* codes_out, void* scales_out, float* tensor_scale_out);

/* Device workspace bytes needed by ocq_mlp_forward for this call shape. */
size_t ocq_workspace_bytes(int M, int hidden, int inter, int prec_mode);

/* Optional plain-layout copies of the intermediates, for parity checks,
 * written by the call's own kernels as they produce them.  Each pointer is a
 * 16-byte-aligned device pointer or NULL.
 *   x_codes [M, hidden] uint8, x_scales [M] float,
 *   h_out:  FP8/NVFP4 modes -> E4M3 codes [M, inter] uint8;
 *           BF16-down mode  -> bf16 bits [M, inter] uint16,
 *   h_scales [M] float (FP8/NVFP4 modes; untouched in BF16-down mode). */
typedef struct {
  void* x_codes;
  void* x_scales;
  void* h_out;
  void* h_scales;
} ocq_taps;

/* One MLP block over M rows, enqueued on `stream` (asynchronous).
 * packed_dev: blob from ocq_pack_weights for (hidden, inter, prec_mode),
 *             packed_bytes >= ocq_packed_bytes(...).
 * x_bf16_dev: bf16 [M, hidden] row-major, finite values.
 * y_bf16_dev: bf16 [M, hidden] row-major, written by the call.
 * workspace_dev: >= ocq_workspace_bytes(M, hidden, inter, prec_mode) bytes;
 *             contents need not be initialized; calls that share a
 *             workspace must be ordered on one stream.
 * taps: NULL or optional intermediate copies (see ocq_taps).
 * The blob header is not read back to the host (that would synchronize);
 * a blob packed for other dimensions or another mode gives wrong results
 * but all reads stay inside packed_bytes.  Use ocq_check_blob to verify. */
ocq_status ocq_mlp_forward(const void* packed_dev, size_t packed_bytes, const void* x_bf16_dev,
                           int M, int hidden, int inter, int prec_mode, void* y_bf16_dev,
                           void* workspace_dev, size_t workspace_bytes, const ocq_taps* taps,
                           void* stream);

/* The same forward call for callers that cannot allocate device memory
 * (code under HIP graph capture that may not call hipMalloc, tight serving
 * loops, hosts that forbid allocation): no workspace argument.  The
 * workspace is a fixed array of ocq_noalloc_scratch_bytes() bytes (32 MiB)
 * in device memory that the library holds on each device it runs on until
 * the process ends; the entry point itself allocates nothing.
 * Arguments, results and errors are those of ocq_mlp_forward, plus
 * OCQ_ERR_BUFFER_TOO_SMALL (before any launch) when
 * ocq_workspace_bytes(M, hidden, inter, prec_mode) exceeds the array.
 * Every call on one device shares that device's array: calls that overlap
 * on one device (different streams, or different threads without ordering)
 * race and give wrong results; calls ordered on one stream are safe.  The
 * array keeps the last call's contents; no call depends on them. */
size_t ocq_noalloc_scratch_bytes(void);
ocq_status ocq_mlp_forward_noalloc(const void* packed_dev, size_t packed_bytes, const void* x_bf16_dev, int M,
                                   int hidden, int inter, int prec_mode, void* y_bf16_dev, const ocq_taps* taps,
                                   void* stream);

/* A stack of L MLP blocks with a precision mode per layer (the pages'
 * mixed-precision scheme at model scale: each layer's weights in the
 * precision chosen for it, BF16 kept for sensitive layers; "OCRia 推理栈：单卡
 * B200 提速近 10 倍", section "Reducing the data moved: workload-aware
 * quantization").  Block l takes the previous block's bf16 output as its x
 * (block 0 takes x_bf16_dev) and the last block writes y_bf16_dev; each block
 * computes exactly what ocq_mlp_forward computes for its mode.
 *
 * ocq_stack_workspace_bytes: device workspace for the call shape (0 if any
 * argument is invalid): the largest block workspace of the schedule plus one
 * bf16 [M, hidden] buffer for the alternating intermediate outputs.
 *
 * ocq_mlp_stack_forward (asynchronous, on `stream`):
 * packed_devs[l]: blob of layer l packed for (hidden, inter, prec_modes[l]),
 *             packed_bytes[l] >= ocq_packed_bytes(hidden, inter, prec_modes[l]);
 * prec_modes: L modes (0, 1 or 2); 1 <= L <= 1024; host arrays, read during
 *             the call only.
 * x_bf16_dev, y_bf16_dev: bf16 [M, hidden]; x is only read, and y must not
 *             overlap x or the workspace.
 * workspace_dev: >= ocq_stack_workspace_bytes(...) bytes.
 * Errors: as ocq_mlp_forward, checked for every layer before any launch.
 * Stage events (ocq_set_stage_events) are not recorded by stack calls. */
size_t ocq_stack_workspace_bytes(int M, int hidden, int inter, const int* prec_modes, int L);
ocq_status ocq_mlp_stack_forward(const void* const* packed_devs, const size_t* packed_bytes,
                                 const int* prec_modes, int L, const void* x_bf16_dev, int M,
                                 int hidden, int inter, void* y_bf16_dev, void* workspace_dev,
                                 size_t workspace_bytes, void* stream);

/* Synchronously read a device blob's header and check it against
 * (hidden, inter, prec_mode): OCQ_OK or OCQ_ERR_BAD_BLOB. */
ocq_status ocq_check_blob(const void* packed_dev, size_t packed_bytes, int hidden, int inter,
                          int prec_mode, void* stream);

/* Per-stage timing hook (profiling).  When set, every later ocq_mlp_forward
 * on this thread records events[i] (hipEvent_t passed as void*, owned by the
 * caller; NULL entries are skipped) on the call's stream at stage boundary i:
 *   0 before the x quantization, 1 start of the gate/up + SiLU kernel,
 *   2 end of the gate/up kernel, 3 before the down projection, 4 after it.
 * Events 1 and 2 are taken by the gate/up launch itself (the kernel's own
 * start and end), so their difference is that kernel's execution time; the
 * others are recorded on the stream between launches.  Not for use while the
 * stream is being captured into a graph.  count must be 5 to enable, 0 (or
 * events == NULL) to disable.  The pointer array is copied; the events must
 * stay valid while the hook is set. */
ocq_status ocq_set_stage_events(void* const* events, int count);

/* Measurement helpers (not part of the block; used by the benchmark and the
 * tests to state what the block's timings and arithmetic are measured
 * against).  All are asynchronous on `stream` and return OCQ_OK,
 * OCQ_ERR_INVALID_ARG (bad size or pointer, checked before any launch) or
 * OCQ_ERR_DEVICE (launch failure).
 *
 * ocq_diag_stream_read: read `bytes` bytes (a multiple of 16, > 0) of the
 *   16-byte-aligned device buffer src_dev with 16-byte loads, `blocks`
 *   workgroups of 256 lanes (1 <= blocks <= 65536), each writing one uint32
 *   to out_dev[block] so the loads are kept: the practical HBM read ceiling
 *   for one launch of that many bytes (the block streams its weights the
 *   same way: "Why decoding dominates latency" in the post, weights read on
 *   every step).
 * ocq_diag_window_read: `blocks` workgroups of 256 lanes each read the same
 *   window of `window_bytes` bytes (a multiple of 32768, at most 2^30) at
 *   src_dev `passes` times with 16-byte loads, each writing one uint32 to
 *   out_dev[block]: with a window that fits L2, the rate at which L2 feeds
 *   the CUs (bytes read = blocks * passes * window_bytes), the ceiling for
 *   operands that many workgroups re-read.
 * ocq_diag_mfma_rate: `blocks` workgroups of 8 waves each issue iters x 16
 *   independent f16 MFMA 16x16x32 on register operands (1 <= iters <= 2^20);
 *   out_dev receives blocks * 512 floats (kept so the work is not dead);
 *   *flops (if non-null) the floating-point operations of the launch: the
 *   matrix-core rate the chip sustains, beside the published dense peak.
 * ocq_diag_empty: one empty kernel (the fixed cost of a launch).
 * ocq_diag_mfma_dot: c[m][n] = sum_k dec(a[m][k]) dec(b[n][k]) over E4M3
 *   codes (a: uint8 [M][K], b: uint8 [N][K], c: float [M][N], row-major,
 *   device, 16-byte aligned; M, N multiples of 16, K a multiple of 128,
 *   M, N, K <= 65536) through one matrix-core instruction form, with the
 *   block's fragment order and per-chunk instruction sequence:
 *     form 0: operands converted exactly to fp16, MFMA 16x16x32 f16 (fp32 sums)
 *     form 1: MFMA 16x16x128 f8f6f4 on the E4M3 codes (unit scales)
 *     form 2: MFMA 16x16x32 fp8 x fp8 on the E4M3 codes
 *   so that each form's sums can be compared against exact ones. */
ocq_status ocq_diag_stream_read(const void* src_dev, size_t bytes, void* out_dev, int blocks, void* stream);
ocq_status ocq_diag_window_read(const void* src_dev, size_t window_bytes, int passes, void* out_dev, int blocks,
                                void* stream);
ocq_status ocq_diag_mfma_rate(int iters, void* out_dev, int blocks, void* stream, double* flops);
ocq_status ocq_diag_empty(void* stream);
ocq_status ocq_diag_mfma_dot(int form, const void* a_dev, const void* b_dev, int M, int N, int K, float* c_dev,
                             void* stream);

/* Per-wave phase stamps of the GEMM main loops, for finding where a kernel's
 * time goes (the roofline method of "Why decoding dominates latency" in the
 * post, applied inside one kernel).  Only a library built with
 * `python -m quantized_memory_bound_amd.build --phase-stamps`
 * (libocq_phases.so) records them; the plain library returns
 * OCQ_ERR_UNSUPPORTED.  Copies, synchronously, the table of the last launch
 * of the chosen kernel family into host_out (caller-owned host memory of at
 * least the stated bytes, else OCQ_ERR_BUFFER_TOO_SMALL), as uint64 values
 * for workgroups 0..511:
 *   kernel 0, LDS-tiled GEMMs (524,288 B): [gate/up, down][workgroup][wave
 *     0..7][load wait, barrier, MFMA batches, LDS-read wait after the batches,
 *     whole loop, stage count], totals in shader-clock ticks;
 *   kernel 1, producer/consumer gate/up (393,216 B): [workgroup][wave 0..11:
 *     8 consumers, then 4 producers][entry, consumer loop start, loop end,
 *     partial tiles stored, wave end, 0, 0, 0], 100 MHz time stamps (the
 *     consumer-only fields are 0 for producers);
 *   kernel 2, x quantization and requantization (32,768 B): [x-quant,
 *     requant][workgroup 0..1023][start, end once its stores have landed],
 *     100 MHz time stamps (0 for workgroups that end early: padding rows,
 *     unused slots of the last group of m-tiles).
 * OCQ_ERR_INVALID_ARG for another kernel value or a null pointer,
 * OCQ_ERR_DEVICE if the copy fails. */
ocq_status ocq_diag_phase_stamps(int kernel, void* host_out, size_t bytes);

/* Where the per-token requantization of h runs (process-wide; mode 0 or 1,
 * default 1; another value: OCQ_ERR_INVALID_ARG).
 * 1: inside the gate/up kernel whenever its whole grid can be resident at
 * once (an occupancy check on the host before each launch): h stays in
 * registers, the row maxima meet through device-scope atomics and the
 * workgroups wait once for each other, bounded by 0.1 s (German page "Wie es
 * funktioniert" of the post: SiLU fused with the quantization, the
 * intermediate kept on chip).  Such a call must not share the GPU with
 * kernels that keep its workgroups from becoming resident for that long; if
 * the wait times out the call's y is NaN.  Where the grid does not fit (the
 * NVFP4 gate/up at 208 rows, the LDS-tiled kernels from 384 rows) or in the
 * BF16-down mode the call takes the two-pass form.  0: always the two-pass
 * form (fp32 h to the workspace, then a requantization kernel).  On MI355X
 * mode 1 is faster by 0.3-1.2 us per block.  Both give bit-identical
 * results. */
ocq_status ocq_set_fused_requant(int mode);

/* Where the last forward call on this thread (ocq_mlp_forward and its
 * no-allocation form, or the last block of ocq_mlp_stack_forward) requantized
 * h: 1 inside the gate/up kernel, 0 in a separate kernel (also the BF16-down
 * mode, which has no requantization), -1 before the first call. */
int ocq_last_requant_in_gateup(void);

/* ------------------------------------------------------------------------
 * The operators around the block in a speculative-verify layer: the norm in
 * front of it, rotary positions with the append to a paged cache, and the
 * attention of each request's new tokens over that cache ("Generate more
 * tokens per target pass" in the post: one verify pass over 1 + drafts tokens
 * per request; full-attention layers with a KV cache, "Why decoding dominates
 * latency").
 *
 * All are asynchronous on `stream`; tensors are bf16 with their last axis
 * contiguous, pointers 16-byte aligned and strides (in elements) multiples of
 * 8.  Sizes are checked on the host before any launch.  The contents of
 * device index arrays are not read by the host: the kernels bound every index
 * they form, so that wrong contents give wrong results, never an access
 * outside the tensors described by the call. */

/* Residual addition, RMSNorm and per-token E4M3 quantization in one pass:
 *   h = x + residual (fp32; residual_dev NULL: h = x)
 *   residual_out = bf16(h)
 *   y = h / sqrt(mean(h^2) + eps) * weight (fp32, of the unrounded h)
 *   scales = fl32(max|y| / 448), codes = E4M3(fl32(y / scale)); a zero row has
 *   scale 0 and codes 0 (with eps 0 too, where y is 0 / 0), any other row whose
 *   squares do not sum to a finite fp32 number, or with a y that is not finite,
 *   has scale NaN and codes 0.  (The
 *   bf16 y of a row whose squares overflow is what the formula gives in fp32:
 *   0 where h is finite.)
 * The codes are for 8-bit products of the caller's; the block of this library
 * takes bf16 and quantizes it itself.
 * x_bf16_dev, residual_bf16_dev: [rows, hidden] with row strides x_stride and
 * residual_stride; weight_bf16_dev [hidden]; residual_out_bf16_dev and
 * y_bf16_dev: [rows, hidden] contiguous, each nullable; codes_dev (uint8
 * [rows, hidden]) and scales_dev (float [rows]) both or neither; y or codes
 * must be given.  residual_out may be x or residual itself where that is
 * contiguous; any other overlap of an output with an input is not allowed.
 * 0 <= rows <= 2^24 (0: nothing is done), hidden a multiple of 8 in
 * [8, 65536], eps >= 0 and finite. */
ocq_status ocq_add_rmsnorm(const void* x_bf16_dev, int64_t x_stride, const void* residual_bf16_dev,
                           int64_t residual_stride, const void* weight_bf16_dev, float eps, int rows, int hidden,
                           void* residual_out_bf16_dev, void* y_bf16_dev, void* codes_dev, void* scales_dev,
                           void* stream);

typedef enum {
  OCQ_CACHE_BF16 = 0,   /* k, v bf16                                                   */
  OCQ_CACHE_E4M3 = 1,   /* k, v E4M3 codes, one fp32 scale (max / 448) per token and head */
  OCQ_CACHE_NVFP4 = 2   /* k, v E2M1 codes, one E4M3 scale (max / 6) per 16 elements       */
} ocq_cache_format;

/* A paged cache of one layer.  k_dev, v_dev: [num_pages, kv_heads, page_size,
 * head_dim] elements (bf16 or E4M3 codes) with the strides below, the same
 * for k and v: any order of the first three axes.  Strides in elements; in
 * bytes they are multiples of 16, a page's below 2^32 and a head's rows of one
 * page within 2^31.  k_scale_dev, v_scale_dev: float
 * [num_pages, kv_heads, page_size] with strides of their own (E4M3 only; a
 * page's below 2^32 elements, a head's scales of one page within 2^30).
 * NVFP4: k_dev, v_dev uint8 [num_pages, kv_heads, page_size, head_dim / 2], element
 * 2 i of a row in the low half of byte i, and k_scale_dev, v_scale_dev E4M3 bytes
 * [num_pages, kv_heads, page_size, head_dim / 16]; all strides in bytes, those of
 * the codes multiples of 16, those of the scales of 4 (their last axis contiguous).
 * An element is code x scale x unit: k_unit and v_unit, read for NVFP4 only, are
 * powers of two in [2^-64, 2^64] that move the scales' range (2^-9 to 448) to where
 * the values are (1 suits values from 0.1 to 2688).
 * page_size: a power of two up to 1024; head_dim 64, 128 or 256. */
typedef struct {
  void* k_dev;
  void* v_dev;
  void* k_scale_dev;
  void* v_scale_dev;
  int64_t page_stride, head_stride, token_stride;
  int64_t scale_page_stride, scale_head_stride, scale_token_stride;
  int num_pages, page_size, kv_heads, head_dim;
  int format;
  float k_unit, v_unit;
} ocq_kv_cache;

/* The tokens of one step.  The new tokens of request r are rows q_start[r] ..
 * q_start[r + 1] of the token axis (q_start[0] = 0, not falling, q_start
 * [requests] = tokens; a request may have none), kv_lens[r] tokens of it are
 * in the cache when these are in it, and place p of the request is row p %
 * page_size of page page_table[r][p / page_size].  New token i of n stands at
 * place kv_lens[r] - n + i.
 * q_start_dev int32 [requests + 1], kv_lens_dev int32 [requests],
 * page_table_dev int32 [requests, max_pages] with row stride table_stride.
 * max_new, max_kv: host bounds of the new tokens and of kv_lens of any
 * request.  Tokens past max_new of a request are not attended, nor are tokens
 * of no request: what out and lse hold for them is not defined.  max_kv only
 * shapes the split of the work, but for NVFP4 calls of many rows (see
 * ocq_paged_attention), which see no key past it.
 * counters_dev: uint32 [OCQ_ATTENTION_COUNTERS] for ocq_paged_attention and
 * ocq_verify_drafts (not read by the others): zeroed by the caller before the first call in that
 * call's order, zero again after every call; calls that share it must
 * be ordered on one stream.  If the device arrays change while a call runs its
 * counts may stay wrong: zero them again.
 * tokens * heads and max_pages * page_size stay below 2^31. */
typedef struct {
  const void* q_start_dev;
  const void* kv_lens_dev;
  const void* page_table_dev;
  int64_t table_stride;
  int requests, tokens, max_pages, max_new, max_kv;
  void* counters_dev;
} ocq_token_batch;
#define OCQ_ATTENTION_COUNTERS 4096

/* Rotary frequencies of rot dimensions (float64 [rot / 2] to inv_freq_out,
 * and to multiplier_out the factor of cos and sin), by a published rule:
 *   OCQ_ROPE_PLAIN   base^(-2 j / rot)
 *   OCQ_ROPE_LINEAR  the same / factor (positions divided by the factor)
 *   OCQ_ROPE_NTK     of the base base * factor^(rot / (rot - 2))
 *   OCQ_ROPE_YARN    (YaRN) those that turn at least beta_fast times in
 *                    context tokens as in PLAIN, at most beta_slow times as in
 *                    LINEAR, a ramp over j between; multiplier 0.1 ln(factor) + 1
 * factor >= 1, base > 1; context > 0 and beta_fast > beta_slow > 0 for YARN.
 * rot: a multiple of 16 in [16, 256].  Host only. */
typedef enum { OCQ_ROPE_PLAIN = 0, OCQ_ROPE_LINEAR = 1, OCQ_ROPE_NTK = 2, OCQ_ROPE_YARN = 3 } ocq_rope_scaling;
ocq_status ocq_rope_frequencies(int rot, double base, int scaling, double factor, double context, double beta_fast,
                                double beta_slow, double* inv_freq_out, float* multiplier_out);

/* Rotate q and k and append k and v to the cache.
 * q_dev [tokens, heads, head_dim], k_dev and v_dev [tokens, kv_heads,
 * head_dim]: token and head strides as given (slices of one projection's
 * output are fine).  inv_freq_dev: float64 [rot / 2]; rot a multiple of 16 up
 * to head_dim, elements past rot are not turned.  interleaved 0: pairs (j, j +
 * rot / 2); 1: pairs (2 j, 2 j + 1).  multiplier scales cos and sin.
 * positions_dev: int32 [tokens] rotary positions, or NULL for each token's
 * place in its request.  q_out_dev: [tokens, heads, head_dim] contiguous, or q
 * itself where that is contiguous.
 * bf16 caches receive bf16(k'), bf16(v); E4M3 caches the codes of the fp32 k'
 * and of v and their scales (a token's head with a value that is not finite:
 * scale NaN, codes 0).  NVFP4 caches receive, for each 16 elements of a head, the
 * scale s = E4M3(fl32(max / 6) / unit) and the codes E2M1(fl32(y / (s unit))) of y =
 * fl32(k'), which is turned in 64 bits (a code next to a border would hang on the
 * last bits of an angle in 32), or of v; nearest, ties to even, saturating; a scale
 * of 0 has codes 0, 16 elements with one that is not finite have scale NaN, codes
 * 0.  A token whose place is outside [0, max_pages *
 * page_size) or whose page is outside [0, num_pages) is not appended (its q is
 * rotated all the same).  Two new tokens must not share a cache slot. */
ocq_status ocq_rope_append(const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, const void* k_dev,
                           int64_t k_token_stride, int64_t k_head_stride, const void* v_dev, int64_t v_token_stride,
                           int64_t v_head_stride, int heads, const void* inv_freq_dev, int rot, int interleaved,
                           float multiplier, const void* positions_dev, const ocq_kv_cache* cache,
                           const ocq_token_batch* batch, void* q_out_dev, void* stream);

/* Attention of the batch's new tokens over the cache.  The token at place p
 * sees the keys j <= p, j < kv_len of its request for which window = 0, or
 * j > p - window, or j < sinks (the first tokens, which stay visible):
 *   out = sum_j softmax_j(scale q.k_j) v_j,  lse = ln sum_j e^(scale q.k_j).
 * A token that sees no key has out 0 and lse -inf.  heads is a multiple of the
 * cache's kv_heads; query head h reads kv head h / (heads / kv_heads).
 * q_dev [tokens, heads, head_dim] with token and head strides; out_dev bf16
 * [tokens, heads, head_dim] contiguous; lse_dev float [tokens, heads] or NULL.
 * scale > 0 and finite, window >= 0 (0: none), sinks >= 0 (0 without a
 * window).  Over NVFP4 caches both products are of fp16 operands: q after a power of
 * two of each row, the probabilities rounded to fp16; but where max_new x heads /
 * kv_heads is 1024 or more the pages are widened to fp16 in the workspace first, if
 * those of max_kv tokens a request fit 1 GiB.  Of a request whose kv_lens is past
 * max_kv, a bound that does not hold, such a call widens the first max_kv keys only:
 * its tokens keep their places (what kv_lens says) and see of those keys what the
 * mask leaves, out 0 and lse -inf where that is nothing.
 * Requests x kv heads x row tiles (of 16 to 128 of the max_new *
 * heads / kv_heads rows) are one launch of fewer than 2^32 lanes, 64 to 256 a
 * tile; beyond that: OCQ_ERR_UNSUPPORTED.  Scores, softmax statistics and sums are fp32; probabilities are
 * rounded to bf16 for the second product.
 * Rows that no token of the request sees (past kv_len, behind a window) never
 * reach a result, whatever the pages hold there.  A page outside [0,
 * num_pages) reads as zeros.  Where a token's value row is not finite, the
 * results of tokens of its request that do not see it may be NaN too, as 0 x
 * inf is.
 * workspace_dev: ocq_attention_workspace_bytes(...) bytes (may be 0), contents
 * need not be initialized; calls that share it must be ordered on one stream. */
size_t ocq_attention_workspace_bytes(int heads, const ocq_kv_cache* cache, const ocq_token_batch* batch, int window,
                                     int sinks);
ocq_status ocq_paged_attention(const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, int heads,
                               const ocq_kv_cache* cache, const ocq_token_batch* batch, float scale, int window,
                               int sinks, void* out_dev, void* lse_dev, void* workspace_dev, size_t workspace_bytes,
                               void* stream);

/* The values that an E4M3 or NVFP4 cache stands for, to move it to another format
 * or to look at it: k_out_dev, v_out_dev bf16 [num_pages, kv_heads, page_size,
 * head_dim] contiguous (NVFP4 values are exact in bf16, E4M3 ones are rounded). */
ocq_status ocq_cache_values(const ocq_kv_cache* cache, void* k_out_dev, void* v_out_dev, void* stream);

/* Which drafted tokens of a verify pass stay, and the token that follows them
 * ("Generate more tokens per target pass" in the post: the target checks every
 * draft at once and keeps those that it accepts).
 * Request r of the batch has rows t0 = q_start[r] .. q_start[r + 1] - 1, n of them:
 * tokens[t0] and its n - 1 drafts; row t of the target is the distribution p of the
 * token after tokens[t]: logits l with p = softmax(l / T) (T = 0: 1 at the largest
 * logit, the first of several), or with probabilities 1 p itself.  Draft i is
 * tokens[t0 + i + 1], drawn from q, row i of the request's draft rows (n - 1 a
 * request, side by side in the order of the requests); draft_dev NULL: q is 1 at
 * the draft (found by lookup or greedily).  The draft stays while
 *   u_accept[t0 + i] q(x) < p(x)
 * and all before it do.  At the first that does not, the next token is drawn from w
 * = max(p - q, 0) (p where that is 0 throughout), after the last one from w = p: the
 * lowest j with sum_{i <= j} w_i > u_next[r] sum_i w_i.  Sums and exponentials of
 * that row are 64-bit; the normalization of an acceptance's p is within 2^-19.
 *   accepted[r]            drafts that stay (0 for a request without tokens beside
 *                          others that have some)
 *   out[t0 .. t0 + n - 1]  those drafts, the next token, then -1; -1 too in rows
 *                          behind the last request
 * A next token of -1 says that the row has none: no weight above 0, or values that
 * are not numbers (at T > 0 also +inf).  Logits of -inf rule tokens out.  A draft
 * outside [0, vocab) is not accepted.
 * target_dev: fp32 (target_bf16 0) or bf16 [tokens, vocab], rows target_stride
 * elements apart, at any alignment of the type, vocab in [1, 2^24]; draft_dev
 * likewise, draft_rows rows.  tokens_dev int32 [tokens], u_accept_dev float
 * [tokens] and u_next_dev float [requests], numbers in [0, 1); temperature_dev float
 * [requests], or NULL: temperature for all (neither is read with probabilities 1).
 * accepted_dev int32 [requests], out_dev int32 [tokens]: not overlapping the inputs;
 * a batch without requests or without tokens has nothing to verify: OCQ_OK, nothing
 * is launched or written, accepted stays as the caller left it.  Of the batch q_start,
 * requests (up to OCQ_ATTENTION_COUNTERS), tokens (up to 2^20) and the counters are
 * used, the counters as attention uses them.
 * workspace_dev: ocq_verify_drafts_workspace_bytes(...) bytes, contents need not be
 * initialized; calls that share it must be ordered on one stream. */
size_t ocq_verify_drafts_workspace_bytes(const ocq_token_batch* batch, int vocab, int probabilities);
ocq_status ocq_verify_drafts(const void* target_dev, int64_t target_stride, int target_bf16, int probabilities,
                             const void* draft_dev, int64_t draft_stride, int64_t draft_rows, int draft_bf16,
                             const void* tokens_dev, const void* u_accept_dev, const void* u_next_dev,
                             const void* temperature_dev, float temperature, int vocab, const ocq_token_batch* batch,
                             void* accepted_dev, void* out_dev, void* workspace_dev, size_t workspace_bytes,
                             void* stream);

/* What a server keeps of its requests between steps, on the GPU: the arrays of an
 * ocq_token_batch, the pages that each request holds, and the free pages.
 * q_start_dev int32 [requests + 1], kv_lens_dev int32 [requests], page_table_dev
 * int32 [requests, max_pages] with row stride table_stride as in a batch; held_dev
 * int32 [requests]: the entries of a request's row that are its pages; ring_dev
 * int32 [ring_size]: page ids, free ones at places counts[0] .. counts[1] - 1 modulo
 * ring_size; counts_dev int64 [2]: entries ever taken out and put in.  ring_size is
 * at least the number of pages in all.  page_size a power of two up to 1024,
 * max_pages up to 2^30, max_pages * page_size and requests * max_pages below 2^31, up
 * to 65536 requests. */
typedef struct {
  void* q_start_dev;
  void* kv_lens_dev;
  void* held_dev;
  void* counts_dev;
  void* page_table_dev;
  void* ring_dev;
  int64_t table_stride;
  int requests, max_pages, ring_size, page_size;
} ocq_page_tables;

/* The tables of the next step.  Of request r's n tokens of the step before (its
 * share of before's q_start) 1 + accepted[r] stay, at most n (accepted_dev NULL:
 * all), and news[r] tokens come (news[r] < 0: the request has ended, keeps nothing
 * and brings nothing):
 *   kv_lens' = kv_lens - n + min(n, 1 + accepted) + news;  q_start' sums news
 *   held' = ceil(kv_lens' / page_size): what it lacks comes from the ring, in the
 *     order of the requests, what it no longer needs goes back there (and can be
 *     taken in the next call; its entries stay in the table, unused)
 * Where the ring has too few pages, or max_pages is too small, missing[0] counts
 * those that lack (at most 2^31 - 1), their entries in the table are -1 and held'
 * counts the others: appended tokens without a page are dropped, and the next call
 * tries again.
 * Per new token, in the order of the token axis (tokens rows, at least the sum of
 * news, up to 2^30; -1 in rows behind it): slots int64 (page * page_size + row in the page, -1
 * without a page), positions int32 (its place in the request), requests int32; each
 * and missing nullable.
 * before and after may be the same; they share the page table and the ring, which
 * are changed in place.  No output may overlap news or accepted. Tables without
 * requests: OCQ_OK, nothing is launched or written. */
size_t ocq_step_tables_workspace_bytes(const ocq_page_tables* tables, int tokens);
ocq_status ocq_step_tables(const ocq_page_tables* before, const ocq_page_tables* after, const void* news_dev,
                           const void* accepted_dev, int tokens, void* slots_dev, void* positions_dev,
                           void* requests_dev, void* missing_dev, void* workspace_dev, size_t workspace_bytes,
                           void* stream);

/* Message for the last failure on this thread ("" if none). */
const char* ocq_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* OCQ_H */

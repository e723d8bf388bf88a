/*
 * fp8bq.h -- C ABI of the B200 (sm_100a) W8A8 FP8 block-scaled linear layer.
 *
 * The method (page "ProCreations/Nanbeige4.3-33B-FP8", introduction and section
 * "Recipe and calibration"): linear layers run in W8A8 FP8 -- E4M3 weights with
 * one scale per 128x128 block (standard min-max, data independent) and
 * activations quantized dynamically per token and per group of 128 channels;
 * embeddings and the output head stay BF16 and are not part of this library.
 *
 * Numerics fixed by this library (the page leaves them open):
 *   - E4M3 is the OCP "e4m3fn" format (largest finite value 448, no infinities).
 *   - scale = amax / 448 computed as one IEEE binary32 division (round to
 *     nearest even); a group or block whose amax is 0 gets scale 1.0.
 *   - code = E4M3 round-to-nearest-even of fl32(x / scale), saturating at
 *     +-448; the sign of zero is kept; finite input never yields the NaN code.
 *   - the GEMM multiplies E4M3 codes exactly, sums each 128-wide K chunk in
 *     FP32, promotes the chunk into an FP32 accumulator multiplied by
 *     act_scale[m, kb] * weight_scale[n/128, kb], and rounds the result to BF16
 *     (round to nearest even).  Y = X W^T (W stored out x in, nn.Linear layout).
 *
 * Layouts: every matrix is dense and row-major (leading dimension = number of
 * columns).  X, Y: BF16 [M, K] / [M, N].  Codes: one byte per element, E4M3
 * bit patterns.  Activation scales: FP32 [M, K/128].  Weight scales: FP32
 * [N/128, K/128].
 *
 * Ownership: the caller allocates and frees every buffer (inputs, outputs and
 * workspace) in device memory of the current device; the library never
 * allocates device memory.  The only host state is a bounded cache of encoded
 * TMA descriptors keyed on address, shape, element type, box and swizzle (an
 * entry describes any tensor with that key, whatever the memory holds, so it
 * never goes stale; fp8bq_clear_cache() empties it).  Descriptors are passed
 * by value to the kernels.
 *
 * Execution: every compute call is asynchronous on the given stream (a
 * cudaStream_t passed as void*; NULL = the legacy default stream) and returns
 * after enqueueing.  It may be captured into a graph, the process's first call too
 * (but see fp8bq_gemm_noalloc).  Argument errors are detected on the host before anything
 * is enqueued and reported synchronously.  A kernel that gives up on an
 * internal wait (FP8BQ_ERR_TIMEOUT) records it in a per-device status word,
 * read by fp8bq_last_device_status().
 *
 * Requirements checked on the host (else the listed status, nothing enqueued):
 *   M >= 0, N > 0, K > 0, N % 128 == 0, K % 128 == 0  (else UNSUPPORTED_SHAPE;
 *     M == 0 is a no-op returning FP8BQ_OK);
 *   M, N, K <= 2^31 - 1 and every tensor smaller than 2^40 bytes (UNSUPPORTED_SHAPE);
 *   non-NULL pointers for every non-empty tensor (INVALID_ARG);
 *   every pointer 16-byte aligned (MISALIGNED);
 *   where a workspace is required (decode GEMMs and the fused linear, see
 *     fp8bq_workspace_size), at least that many bytes (WORKSPACE).
 * Inputs must be finite; NaN or infinite inputs give unspecified codes.
 *
 * Thread safety: calls on different streams may run concurrently as long as
 * they use different output and workspace buffers.
 */
#ifndef FP8BQ_H
#define FP8BQ_H

#include <stddef.h>
#include <stdint.h>

/* Symbols of this ABI are the only ones the shared library exports. */
#if defined(__GNUC__)
#define FP8BQ_API __attribute__((visibility("default")))
#else
#define FP8BQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FP8BQ_OK = 0,
    FP8BQ_ERR_INVALID_ARG = 1,       /* NULL pointer or negative size */
    FP8BQ_ERR_UNSUPPORTED_SHAPE = 2, /* N or K not a multiple of 128, or too large */
    FP8BQ_ERR_MISALIGNED = 3,        /* a pointer is not 16-byte aligned */
    FP8BQ_ERR_WORKSPACE = 4,         /* workspace missing or smaller than required */
    FP8BQ_ERR_CUDA = 5,              /* a CUDA runtime or driver call failed */
    FP8BQ_ERR_TIMEOUT = 6,           /* a kernel abandoned a bounded wait */
    FP8BQ_ERR_NO_DEVICE = 7,         /* no sm_100 device is current */
    FP8BQ_ERR_INDEX = 8              /* device side: a slot, page or length was out of range */
} fp8bq_status;

/* Operation selector for fp8bq_workspace_size. */
typedef enum { FP8BQ_OP_GEMM = 0, FP8BQ_OP_LINEAR = 1, FP8BQ_OP_GEMM_SILU = 2 } fp8bq_op;

/*
 * Dynamic per-token, group-128 activation quantization (page
 * "ProCreations/Nanbeige4.3-33B-FP8", introduction: activations get one scale
 * per token and per 128-channel group, computed at run time).
 *   x_bf16 : in,  BF16 [M, K]
 *   q_e4m3 : out, E4M3 codes [M, K]
 *   sa     : out, FP32 [M, K/128]; sa[m, g] = amax(|x[m, 128g : 128g+128]|) / 448, or 1
 * Codes and scales are bit-exact with the definition above.
 */
FP8BQ_API fp8bq_status fp8bq_quantize_act(const void *x_bf16, int64_t M, int64_t K, uint8_t *q_e4m3,
                                float *sa, void *stream);

/*
 * Offline 128x128-block min-max weight quantization (same page, section
 * "Recipe and calibration": one scale per 128x128 block of the E4M3 weights,
 * chosen by plain min-max without calibration data).
 *   w_bf16 : in,  BF16 [N, K] (out x in)
 *   q_e4m3 : out, E4M3 codes [N, K]
 *   sw     : out, FP32 [N/128, K/128]; sw[i, j] = amax of block (i, j) / 448, or 1
 * Codes and scales are bit-exact with the definition above.
 */
FP8BQ_API fp8bq_status fp8bq_quantize_weight(const void *w_bf16, int64_t N, int64_t K, uint8_t *q_e4m3,
                                   float *sw, void *stream);

/*
 * Block-scaled FP8 GEMM (same page, introduction: W8A8 FP8 linear layers with
 * BF16 activations in and out): Y[m, n] = BF16( sum_kb sa[m,kb] sw[n/128,kb]
 * sum_{k in kb} e4m3(qa[m,k]) e4m3(qw[n,k]) ).
 *   qa, sa : in, activation codes [M, K] and scales [M, K/128]
 *   qw, sw : in, weight codes [N, K] and scales [N/128, K/128]
 *   y_bf16 : out, BF16 [M, N]
 *   workspace, ws_bytes : device scratch of at least
 *       fp8bq_workspace_size(FP8BQ_OP_GEMM, M, N, K) bytes (may be NULL when
 *       that is 0; optional for M > 128, see fp8bq_workspace_size).  Its
 *       contents must be the state left by
 *       fp8bq_workspace_init() or by any previous successful fp8bq_gemm or
 *       fp8bq_linear call, of any shape (every successful call restores that
 *       state); calls that share a workspace must be ordered (same stream).
 * Output accuracy: |y - ref| <= 1e-2 |ref| + 2e-3 rms(ref) against the FP64 sum
 * of the dequantized operands; results are deterministic for a given shape.
 * Every operand is read only after the previous kernel in the stream has
 * completed; the call lets the next kernel launch early (programmatic
 * dependent launch) and that kernel waits for this one before reading its
 * output.
 */
FP8BQ_API fp8bq_status fp8bq_gemm(const uint8_t *qa, const float *sa, const uint8_t *qw, const float *sw,
                        int64_t M, int64_t N, int64_t K, void *y_bf16, void *workspace,
                        size_t ws_bytes, void *stream);

/*
 * Linear layer with the activation quantization fused into the call:
 * Y = gemm(quantize_act(X), qw, sw) with identical codes and scales.
 *   x_bf16 : in, BF16 [M, K]; qw / sw / y_bf16 as in fp8bq_gemm
 *   workspace : at least fp8bq_workspace_size(FP8BQ_OP_LINEAR, M, N, K) bytes,
 *               same state rule as fp8bq_gemm.
 * On the decode path the call starts reading qw / sw while earlier kernels in
 * the stream may still be running (programmatic dependent launch).  This is
 * safe against this library's weight quantizers, which never let a successor
 * start early; qw / sw must not be written by a foreign kernel that does.
 */
FP8BQ_API fp8bq_status fp8bq_linear(const void *x_bf16, const uint8_t *qw, const float *sw, int64_t M,
                          int64_t N, int64_t K, void *y_bf16, void *workspace, size_t ws_bytes,
                          void *stream);

/*
 * FP8 E4M3 KV-cache write with unit scales (page "ProCreations/Nanbeige4.3-33B-FP8",
 * "Serving" and the "Speed on Vega" table: --kv-cache-dtype fp8_e4m3 with unit
 * cache scales).  For every token t:
 *     k_cache[loc[t], i] = e4m3(k[t, i]),  v_cache[loc[t], i] = e4m3(v[t, i])
 * where e4m3(x) is the saturating round-to-nearest-even E4M3 code of x / 1 = x
 * (the same rule as every other code; NaN stays NaN, +-infinity gives +-448).
 *   k_bf16, v_bf16 : in, BF16 rows, row t at (element) offset t * row_stride;
 *       width elements per row (all KV heads of the token, e.g. the K and V
 *       column ranges of the fused QKV output, row_stride = its width).
 *   loc            : in, int64 [T] cache slot of each token (device memory).
 *   k_cache, v_cache : in/out, E4M3 codes, slot s at byte offset s * slot_stride;
 *       the first width bytes of each written slot are replaced, nothing else.
 *   num_slots      : slots in each cache.
 * Requirements: width and row_stride multiples of 8, slot_stride a multiple of
 * 16 and >= width, k/v/caches 16-byte and loc 8-byte aligned (MISALIGNED
 * otherwise).  Distinct tokens should have distinct slots (with duplicates,
 * which row a slot keeps is unspecified).  A token whose slot is outside
 * [0, num_slots) is skipped on the device and FP8BQ_ERR_INDEX is recorded in
 * the device status word (read with fp8bq_last_device_status).
 */
FP8BQ_API fp8bq_status fp8bq_kv_write_e4m3(const void *k_bf16, const void *v_bf16,
                                           int64_t row_stride, int64_t T, int64_t width,
                                           const int64_t *loc, uint8_t *k_cache,
                                           uint8_t *v_cache, int64_t num_slots,
                                           int64_t slot_stride, void *stream);

/*
 * SiLU-gated MLP product, quantized for the down projection (page
 * "ProCreations/Nanbeige4.3-33B-FP8", introduction: dynamic per-token group-128
 * activation quantization for every linear layer).  With gate = gu[:, :I] and
 * up = gu[:, I:],
 *     h = BF16( silu(gate) * up ),  silu(g) = g / (1 + exp(-g)),
 * and (q_e4m3, s) = the group-128 quantization of h, exactly what
 * fp8bq_quantize_act would produce from that BF16 h.  h itself differs from
 * the exactly rounded silu(gate) * up by at most one BF16 step (the
 * exponential is the hardware one).
 *   gu_bf16 : in, BF16 [M, 2I] row-major.
 *   q_e4m3  : out, E4M3 [M, I];  s : out, FP32 [M, I/128].
 *   h_bf16  : out, optional BF16 [M, I] (NULL: h is not stored).
 * I must be a multiple of 128; pointers 16-byte aligned.
 */
FP8BQ_API fp8bq_status fp8bq_silu_mul_quantize(const void *gu_bf16, int64_t M, int64_t I,
                                               uint8_t *q_e4m3, float *s, void *h_bf16,
                                               void *stream);

/*
 * Gate/up projection of the MLP with the SiLU-gated product quantized for the
 * down projection in the same pass (pages "ProCreations/Nanbeige4.3-33B-DFlash2",
 * "Architecture and checkpoint format": separate gate and up projections of the
 * MLP; "ProCreations/Nanbeige4.3-33B-FP8", introduction: every linear layer,
 * the down projection included, takes group-128 dynamically quantized
 * activations).  With gu = gemm(qa, sa, qw, sw) the BF16 [M, 2I] output of the
 * fused gate/up weight, this computes exactly
 *     fp8bq_silu_mul_quantize(gu, M, I, q_e4m3, s, h_bf16)
 * (same codes, scales and h, bit for bit) without gu ever reaching memory for
 * M > 128: there the GEMM's epilogue holds 128 gate channels and the same 128
 * up channels of a row and writes their h codes and scale directly.
 *   qa, sa : in, activation codes [M, K] and scales [M, K/128]
 *   qw, sw : in, the fused gate/up weight: codes [2I, K] (gate rows [0, I), up
 *            rows [I, 2I)) and scales [2I/128, K/128], e.g. from
 *            fp8bq_quantize_weight of the BF16 [2I, K] weight
 *   q_e4m3, s : out, the down projection's input codes [M, I], scales [M, I/128]
 *   h_bf16 : out, optional BF16 h [M, I] (NULL: not stored)
 *   workspace : at least fp8bq_workspace_size(FP8BQ_OP_GEMM_SILU, M, 2I, K)
 *       bytes (0 for M > 128; for M <= 128 the call runs the decode GEMM into
 *       the workspace and then the SiLU kernel), same state rule as fp8bq_gemm.
 * I a multiple of 128, K a multiple of 128; pointers 16-byte aligned.
 */
FP8BQ_API fp8bq_status fp8bq_gemm_silu_mul_quantize(const uint8_t *qa, const float *sa,
                                                    const uint8_t *qw, const float *sw, int64_t M,
                                                    int64_t I, int64_t K, uint8_t *q_e4m3,
                                                    float *s, void *h_bf16, void *workspace,
                                                    size_t ws_bytes, void *stream);

/*
 * Root-mean-square norm with the residual's addition, quantized for the linear
 * layer that follows (page "ProCreations/Nanbeige4.3-33B-DFlash2",
 * "Architecture and checkpoint format": RMSNorm; page
 * "ProCreations/Nanbeige4.3-33B-FP8", introduction: every linear layer's input
 * is quantized per token and 128-channel group).  For every row:
 *     r = BF16(x + residual)            (r = x when residual is NULL)
 *     h = r * (mean(r^2) + eps)^(-1/2) * weight     in FP32
 *     s[g] = amax(|h[128g : 128g+128]|) / 448, or 1 when that is 0
 *     q = E4M3(h / s)                   nearest, ties to even, saturating
 * The codes come from the FP32 h, not from its BF16 copy.
 *   x_bf16            : in, BF16 [M, K]
 *   residual_bf16     : in, BF16 [M, K], or NULL
 *   weight_bf16       : in, BF16 [K]
 *   residual_out_bf16 : out, BF16 [M, K], r; given exactly when residual_bf16
 *                       is; may be the same buffer as residual_bf16 or x_bf16
 *   q_e4m3, s         : out, codes [M, K] and scales [M, K/128]; both or neither
 *   h_bf16            : out, optional BF16 [M, K], BF16(h); required without q_e4m3
 * The sum of squares is FP32: |r| and |weight| below 2^60, and a row whose root mean
 * square is below 2^-50 needs eps >= 2^-100 (without it an all-zero row has no h; its
 * codes are 0).
 * K a multiple of 128, at most 32768; eps >= 0 and finite.  Other than the
 * aliasing named above, buffers must not overlap.
 */
FP8BQ_API fp8bq_status fp8bq_rms_norm_quantize(const void *x_bf16, const void *residual_bf16,
                                               const void *weight_bf16, float eps, int64_t M,
                                               int64_t K, void *residual_out_bf16,
                                               uint8_t *q_e4m3, float *s, void *h_bf16,
                                               void *stream);

/* How the rotary frequencies are stretched for contexts longer than trained. */
typedef enum {
    FP8BQ_ROPE_PLAIN = 0,  /* f_i = base^(-2i/rot_dim) */
    FP8BQ_ROPE_LINEAR = 1, /* f_i / factor (positions interpolated) */
    FP8BQ_ROPE_NTK = 2,    /* base * factor^(rot_dim / (rot_dim - 2)) */
    FP8BQ_ROPE_YARN = 3,   /* f_i up to the pair that turns beta_fast times in old_context, rounded
                              down, f_i / factor from the pair that turns beta_slow times,
                              rounded up, linear in i between; both ends within
                              [0, rot_dim - 1], at least 0.001 apart.  This is what YaRN
                              checkpoints are trained and served with.  cos and sin times
                              0.1 ln(factor) + 1 */
    FP8BQ_ROPE_YARN_EXACT = 4 /* the same with both ends as they are, not rounded */
} fp8bq_rope_scaling;

/*
 * Host helper: fills inv_freq[rot_dim / 2] (host memory) with the FP32 rotary
 * frequencies and *mscale with the factor on cosine and sine.  factor >= 1 is
 * used by every scaling but PLAIN; old_context, beta_fast > beta_slow > 0 by
 * the two YARN ones only.  A user with another schedule fills the table itself.
 */
FP8BQ_API fp8bq_status fp8bq_rope_inv_freq(int64_t rot_dim, double base, fp8bq_rope_scaling scaling,
                                           double factor, double old_context, double beta_fast,
                                           double beta_slow, float *inv_freq, float *mscale);

/*
 * Rotary positions of the fused QKV output, keys and values written to the
 * E4M3 cache (pages "ProCreations/Nanbeige4.3-33B-DFlash2", "Architecture and
 * checkpoint format": rotary positions, base 1.2e8; "ProCreations/
 * Nanbeige4.3-33B-FP8", "Serving": fp8_e4m3 cache with unit scales).  With
 * u = positions[t] * inv_freq[j] (the exact product) and for pair j of each
 * query and key head's first rot_dim channels
 *     (a, b) -> mscale * (a cos u - b sin u, b cos u + a sin u),
 * where (a, b) are channels (j, j + rot_dim/2), or (2j, 2j + 1) when
 * interleaved is not 0; channels from rot_dim on pass unchanged.  Queries are
 * rounded to BF16; keys are rounded once, to E4M3 (saturating), into slot
 * loc[t] of k_cache; values go to v_cache as fp8bq_kv_write_e4m3 writes them.
 *   qkv_bf16   : in, BF16 rows at (element) stride row_stride, columns
 *                [q_heads | kv_heads | kv_heads] x head_dim
 *   positions  : in, int64 [T];  loc : in, int64 [T] cache slots
 *   inv_freq   : in, FP32 [rot_dim / 2], device memory
 *   q_out_bf16 : out, BF16 rows at stride q_stride, [q_heads x head_dim]; may be
 *                qkv_bf16 itself (then q_stride == row_stride), else no overlap
 *   k_cache, v_cache, num_slots, slot_stride : as in fp8bq_kv_write_e4m3
 * head_dim a multiple of 16 up to 256, rot_dim a multiple of 16 up to
 * head_dim, strides multiples of 8 (slot_stride of 16), at most 1024 heads of
 * each kind; qkv, q_out and the caches 16-byte, positions and loc 8-byte
 * aligned.  Distinct tokens should have distinct slots (with duplicates, which of
 * the tokens each 8 bytes of a slot come from is unspecified).
 * A token with loc -1 is padding: nothing of it is written.  Any
 * other slot outside [0, num_slots) skips the token too and is reported as
 * FP8BQ_ERR_INDEX through fp8bq_last_device_status.
 */
FP8BQ_API fp8bq_status fp8bq_rope_kv_write_e4m3(
    const void *qkv_bf16, int64_t row_stride, int64_t T, int64_t q_heads, int64_t kv_heads,
    int64_t head_dim, const int64_t *positions, const float *inv_freq, int64_t rot_dim,
    int interleaved, float mscale, const int64_t *loc, void *q_out_bf16, int64_t q_stride,
    uint8_t *k_cache, uint8_t *v_cache, int64_t num_slots, int64_t slot_stride, void *stream);

/*
 * Attention of new tokens over the paged E4M3 cache (unit scales), for one
 * token per sequence (decode), a few (a drafter's block) or many (a prefill
 * chunk), mixed in one batch.  Page "ProCreations/Nanbeige4.3-33B-FP8",
 * "Serving": chunked prefill and decode over an fp8_e4m3 cache.
 * Sequence b has new tokens cu_q[b] .. cu_q[b+1] - 1 (rows of q and out) and
 * seq_lens[b] cache positions, the new tokens' own among them (already
 * written, e.g. by fp8bq_rope_kv_write_e4m3).  Position c lives in slot
 * page_table[b, c / page_size] * page_size + c % page_size.  New token i sees
 * positions 0 .. seq_lens[b] - q_len + i (causal != 0) or all seq_lens[b].
 * For query head h and kv head h / (q_heads / kv_heads):
 *     z_c = scale * (q . k_c),  lse = log sum_c exp(z_c),
 *     out = BF16( sum_c exp(z_c - lse) v_c ).
 * A token that sees no position gives zeros and lse = -infinity.
 *   q_bf16, out_bf16 : BF16 rows at (element) strides q_stride, out_stride,
 *                      [q_heads x 128]; must not overlap
 *   k_cache, v_cache : in, E4M3 codes, slot s at byte offset s * slot_stride,
 *                      [kv_heads x 128] (the layout fp8bq_kv_write_e4m3 writes)
 *   page_table       : in, int32 [B, max_pages] at stride table_stride;
 *                      entries beyond a sequence's length are not read
 *   seq_lens [B], cu_q [B + 1] : in, int32, device memory, cu_q ascending from 0
 *   max_q_len        : the most new tokens of any sequence
 *   lse              : out, optional FP32 [T, q_heads]
 *   workspace        : at least fp8bq_paged_attention_workspace_size(T, B, q_heads,
 *                      kv_heads, max_q_len) bytes, same state rule as fp8bq_gemm
 *                      (one workspace may serve both, in stream order)
 * Heads have 128 channels; q_heads a multiple of kv_heads, at most 1024;
 * page_size a power of two from 8 to 2^20, max_pages * page_size <= 2^25;
 * B <= 65536, T < 2^21; scale > 0; q, out and the caches 16-byte aligned,
 * q_stride and out_stride multiples of 8, slot_stride of 16.
 * Scores, softmax sums and outputs are accumulated in FP32.  What multiplies K
 * and V is rounded, the sums' weights are not.  Up to 16 new tokens x heads of a
 * group: queries exact down to 2^-14 of a row's largest channel and within 2^-22 of
 * it below; weights within 2^-8 of themselves, or 2^-23 of the largest weight in
 * the same run of at most 1920 positions if that is more.  Above 16: queries exact
 * down to 2^-9 and within 2^-17; weights within 2^-11, or 2^-32 of the row's largest.
 * Slots at or behind a sequence's length may hold anything, NaN codes too;
 * the cache positions that a sequence has must hold finite values, and q too,
 * with |z_c| below 2^21 (an FP32 score of that size is off by 0.1 as it is).
 * Rows of q and out at or behind cu_q[B] are padding: neither read nor written.
 * What the host cannot see is checked on the device, without a fault, and
 * reported as FP8BQ_ERR_INDEX through fp8bq_last_device_status: a page outside
 * the cache (its positions read as zeros), a length that is negative or beyond
 * max_pages * page_size (clamped), new tokens beyond max_q_len or T (skipped).
 */
FP8BQ_API fp8bq_status fp8bq_paged_attention(
    const void *q_bf16, int64_t q_stride, const uint8_t *k_cache, const uint8_t *v_cache,
    int64_t num_slots, int64_t slot_stride, const int32_t *page_table, int64_t table_stride,
    int64_t max_pages, int64_t page_size, const int32_t *seq_lens, const int32_t *cu_q, int64_t B,
    int64_t T, int64_t q_heads, int64_t kv_heads, int64_t max_q_len, float scale, int causal,
    void *out_bf16, int64_t out_stride, float *lse, void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace fp8bq_paged_attention requires (0 when none, and for
 * arguments it would reject).  Always a multiple of 256. */
FP8BQ_API size_t fp8bq_paged_attention_workspace_size(int64_t T, int64_t B, int64_t q_heads,
                                                      int64_t kv_heads, int64_t max_q_len);

/*
 * NVFP4 weight-only format with BF16 activations (page
 * "ProCreations/Nanbeige4.3-33B-NVFP4-A16", recipe paragraph: FP4 E2M1 weights
 * in groups of 16 with E4M3 block scales and a global weight scale; activations
 * BF16).  A weight is w[n, k] = e2m1(q[n, k]) * e4m3(sb[n, k/16]) * g.
 * Layout: packed [N, K/2] bytes, element 2j in the low nibble and 2j+1 in the
 * high nibble of byte j of its row; sb [N, K/16] E4M3 codes; g one FP32 value.
 *
 * fp8bq_nvfp4_quantize_weight: plain min-max quantization (the page's own
 * scales come from a data-driven search, which needs calibration data):
 *   g  = fl32(amax(|W|) / 2688)   (2688 = 6 * 448; 1.0 when W is all zero)
 *   sb = E4M3_RNE_sat(fl32(amax_group / fl32(6 g)))
 *   q  = E2M1_RNE_sat(fl32(w / fl32(e4m3(sb) * g)))   (0 when that scale is 0)
 *   w_bf16 : in, BF16 [N, K], K a multiple of 16.
 *   packed : out, [N, K/2];  sb : out, [N, K/16];  g : out, one float (device).
 * Codes, block scales and g are bit-exact with that definition.  Pointers
 * 16-byte aligned (g: 4).  Three kernels and a 4-byte memset on `stream`.
 */
FP8BQ_API fp8bq_status fp8bq_nvfp4_quantize_weight(const void *w_bf16, int64_t N, int64_t K,
                                                   uint8_t *packed, uint8_t *sb, float *g,
                                                   void *stream);

/*
 * Y[m, n] = BF16( sum_k x[m, k] * w[n, k] ) for BF16 X [M, K] and an NVFP4 W
 * [N, K] in the layout above; g is read from device memory (e.g. as written by
 * fp8bq_nvfp4_quantize_weight).  N a multiple of 128, K a multiple of 256;
 * pointers 16-byte aligned (g: 4).  No workspace.  Accuracy as fp8bq_gemm:
 * |y - ref| <= 1e-2 |ref| + 2e-3 rms(ref) against the FP64 sum.  Built for
 * decode-sized M; every 16 rows of M stream the weights once.
 */
FP8BQ_API fp8bq_status fp8bq_nvfp4_gemm_a16(const void *x_bf16, const uint8_t *packed,
                                            const uint8_t *sb, const float *g, int64_t M,
                                            int64_t N, int64_t K, void *y_bf16, void *stream);

/*
 * fp8bq_gemm without a workspace argument, for callers that cannot allocate
 * device memory: code running where no allocator is reachable (an embedding
 * runtime that hands out only fixed buffers, or a context where cudaMalloc is
 * not permitted).  The pages describe no such call; it is a convenience of the
 * library.  Same arguments, results and accuracy as fp8bq_gemm, minus the
 * workspace.  Its scratch is a 4 MiB array inside the library (held on every
 * GPU that loads it until the process exits).  Problems whose split-K scratch
 * would exceed it are rejected with FP8BQ_ERR_WORKSPACE when M <= 16 (that
 * is, N > 32512); for 16 < M <= 128 they run on the prefill kernel instead,
 * which needs no scratch, and M > 128 never needs any.  It calls no allocator.
 *   - The first call on a device looks up the array's device address (a
 *     one-time set-up); make that first call before any stream capture.
 *   - All calls share the one array: calls that overlap on the GPU (other
 *     streams, other host threads) race and give wrong results; order them.
 *   - Each call first clears the part of the array that must start at zero
 *     (a memset on its stream).
 */
FP8BQ_API fp8bq_status fp8bq_gemm_noalloc(const uint8_t *qa, const float *sa, const uint8_t *qw,
                                          const float *sw, int64_t M, int64_t N, int64_t K,
                                          void *y_bf16, void *stream);

/* Bytes of workspace the operation uses for this shape (0 when none, and for
 * arguments the call would reject).  Always a multiple of 256.  For M <= 128
 * the call requires at least this much.  For M > 128 (the prefill GEMM) any
 * workspace is accepted, NULL included, and the size is 0 unless K >= 16384.
 * There, with at least this much, a last wave of at most 16 output tiles on
 * the persistent grid is split K-wise over more CTAs (FP32 partials summed in
 * a fixed order, so results stay deterministic and within the same
 * tolerance), which a smaller workspace goes without.  The fused linear
 * requires, besides the GEMM's part (never less than its 16 KB counter
 * header), its activation codes and scales.  FP8BQ_OP_GEMM_SILU takes N = 2I
 * (the fused gate/up weight's rows): 0 for M > 128, else the GEMM's part (at
 * least the header) and the BF16 gate/up output [M, 2I].
 * Every workspace starts with the same 16 KB header of split-K counters, at
 * offset 0 for every operation and shape, and every successful call leaves
 * them at zero: one workspace, large enough for each call, can serve any
 * sequence of fp8bq_gemm, fp8bq_linear and fp8bq_gemm_silu_mul_quantize calls
 * in stream order. */
FP8BQ_API size_t fp8bq_workspace_size(int op, int64_t M, int64_t N, int64_t K);

/* Put a workspace into its initial state (zero-fills ws_bytes bytes on the
 * stream).  Needed once after allocation and after a call that reported
 * FP8BQ_ERR_TIMEOUT. */
FP8BQ_API fp8bq_status fp8bq_workspace_init(void *workspace, size_t ws_bytes, void *stream);

/* Synchronizes the stream, then returns and clears the current device's status
 * word: FP8BQ_OK, or FP8BQ_ERR_TIMEOUT if a kernel abandoned a wait since the
 * last read.  A failed synchronize returns FP8BQ_ERR_CUDA. */
FP8BQ_API fp8bq_status fp8bq_last_device_status(void *stream);

/* Static description of a status code (never NULL). */
FP8BQ_API const char *fp8bq_status_string(fp8bq_status status);

/* Diagnostic for the failure path: launches a kernel whose only internal wait
 * can never complete, with the same bounded wait every kernel of the library
 * uses, limited to limit_us microseconds (1 .. 2e6).  It returns after
 * enqueueing; afterwards fp8bq_last_device_status() reports FP8BQ_ERR_TIMEOUT
 * (and clears it).  Nothing faults or hangs; the context stays usable. */
FP8BQ_API fp8bq_status fp8bq_selftest_timeout(uint32_t limit_us, void *stream);

/* Number of kernels this library has launched in this process (all devices). */
FP8BQ_API uint64_t fp8bq_launch_count(void);

/* ABI version: major * 10000 + minor * 100 + patch. */
FP8BQ_API int fp8bq_version(void);

/* The library keeps the TMA descriptors it encodes, keyed on everything an
 * encoding depends on (address, shape, element type, box, swizzle), so a
 * repeated call skips the encoding; an entry is valid for any tensor matching
 * its key, so entries never go stale.  The cache is bounded (it empties itself
 * when full); this call empties it now.  Host memory only; thread-safe. */
FP8BQ_API void fp8bq_clear_cache(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_H */

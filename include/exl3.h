/*
 * exl3.h - C ABI of the MI355X (gfx950) EXL3 quantized-linear library.
 *
 * The operation (sources: the exl3xpu README, sections "MoE (routed experts)",
 * "Prefill: int8 linears ..." and "Adding a model"; the Arc 140V MoE post,
 * sections 1 and 2A-2D; TensorFold issue #832, "Description"):
 *
 *   An EXL3 tensor of shape k x n (k = in_features, n = out_features, both
 *   multiples of 128) stores 16x16 weight tiles as K-bit trellis codes
 *   (K = 1..8): a uint16 array trellis[k/16][n/16][16*K], plus fp16 sign
 *   vectors suh[k] and svh[n] and an optional fp16 bias[n].  Decoding a tile
 *   gives the Hadamard-domain weight W~ (fp16, k x n), and the layer is
 *
 *       y = ((x .* suh) Hk  W~  Hn) .* svh (+ bias)
 *
 *   where Hd applies the orthonormal 128-point Walsh-Hadamard transform
 *   (Sylvester order, scaled by 1/sqrt(128)) to each block of 128 consecutive
 *   elements.
 *
 *   Decode of tile (a, b): its 16*K words, read in index order and each word
 *   most-significant bit first, form a cyclic bitstream of 256*K bits.  State
 *   j (0..255) is the 16-bit window starting at bit K*j (wrapping around).
 *   The mul1 codebook (marker EXL3_CODEBOOK_MUL1, the pages' "cb=2") maps a
 *   state S to fp16_RN((sigma - 510) * 1775 / 2^18), sigma being the sum of
 *   the four bytes of (S * 0x9E3779) mod 2^32; every value lies within
 *   +-3.453125.  State j is weight W~[16a + j/16][16b + j%16].
 *
 * Conventions for every entry point:
 *   - Pointers named as device pointers must point to GPU memory of the
 *     current HIP device; the caller allocates and owns every buffer.  The
 *     library keeps no pointer after a call returns and allocates nothing.
 *   - Every call only enqueues work on `stream` (NULL = the default stream):
 *     no host synchronisation, no read-back of device data.
 *   - Arguments are validated on the host before anything is enqueued; on any
 *     error nothing is enqueued and a status other than EXL3_OK is returned.
 *     There is no fallback to another code path.
 *   - Device pointers must be 16-byte aligned unless stated otherwise.
 *   - A tensor holds fewer than 2^31 tiles: (k/16) * (n/16) < 2^31, and its
 *     trellis is smaller than 4 GiB (k * n * bits / 8 < 2^32 bytes); for an
 *     arena this holds for each (expert, slot) tensor, at width 8 when the
 *     width is per expert.
 *   - Sizes whose launches would not fit the hardware's grid limit (2^24 - 1
 *     workgroups of 256 threads) return EXL3_E_INVALID: calls with m > 2^24
 *     rows; prefill calls with ceil(m/16) * (k/128) or ceil(m/64) * (n/128)
 *     at or above that limit; exl3_reconstruct* with (k/16) * (n/16) >= 2^29;
 *     exl3_hadamard with rows * (dim/128) >= 2^26.  Workspace-size queries
 *     return 0 for m > 2^24.
 *   - Calls on different streams may run concurrently; a call must not
 *     overlap another call that writes the same output or workspace.
 */
#ifndef EXL3_H
#define EXL3_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define EXL3_ABI_VERSION 1

/* The only codebook this library decodes (the pages' "mul1", marker cb=2). */
#define EXL3_CODEBOOK_MUL1 2

/* Largest supported routing fan-out for exl3_grouped_experts. */
#define EXL3_MAX_TOPK 16

/* Largest number of tensors in one exl3_linear_multi call. */
#define EXL3_MAX_MULTI 8

typedef struct ihipStream_t* exl3_stream_t; /* same type as hipStream_t */

typedef enum exl3_status {
    EXL3_OK = 0,
    EXL3_E_INVALID = 1,     /* bad size, width, pointer or alignment */
    EXL3_E_UNSUPPORTED = 2, /* codebook other than mul1 (fail-closed) */
    EXL3_E_WORKSPACE = 3,   /* workspace missing or too small */
    EXL3_E_HIP = 4          /* a HIP launch reported an error */
} exl3_status;

typedef enum exl3_dtype {
    EXL3_F16 = 0,
    EXL3_F32 = 1
} exl3_dtype;

/* One EXL3 tensor (all pointers are device pointers).
 *   trellis  uint16 [k/16][n/16][16*bits], row-major, 16-byte aligned
 *   suh      fp16 [k] (sign applied before the input transform)
 *   svh      fp16 [n] (sign applied after the output transform)
 *   bias     fp16 [n] or NULL (added last)
 *   k, n     multiples of 128 (16 suffices for exl3_reconstruct)
 *   bits     trellis width K, 1..8
 *   codebook must be EXL3_CODEBOOK_MUL1                                   */
typedef struct exl3_weight {
    const uint16_t* trellis;
    const uint16_t* suh;
    const uint16_t* svh;
    const uint16_t* bias;
    int32_t k;
    int32_t n;
    int32_t bits;
    int32_t codebook;
} exl3_weight;

/* A packed arena of per-expert EXL3 tensors, one allocation per tensor kind
 * (Arc 140V MoE post, section 2A: w13 [E, 2, ...] and w2 [E, 1, ...]).
 *   trellis  uint16 [experts][slots][k/16][n/16][16*bits]
 *   suh      fp16 [experts][slots][k]
 *   svh      fp16 [experts][slots][n]
 * Width and codebook are uniform over the arena (exl3_grouped_experts), or
 * the width is per expert (exl3_expert_widths, exl3_grouped_experts_mixed). */
typedef struct exl3_expert_weights {
    const uint16_t* trellis;
    const uint16_t* suh;
    const uint16_t* svh;
    int32_t experts;
    int32_t slots;
    int32_t k;
    int32_t n;
    int32_t bits;
    int32_t codebook;
} exl3_expert_weights;

/* Returns EXL3_ABI_VERSION of the built library. */
int32_t exl3_abi_version(void);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* exl3_status_str(exl3_status status);

/* exl3_reconstruct - decode a whole tensor to W~ (Hadamard domain, no signs).
 * The exl3xpu README ("Correctness") gates every kernel path on bit-identical
 * dequantized weights; this entry point exposes the decode for that check.
 *   w_out  fp16 [k][n] row-major, device pointer, 16-byte aligned.
 * Requires k, n multiples of 16.  Output is bit-exact by definition.       */
exl3_status exl3_reconstruct(const exl3_weight* w, uint16_t* w_out, exl3_stream_t stream);

/* exl3_hadamard - out = ((in .* sign_before) Hdim) .* sign_after, row by row
 * (the standalone randomized Hadamard transform of the exl3xpu README,
 * "Layout": Hadamard in/out kernels; and the MoE post, section 2C).
 *   in, out      [rows][ld_*] of `dtype` (EXL3_F16 or EXL3_F32); in-place
 *                (in == out with equal strides) is allowed
 *   dim          multiple of 128; transformed in blocks of 128
 *   ld_in/ld_out row strides in elements, >= dim, multiples of 8
 *   sign_before, sign_after  fp16 [dim] device pointers or NULL
 * Arithmetic is fp32; an fp16 output is rounded to nearest.               */
exl3_status exl3_hadamard(const void* in, void* out, int32_t dtype, int64_t rows, int64_t dim,
                          int64_t ld_in, int64_t ld_out, const uint16_t* sign_before,
                          const uint16_t* sign_after, exl3_stream_t stream);

/* Bytes of device workspace exl3_linear needs for m rows of this tensor
 * (0 if the arguments are invalid). */
size_t exl3_linear_workspace_size(const exl3_weight* w, int64_t m);

/* exl3_linear - y = ((x .* suh) Hk W~ Hn) .* svh (+ bias).
 * (exl3xpu README "Layout": the linear op dispatches on the row count; the
 * GEMM runs in the Hadamard domain per "Prefill: int8 linears ...";
 * TensorFold issue #832: rows are computed independently of the batch.)
 *   x      fp16 [m][ldx] device pointer, ldx >= k, ldx multiple of 8
 *   y      [m][ldy] of y_dtype (EXL3_F16 or EXL3_F32; fp32 outputs are the
 *          issue's "decodeF32/promptF32" contract), ldy >= n, multiple of 8
 *   ws     device workspace of at least exl3_linear_workspace_size(w, m)
 *          bytes (may be NULL when that size is 0): scratch of the call
 *          (partial sums, the transformed activations).  Nothing is kept in
 *          it between calls, so it needs no clearing and serves later calls
 *          of any size on the same stream; calls that overlap on it race.
 * m == 0 returns EXL3_OK without enqueueing anything.  The kernel (decode
 * GEMV for m <= 16, MFMA GEMM above) is chosen internally from m.  Within
 * each of the ranges 1 <= m <= 16 and m > 16 a row's result does not depend
 * on m or on the other rows (bit for bit); across them the summation order
 * differs, so results agree to rounding.
 * The trellis of the tensor must be smaller than 4 GiB (k * n * bits / 8 <
 * 2^32 bytes), else EXL3_E_INVALID.                                        */
exl3_status exl3_linear(const exl3_weight* w, const void* x, int64_t m, int64_t ldx, void* y,
                        int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                        exl3_stream_t stream);

/* Bytes of the device array behind exl3_linear_no_workspace (32 MiB). */
#define EXL3_SCRATCH_BYTES ((size_t)32 << 20)

/* exl3_linear_no_workspace - exl3_linear without a workspace argument, for
 * callers that cannot allocate device memory at all: code recorded into a
 * graph, tight serving loops, harnesses that forbid allocation.  The same
 * operation, arguments (minus ws and ws_bytes), validation, kernels and
 * results, bit for bit, as exl3_linear with a workspace.  The workspace is a
 * device array of EXL3_SCRATCH_BYTES that the library holds on every GPU it
 * runs on until the process ends; the call itself allocates nothing.
 *   - A call that needs more than EXL3_SCRATCH_BYTES of workspace
 *     (exl3_linear_workspace_size(w, m) > EXL3_SCRATCH_BYTES) returns
 *     EXL3_E_WORKSPACE with nothing enqueued.  Every decode call (m <= 16)
 *     of tensors up to 5120 x 17408 fits, and prefill calls while
 *     m * k * 2 bytes (plus a small head) fit.
 *   - All calls on one GPU share that GPU's array: two calls whose work
 *     overlaps in time on one GPU (other streams, other host threads) race
 *     and give undefined results.  Calls in order on one stream are safe.
 *     Nothing in the array needs to start at zero (these kernels keep no
 *     state in it between calls).
 *   - The first call on each GPU looks up the array's device address (a
 *     host-side query, nothing enqueued); make it outside graph capture.   */
exl3_status exl3_linear_no_workspace(const exl3_weight* w, const void* x, int64_t m, int64_t ldx,
                                     void* y, int64_t ldy, int32_t y_dtype, exl3_stream_t stream);

/* Bytes of device workspace exl3_linear_multi needs for m rows of these
 * tensors (0 if the arguments are invalid). */
size_t exl3_linear_multi_workspace_size(const exl3_weight* const* w, int32_t count, int64_t m);

/* exl3_linear_multi - y[i] = exl3_linear(w[i], x) for i < count, for the
 * projections that read one input (q, k and v; gate and up), each tensor with
 * its own width, shape, signs and bias (TensorFold issue #832,
 * "Description": widths are mixed per tensor; the fused multi-tensor launch
 * is the issue's "fused-shard" idea).
 *   w      host array of count tensor records, 1 <= count <= EXL3_MAX_MULTI,
 *          all with the same k (the records' buffers are device pointers)
 *   x      fp16 [m][ldx] device pointer, as for exl3_linear
 *   y      host array of count device pointers, y[i] is [m][ldy[i]] of
 *          y_dtype with ldy[i] >= w[i]->n, multiple of 8
 *   ws     device workspace of at least exl3_linear_multi_workspace_size
 *          bytes, scratch of the call as for exl3_linear
 * m == 1 runs all tensors in one decode-GEMV launch and one finishing
 * launch (each tensor keeps its own split over a share of the waves, in
 * proportion to its trellis bytes, so its results agree with exl3_linear to
 * rounding); m >= 2 runs the tensors one after another through exl3_linear
 * (bit-identical to separate calls).  m == 0 returns EXL3_OK.  Validation of
 * every tensor happens before anything is enqueued.                       */
exl3_status exl3_linear_multi(const exl3_weight* const* w, int32_t count, const void* x, int64_t m,
                              int64_t ldx, void* const* y, const int64_t* ldy, int32_t y_dtype,
                              void* ws, size_t ws_bytes, exl3_stream_t stream);

/* exl3_reconstruct_int8 - the int8 weights W_q of the int8 prefill (exl3xpu
 * README, "Prefill: int8 linears ...": one static weight scale fused into
 * reconstruct).  W_q = RNE((sigma - 510) * 1775 / 2^18 * 127 / 3.453125) for
 * each state's byte sum sigma, taken from the codebook value before its fp16
 * rounding; |W_q| <= 127.
 *   w_out  int8 [k][n] row-major, device pointer, 16-byte aligned.
 * Requires k, n multiples of 16.  Output is bit-exact by definition.       */
exl3_status exl3_reconstruct_int8(const exl3_weight* w, int8_t* w_out, exl3_stream_t stream);

/* Bytes of device workspace exl3_linear_int8 needs for m rows of this tensor
 * (0 if the arguments are invalid or m == 0). */
size_t exl3_linear_int8_workspace_size(const exl3_weight* w, int64_t m);

/* exl3_linear_int8 - the int8 prefill linear (exl3xpu README, "Prefill: int8
 * linears ..."): activations get one int8 scale per row inside the input
 * transform, weights the static scale of exl3_reconstruct_int8, and the
 * product runs on int8 matrix cores with both scales applied:
 *   x' = (x .* suh) Hk;  a_r = max |x'_r|;  x_q = RNE(127 x' / a_r)
 *   y  = ((x_q W_q) * (a_r / 127) * (3.453125 / 127)) Hn .* svh (+ bias)
 * The integer product is exact; x' and the scales are fp32.
 *   x, y, ldx, ldy, y_dtype  as for exl3_linear
 *   ws     device workspace of at least exl3_linear_int8_workspace_size(w, m)
 *          bytes (x_q and the row scales; no state is kept between calls)
 * Any m >= 1 is accepted (the pages use it for prefill, more than 128 rows);
 * rows are independent, so a row's result does not depend on m or on the
 * other rows, bit for bit.  An all-zero row gives y = bias.  m == 0 returns
 * EXL3_OK.  Compared with exl3_linear the outputs differ by the int8
 * rounding of activations and weights (about 1e-2 relative).              */
exl3_status exl3_linear_int8(const exl3_weight* w, const void* x, int64_t m, int64_t ldx, void* y,
                             int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                             exl3_stream_t stream);

/* Bytes of device workspace exl3_grouped_experts needs (0 if invalid). */
size_t exl3_grouped_experts_workspace_size(const exl3_expert_weights* gate_up,
                                           const exl3_expert_weights* down, int64_t t,
                                           int32_t topk);

/* exl3_grouped_experts - routed-expert SwiGLU MLP, routed contribution only.
 * (exl3xpu README "MoE (routed experts)": computed in fp32 with the routing
 * weight applied to the down-projection output, never to its input; one
 * launch per projection with routing kept on device; MoE post section 2:
 * SiLU between the two launches, device-side token binning, fp32 gather.)
 *   gate_up  arena with slots == 2 (slot 0 = gate, slot 1 = up), k = hidden,
 *            n = intermediate
 *   down     arena with slots == 1, k = intermediate, n = hidden, same
 *            number of experts
 *   x             fp16 [t][hidden] device pointer (row stride = hidden)
 *   topk_ids      int32 [t][topk] device pointer, each in [0, experts)
 *   topk_weights  fp32 [t][topk] device pointer
 *   y             fp32 [t][hidden] device pointer, overwritten with
 *                 Y[i] = sum over s in slot order of w[i][s] * down_e(a),
 *                 a = silu(gate_e(x_i)) * up_e(x_i), e = topk_ids[i][s]
 *   ws            device workspace of at least the queried size, zero-filled
 *                 before its first use; calls leave its arrival counts at
 *                 zero, so it serves later calls without clearing
 * 1 <= topk <= EXL3_MAX_TOPK.  t == 0 returns EXL3_OK without work.
 * Out-of-range ids are a contract violation and are not checked by default.
 * With the environment variable EXL3_CHECK_IDS set (not "0"; read at every
 * call), the call first counts the ids outside [0, experts) on the device,
 * waits for that count on the host (so such calls block and cannot be
 * graph-captured), and returns EXL3_E_INVALID, with nothing else enqueued,
 * if there is any.  With EXL3_CHECK_IDS set, a call on a stream that is
 * being captured returns EXL3_E_INVALID without enqueueing anything (the
 * capture stays valid).  The same holds for exl3_grouped_experts_mixed.
 * Small calls (t * topk <= 224) hand partial sums between workgroups planned
 * on one XCD (the XCD each group was finished on in the previous call, kept
 * in the workspace's counters); a workgroup that finds itself on another XCD
 * takes a device-scope release/acquire hand-off instead, so results never
 * depend on the dispatch order.  The environment variable
 * EXL3_FORCE_DEVICE_SCOPE (not "0"; read at every call) makes every
 * workgroup take that hand-off: the results are the same bits, only slower
 * (a debug check of the guard).                                            */
exl3_status exl3_grouped_experts(const exl3_expert_weights* gate_up,
                                 const exl3_expert_weights* down, const void* x,
                                 const int32_t* topk_ids, const float* topk_weights, int64_t t,
                                 int32_t topk, float* y, void* ws, size_t ws_bytes,
                                 exl3_stream_t stream);

/* The widths of an arena whose experts each have their own width
 * (TensorFold issue #832, "Activity": the consolidated module keeps a width
 * per expert in the representation).  The arena record then has bits == 0,
 * and expert e's tensors are bits_host[e] bits wide:
 *   bits_host  int32 [experts] host pointer, each in 1..8; checked on the
 *              host during the call (nothing is enqueued if one is not)
 *   bits       int32 [experts] device pointer, 4-byte aligned, the same
 *              values (read by the kernels)
 *   offsets    int64 [experts] device pointer, 8-byte aligned: the word
 *              index in the arena's trellis where expert e's slot 0 starts,
 *              a multiple of 8; slot s follows at
 *              offsets[e] + s * (k/16) * (n/16) * 16 * bits[e].
 *              Experts may be packed in any order.
 * suh and svh keep the uniform layout [experts][slots][k or n].  Device
 * values that differ from bits_host, or offsets past the trellis allocation,
 * are a contract violation and are not checked on device (a device width
 * outside 1..8 leaves that expert's pairs uncomputed, the output undefined
 * and the workspace to be zero-filled again before its next use).        */
typedef struct exl3_expert_widths {
    const int32_t* bits_host;
    const int32_t* bits;
    const int64_t* offsets;
} exl3_expert_widths;

/* Bytes of device workspace exl3_grouped_experts_mixed needs (0 if
 * invalid); the same figure as for uniform arenas of the same shapes.     */
size_t exl3_grouped_experts_mixed_workspace_size(const exl3_expert_weights* gate_up,
                                                 const exl3_expert_widths* gate_up_widths,
                                                 const exl3_expert_weights* down,
                                                 const exl3_expert_widths* down_widths,
                                                 int64_t t, int32_t topk);

/* exl3_grouped_experts_mixed - exl3_grouped_experts over arenas with a width
 * per expert (gate_up_widths for the gate/up arena, down_widths for the down
 * arena; an expert's gate and up share its width).  Arguments, workspace
 * rules, errors and the result are those of exl3_grouped_experts; each
 * (token, slot) pair is computed by the same kernels and in the same order
 * as a uniform arena of its expert's width would compute it, so when every
 * expert has one width the result is bit-identical to exl3_grouped_experts.
 * Each projection is still one launch: every workgroup reads its expert's
 * width and runs the decode of that width.                                 */
exl3_status exl3_grouped_experts_mixed(const exl3_expert_weights* gate_up,
                                       const exl3_expert_widths* gate_up_widths,
                                       const exl3_expert_weights* down,
                                       const exl3_expert_widths* down_widths, const void* x,
                                       const int32_t* topk_ids, const float* topk_weights,
                                       int64_t t, int32_t topk, float* y, void* ws,
                                       size_t ws_bytes, exl3_stream_t stream);

/* ---------------------------------------------------------------------------
 * MXFP4: microscaled 4-bit floating point (the block format of the OCP
 * Microscaling Formats specification, version 1.0: E2M1 elements, E8M0
 * scales, blocks of 32), the matrix cores' own 4-bit format on gfx950.
 *
 * A matrix of `rows` rows and k columns (k a multiple of 32) is held as
 *   codes   uint8 [rows][k/2], row-major: element 2i of a row in the low half
 *           of byte i, element 2i+1 in the high half.  Bit 3 of a code is the
 *           sign, bits 0..2 name 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   scales  uint8 [rows][k/32], row-major: one byte s per 32 consecutive
 *           elements, the factor 2^(s - 127); 255 is NaN (the whole block)
 * Both device pointers 16-byte aligned.  0 < k < 2^24, 0 <= rows <= 2^24.
 * A weight of a linear layer is stored [out_features][in_features].
 * ------------------------------------------------------------------------ */
#define EXL3_MX4_BLOCK 32

typedef struct exl3_mx4 {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t rows;
    int64_t k;
} exl3_mx4;

/* exl3_mx4_quantize - rows of fp16 or fp32 to MXFP4.
 *   S = 2^(floor(log2 max|x|) - 2) over each block of 32 (the specification's
 *   rule: E2M1's largest exponent is 2), the exponent not below -127;
 *   code = x / S rounded to the nearest E2M1 value, ties to the even code,
 *   magnitudes above 6 to 6; the sign bit is x's, also where x / S rounds to 0
 *   x       [rows][ldx] of `dtype` (EXL3_F16 or EXL3_F32), ldx >= k, multiple
 *           of 8, 16-byte aligned
 *   codes, scales  as above, written whole; they may not overlap x
 * A block of zeros gets scale byte 0.  A block that holds a NaN or an
 * infinity becomes a NaN block: scale byte 255, codes 0.  Every decision is
 * exact, so the output is bit-exact by definition.  rows == 0 returns
 * EXL3_OK.  rows * k at most 2^35 - 2048 (launch size).                    */
exl3_status exl3_mx4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t k, int64_t ldx,
                              uint8_t* codes, uint8_t* scales, exl3_stream_t stream);

/* exl3_mx4_reconstruct - the values an MXFP4 matrix stands for.
 *   out     [rows][ld_out] of `dtype` (EXL3_F16 or EXL3_F32), ld_out >= k,
 *           multiple of 8, 16-byte aligned
 * Values are exact in fp32 except past its range (scale bytes 253 and 254:
 * magnitudes from 2^128 become infinity); fp16 rounds to nearest once.  What
 * exl3_mx4_quantize made of fp16 rows is exact in fp16.  NaN blocks give NaN.
 * rows * k must stay below 2^35.                                           */
exl3_status exl3_mx4_reconstruct(const exl3_mx4* w, void* out, int32_t dtype, int64_t ld_out,
                                 exl3_stream_t stream);

/* Bytes of device workspace exl3_mx4_matmul needs (0 if none is needed, or
 * the arguments are invalid). */
size_t exl3_mx4_matmul_workspace_size(const exl3_mx4* a, const exl3_mx4* b);

/* exl3_mx4_matmul - y = A B^T (+ bias), both operands MXFP4, on the scaled
 * 4-bit matrix cores.  Products are exact, sums fp32, one rounding to an fp16
 * output.
 *   a      [m][k] (rows = m), b [n][k] (rows = n), the same k; m and n any
 *   bias   fp16 [n] device pointer or NULL (added last, in fp32)
 *   y      [m][ldy] of y_dtype (EXL3_F16 or EXL3_F32), ldy >= n; rows need no
 *          alignment beyond the element's own.  y may not overlap an operand
 *   ws     device workspace of at least the queried size (may be NULL when
 *          that is 0), 16-byte aligned: scratch, whatever it holds before and
 *          after.  Calls that overlap in time on one workspace race.
 * m == 0 or n == 0 returns EXL3_OK.  Calls whose launch would not fit the
 * hardware's grid return EXL3_E_INVALID: ceil(m/16) * ceil(n/16) >= 2^26, or,
 * from (m + n) ceil(k/256) >= 2^29 on, ceil(m/64) * ceil(n/32) >= 2^23.
 * Results are the same bits on every run of one shape; a row's result may
 * depend on m (the tile is chosen by size), to rounding.                   */
exl3_status exl3_mx4_matmul(const exl3_mx4* a, const exl3_mx4* b, const uint16_t* bias, void* y,
                            int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                            exl3_stream_t stream);

/* Largest row count of exl3_mx4_linear. */
#define EXL3_MX4_LINEAR_MAX_ROWS 64

/* Bytes of device workspace exl3_mx4_linear needs for m rows (0 if none is
 * needed, or the arguments are invalid). */
size_t exl3_mx4_linear_workspace_size(const exl3_mx4* w, int64_t m);

/* exl3_mx4_linear - y = x W^T (+ bias) for decode and verify batches: fp16
 * activations, unrounded, against MXFP4 weights; products exact in fp32, sums
 * fp32.  For more than EXL3_MX4_LINEAR_MAX_ROWS rows the weights' bytes no
 * longer bound the product: call it for so many at a time, or, where rows rounded
 * to 4 bits will do, quantize them and call exl3_mx4_matmul.
 *   w      [n][k] (rows = n).  Blocks with scale bytes outside 104 .. 140, whose
 *          values fp16 cannot hold, are taken in a second, slower way
 *   x      fp16 [m][ldx], ldx >= k, multiple of 8, 16-byte aligned
 *   bias, y, ldy, y_dtype, ws   as for exl3_mx4_matmul
 * 0 <= m <= EXL3_MX4_LINEAR_MAX_ROWS; m == 0 or n == 0 returns EXL3_OK.
 * Results are the same bits on every run of one shape; a row's result may
 * depend on m, to rounding.                                                */
exl3_status exl3_mx4_linear(const exl3_mx4* w, const uint16_t* bias, const void* x, int64_t m,
                            int64_t ldx, void* y, int64_t ldy, int32_t y_dtype, void* ws,
                            size_t ws_bytes, exl3_stream_t stream);

/* Packed MXFP4 tensors of experts:
 *   codes   uint8 [experts][slots][n][k/2]
 *   scales  uint8 [experts][slots][n][k/32]
 * n and k multiples of 32, at most 65536.                                  */
typedef struct exl3_mx4_experts {
    const uint8_t* codes;
    const uint8_t* scales;
    int32_t experts;
    int32_t slots;
    int32_t n;
    int32_t k;
} exl3_mx4_experts;

/* How a router's logits become choices and weights (l = x W_r^T, b the bias,
 * 0 where there is none):
 *   EXL3_ROUTE_SOFTMAX  chosen by l + b, weight softmax(l + b) over all experts
 *   EXL3_ROUTE_SIGMOID  chosen by sigmoid(l) + b, weight sigmoid(l).  Without a
 *                       bias chosen by l: the same order, where sigmoid(l)
 *                       has not yet rounded to 1                             */
typedef enum exl3_route {
    EXL3_ROUTE_SOFTMAX = 0,
    EXL3_ROUTE_SIGMOID = 1
} exl3_route;

/* One mixture-of-experts layer.
 *   router       fp16 [experts][hidden], row-major, 16-byte aligned
 *   router_bias  fp32 [experts], 4-byte aligned, or NULL
 *   scoring      exl3_route
 *   renormalize  not 0: a token's weights are divided by their sum
 *   scale        factor of the routed weights (after the division)
 *   gate_up      slots == 2 (slot 0 = gate, slot 1 = up), k = hidden,
 *                n = intermediate
 *   down         slots == 1, k = intermediate, n = hidden, as many experts
 *   shared_gate_up, shared_down   the shared expert (experts == 1, slots as
 *                above, its own intermediate width), or codes == NULL in both
 *   shared_gate  fp16 [hidden], 16-byte aligned, or NULL: the shared expert's
 *                weight is sigmoid(x . shared_gate), or 1                    */
typedef struct exl3_mx4_moe_layer {
    const uint16_t* router;
    const float* router_bias;
    int32_t scoring;
    int32_t renormalize;
    float scale;
    exl3_mx4_experts gate_up;
    exl3_mx4_experts down;
    exl3_mx4_experts shared_gate_up;
    exl3_mx4_experts shared_down;
    const uint16_t* shared_gate;
} exl3_mx4_moe_layer;

/* Limits of exl3_mx4_moe. */
#define EXL3_MX4_MOE_MAX_TOKENS 16
#define EXL3_MX4_MOE_MAX_EXPERTS 1024

/* Bytes of device workspace exl3_mx4_moe needs (0 if the arguments are
 * invalid or t == 0). */
size_t exl3_mx4_moe_workspace_size(const exl3_mx4_moe_layer* layer, int64_t t, int32_t topk);

/* exl3_mx4_moe - a whole mixture-of-experts layer for a few tokens:
 *   y[i] = sum over the chosen experts e of w[i][e] * down_e(a_e)
 *          (+ w_s[i] * down_s(a_s)),   a = silu(gate(x_i)) * up(x_i)
 * Activations are not rounded to 4 bits: x enters as fp16, a is held to 24
 * bits, every sum and the routing in fp32.
 *   x             fp16 [t][ldx], ldx >= hidden, multiple of 8, 16-byte aligned
 *   topk          experts per token, 1..min(EXL3_MAX_TOPK, experts); equal
 *                 scores go to the lower expert
 *   y             [t][ldy] of y_dtype (EXL3_F16 or EXL3_F32), ldy >= hidden;
 *                 it may not overlap x
 *   topk_ids      int32 [t][topk] device pointer or NULL: the choices, best
 *                 first
 *   topk_weights  fp32 [t][topk] device pointer or NULL: their weights
 *   ws            device workspace of at least the queried size, 16-byte
 *                 aligned, zero-filled before its first use and then left to
 *                 this entry point, which leaves its arrival counts at zero
 *                 (calls of any layer and size may share it, one after the
 *                 other); calls that overlap on it race
 * 0 <= t <= EXL3_MX4_MOE_MAX_TOKENS, experts <= EXL3_MX4_MOE_MAX_EXPERTS;
 * t == 0 returns EXL3_OK.  A NaN score counts as the lowest, so the ids are
 * always valid; the weights are what the formulas give.  EXL3_ROUTE_SOFTMAX: all
 * of a token's are NaN if an l + b is NaN or +infinity or every one -infinity; a
 * -infinity next to finite ones has weight 0.  EXL3_ROUTE_SIGMOID: 1 for an l of
 * +infinity, 0 for -infinity, NaN for a NaN that is chosen.  Divided by their sum,
 * all are NaN if one is, or if the sum is 0.
 * More tokens are taken EXL3_MX4_MOE_MAX_TOKENS a call (a token's result may depend
 * on the others of its call, to rounding): no entry point takes MXFP4 experts for
 * more at once, and exl3_grouped_experts takes trellis tensors.              */
exl3_status exl3_mx4_moe(const exl3_mx4_moe_layer* layer, const void* x, int64_t t, int64_t ldx,
                         int32_t topk, void* y, int64_t ldy, int32_t y_dtype, int32_t* topk_ids,
                         float* topk_weights, void* ws, size_t ws_bytes, exl3_stream_t stream);

/* ---------------------------------------------------------------------------
 * Routing to experts: from hidden rows or logits to the topk_ids and
 * topk_weights that exl3_grouped_experts takes.
 * ------------------------------------------------------------------------ */
#define EXL3_ROUTE_MAX_EXPERTS 1024
#define EXL3_ROUTE_MAX_GROUPS 64

/* What grades a group of experts. */
typedef enum exl3_group_score {
    EXL3_GROUP_MAX = 0, /* its best choice value */
    EXL3_GROUP_TOP2 = 1 /* the sum of its two best choice values (of its two best
                           scores where there is no balance) */
} exl3_group_score;

/* How logits l become choices and weights:
 *   scores         s = softmax(l) over all experts (EXL3_ROUTE_SOFTMAX) or
 *                  sigmoid(l) (EXL3_ROUTE_SIGMOID)
 *   choice values  v = s + balance, or l itself without a balance (the same order)
 *   groups         experts / groups consecutive experts each, 1 for none; the
 *                  topk_groups best graded ones are kept, equal grades going to the
 *                  lower group
 *   choices        the topk best of the kept groups, best first, equal values going
 *                  to the lower expert
 *   weights        s of the chosen, divided by their sum if renormalize is not 0,
 *                  times scale
 * Here a balance shifts choices only, for softmax scores too; a bias of the router's
 * linear, which shifts logits, is exl3_router_weight's.
 *   balance      fp32 [experts] device pointer, 4-byte aligned, or NULL
 *   experts      1..EXL3_ROUTE_MAX_EXPERTS, a multiple of groups
 *   topk         1..EXL3_MAX_TOPK, at most topk_groups * (experts / groups)
 *   groups       1..EXL3_ROUTE_MAX_GROUPS; EXL3_GROUP_TOP2 needs groups of two
 *   topk_groups  1..groups
 * Without a balance logits are compared as they are.  With one, and for
 * EXL3_GROUP_TOP2, values are computed in 64 bits and compared to 42 significant
 * bits (scores below 10^-300 to fewer), so that choices do not depend on how 32 bits
 * would have rounded.
 * A NaN value counts as the lowest, so the ids are always valid and a token's are
 * distinct.  Weights are what the formulas give: softmax of a token with a NaN or
 * +infinite logit, or with -infinite ones only, is NaN throughout; a -infinite logit
 * next to finite ones has the score 0, for sigmoid too.  They are fp32: a score below
 * 2^-125 is held to 2^-17 of itself, one below 2^-128 is 0 for sigmoid, and weights
 * divided by a sum of 0 are NaN. */
typedef struct exl3_route_rule {
    const float* balance;
    int32_t experts;
    int32_t topk;
    int32_t scoring;
    int32_t groups;
    int32_t topk_groups;
    int32_t group_score;
    int32_t renormalize;
    float scale;
} exl3_route_rule;

/* exl3_route_topk - choices and weights of t tokens from their logits.
 *   logits        [t][ldl] of `dtype` (EXL3_F16 or EXL3_F32), ldl >= experts; rows
 *                 need no alignment beyond the element's own
 *   topk_ids      int32 [t][topk]
 *   topk_weights  fp32 [t][topk]; neither may overlap the logits
 * 0 <= t <= 2^24; t == 0 returns EXL3_OK.  The same bits on every run; a token's
 * result does not depend on the others of its call.                          */
exl3_status exl3_route_topk(const exl3_route_rule* rule, const void* logits, int32_t dtype, int64_t t, int64_t ldl,
                            int32_t* topk_ids, float* topk_weights, exl3_stream_t stream);

/* A router's linear: l = x W^T (+ bias).
 *   weight   fp16 [experts][hidden], row-major, 16-byte aligned
 *   bias     fp32 [experts] device pointer, 4-byte aligned, or NULL
 *   experts  1..EXL3_ROUTE_MAX_EXPERTS
 *   hidden   a multiple of 8, at most 65536                                  */
typedef struct exl3_router_weight {
    const uint16_t* weight;
    const float* bias;
    int32_t experts;
    int32_t hidden;
} exl3_router_weight;

/* Bytes of device workspace exl3_router_linear needs (0 if none is needed, or the
 * arguments are invalid). */
size_t exl3_router_linear_workspace_size(const exl3_router_weight* w, int64_t t);

/* exl3_router_linear - the logits of t tokens: fp16 rows and weights, products exact
 * in fp32, sums fp32, not rounded (products of subnormal elements are summed as if those
 * were 2^-14: alone, they keep fewer bits).
 *   x       fp16 [t][ldx], ldx >= hidden, multiple of 8, 16-byte aligned
 *   logits  fp32 [t][ldl], ldl >= experts, 4-byte aligned; it may not overlap x
 *   ws      device workspace of at least the queried size (may be NULL when that is
 *           0), 16-byte aligned, zero-filled before its first use and then left to
 *           the router's entry points, which leave its arrival counts at zero (calls
 *           of any router and size may share it, one after the other); calls that
 *           overlap on it race
 * 0 <= t <= 2^24; t == 0 returns EXL3_OK.  The same bits on every run of one shape; a
 * row's result may depend on t, to rounding.                                */
exl3_status exl3_router_linear(const exl3_router_weight* w, const void* x, int64_t t, int64_t ldx, float* logits,
                               int64_t ldl, void* ws, size_t ws_bytes, exl3_stream_t stream);

/* Bytes of device workspace exl3_router needs (0 if none is needed, or the arguments
 * are invalid); logits: not 0 if the call is given memory for them. */
size_t exl3_router_workspace_size(const exl3_router_weight* w, int64_t t, int32_t logits);

/* exl3_router - a router's linear and the routing of its logits in one call (one
 * launch for a few tokens).  Arguments and limits are those of exl3_router_linear and
 * exl3_route_topk.  The logits are summed in shares of k of their own: they are
 * exl3_router_linear's to rounding, and choices of values that near may differ from
 * those of the two calls.  The choices and weights are, bit for bit, exl3_route_topk's of
 * the logits that this call gives, whether it stores them or not.
 *   logits  fp32 [t][ldl], or NULL where the caller has no use for them
 *   ws      as for exl3_router_linear, and it may be the same one             */
exl3_status exl3_router(const exl3_router_weight* w, const exl3_route_rule* rule, const void* x, int64_t t,
                        int64_t ldx, float* logits, int64_t ldl, int32_t* topk_ids, float* topk_weights, void* ws,
                        size_t ws_bytes, exl3_stream_t stream);

/* ---------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection.
 * ------------------------------------------------------------------------ */
#define EXL3_LORA_MAX_RANK 256
#define EXL3_LORA_MAX_ADAPTERS 4096

/* A stack of adapters of one projection [k] -> [n]:
 *   a       fp16 [adapters][rank][k], row-major, 16-byte aligned
 *   b       fp16 [adapters][n][rank], row-major, 16-byte aligned
 *   scales  fp32 [adapters] device pointer, 4-byte aligned, or NULL (1)
 *   ranks   int32 [adapters] device pointer, 4-byte aligned, or NULL: the rank of each
 *           adapter, taken between 0 and `rank`; what a and b hold past it has no say
 *   adapters  0..EXL3_LORA_MAX_ADAPTERS (a and b may be NULL when 0)
 *   rank      a multiple of 8, at most EXL3_LORA_MAX_RANK
 *   k, n      at most 2^20, k a multiple of 8                               */
typedef struct exl3_lora_stack {
    const uint16_t* a;
    const uint16_t* b;
    const float* scales;
    const int32_t* ranks;
    int32_t adapters;
    int32_t rank;
    int64_t k;
    int64_t n;
} exl3_lora_stack;

/* Bytes of device workspace exl3_lora needs for m rows (0 if none is needed, or the
 * arguments are invalid). */
size_t exl3_lora_workspace_size(const exl3_lora_stack* l, int64_t m);

/* exl3_lora - y_i = base_i + scale_a B_a (A_a x_i), a = rows[i]: what the adapter of
 * each row's request adds to a projection's output (exl3_linear, exl3_mx4_linear, ...).
 * Products of A are exact in fp32, sums fp32; between the products A x is kept to 23 bits
 * at least (each element within 2^-23 of itself; below 2^-29 of the row's largest, within
 * 2^-51 of that); one rounding to an fp16 output.  The matrix cores sum the product of a
 * subnormal fp16 as if it were one of 2^-14: sums of subnormal elements alone keep fewer
 * bits.
 *   x     fp16 [m][ldx], ldx >= k, multiple of 8, 16-byte aligned
 *   rows  int32 [m] device pointer, 4-byte aligned: each row's adapter; a value outside
 *         0 .. adapters-1 (-1, say) stands for none, and y_i is base_i
 *   base  [m][ldb] of y's type, ldb >= n, or NULL (zeros)
 *   y     [m][ldy] of y_dtype (EXL3_F16 or EXL3_F32), ldy >= n; y may be base itself
 *         (ldb == ldy: added in place, rows without an adapter left alone), but may not
 *         overlap it, x or the adapters otherwise.  Rows of base and y need no alignment
 *         beyond the element's own
 *   ws    device workspace of at least the queried size (may be NULL when that is 0),
 *         16-byte aligned: scratch, whatever it holds before and after.  Calls that
 *         overlap in time on one workspace race.
 * 0 <= m <= 2^24; m == 0 returns EXL3_OK.  A row whose x, base or adapter holds NaN or
 * an infinity gets what the formula gives; other rows are not touched by it.  The same
 * bits on every run of one shape and assignment of rows; a row's result may depend on
 * the others', to rounding.                                                  */
exl3_status exl3_lora(const exl3_lora_stack* l, const void* x, int64_t m, int64_t ldx, const int32_t* rows,
                      const void* base, int64_t ldb, void* y, int64_t ldy, int32_t y_dtype, void* ws, size_t ws_bytes,
                      exl3_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_H */

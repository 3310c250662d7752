/*
 * moeq.h -- C ABI of libmoeq: NF4 / row-wise int8 quantization of fused MoE
 * expert tensors and the routed experts forward straight from the packed
 * storage, on AMD Instinct MI355X (gfx950).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every data pointer is a DEVICE pointer to caller-owned memory.  The
 *   library allocates nothing and keeps no state between calls.
 * - Calls are asynchronous on `stream` (a hipStream_t; NULL is the default
 *   stream).  MOEQ_OK means validation passed and every kernel was enqueued;
 *   a HIP launch error maps to MOEQ_EDEVICE.  No call synchronises the host.
 * - All validation happens on the host before any HIP call, so a rejected
 *   call has no side effect.  No call ever no-ops silently on bad input: the
 *   pages describe expert tensors silently left unquantized, and a packed
 *   uint8 tensor silently reaching a float kernel, as the failures to avoid
 *   (bitsandbytes issue #1849, comment thread; unsloth-zoo issue #850).
 * - Tensors are row-major and contiguous.  An expert tensor is
 *   [E][rows][cols] with each [e] slice an [out_features, in_features]
 *   weight: gate_up_proj is [E][2I][H] and down_proj is [E][H][I]
 *   (bitsandbytes issue #1849, Description code and maintainer thread).
 * - bf16 values travel as their uint16_t bit patterns.
 */
#ifndef MOEQ_H
#define MOEQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOEQ_ABI_VERSION 3
#define MOEQ_NF4_BLOCKSIZE 64
#define MOEQ_DQ_GROUP 256 /* NF4 blocks per double-quantization group */
#define MOEQ_MXFP4_BLOCKSIZE 32
#define MOEQ_FP8_BLOCKSIZE 128
#define MOEQ_MAX_EXPERTS 1024

typedef int32_t moeq_status;
enum {
  MOEQ_OK = 0,
  MOEQ_EINVAL = -1,     /* null pointer, a dimension <= 0, K < 1, T < 0, scale_codes
                           set for a format without them (or missing for NF4_DQ)   */
  MOEQ_ESHAPE = -2,     /* gate_up / down / hidden dimensions inconsistent          */
  MOEQ_EBLOCK = -3,     /* NF4: blocksize != 64 or cols % 64 != 0; int8: blocksize != cols */
  MOEQ_EFORMAT = -4,    /* format tag not what the call needs, or gate_up and down differ */
  MOEQ_EALIGN = -5,     /* a pointer is not 16-byte aligned                          */
  MOEQ_EWORKSPACE = -6, /* workspace null or smaller than moeq_experts_forward_workspace_bytes */
  MOEQ_EDEVICE = -7     /* a HIP call failed                                         */
};

enum {
  MOEQ_FMT_NF4 = 1,
  MOEQ_FMT_INT8_ROWWISE = 2,
  MOEQ_FMT_NF4_DQ = 3,
  MOEQ_FMT_MXFP4 = 4,
  MOEQ_FMT_FP8_ROW = 5,
  MOEQ_FMT_FP8_TILE = 6
};

/* Element types of gradients. */
enum { MOEQ_DTYPE_BF16 = 1, MOEQ_DTYPE_FP32 = 2 };

/*
 * A quantized expert tensor [E][rows][cols] in caller-owned device memory.
 *
 * NF4 (format MOEQ_FMT_NF4, blocksize 64; "MoE Expert Quantization",
 * Implementation details: 4-bit mode is NF4; bitsandbytes issue #1849,
 * maintainer thread: plain packed storage plus a module-owned absmax
 * [num_experts, blocks_per_expert], in_features divisible by the blocksize):
 *   qdata  uint8 [E][rows][cols/2]; column 2m in the high nibble of byte m,
 *          column 2m+1 in the low nibble.
 *   scales fp32 [E][rows*cols/64]: the absmax of each 64-element block along
 *          a row, blocks in row order.
 * int8 row-wise (format MOEQ_FMT_INT8_ROWWISE, blocksize == cols;
 * "MoE Expert Quantization", Implementation details: 8-bit mode is a
 * row-wise int8 parametrization):
 *   qdata  int8 [E][rows][cols], codes in [-127, 127].
 *   scales fp32 [E][rows]: absmax(row) / 127.
 * NF4 with double-quantized absmax (format MOEQ_FMT_NF4_DQ, blocksize 64;
 * bitsandbytes issue #1849, Reproduction: the 4-bit config turns double
 * quantization on; maintainer thread: per-expert compress_statistics, the
 * absmax itself quantized, deferred from the first version; the pages fix
 * no format, this one is the library's own):
 *   qdata        as for NF4.
 *   scale_codes  uint8 [E][nb], nb = rows*cols/64: absmax code c of each
 *                block, c = round_half_even(fp32(fp32(255 a) / m)).
 *   scales       fp32 [E][ceil(nb/256)]: group scale s2 = fp32(m / 255),
 *                m the largest absmax of the group (groups of MOEQ_DQ_GROUP
 *                consecutive blocks of one expert, the last one possibly
 *                shorter; an all-zero group stores s2 = 0 and codes 0).
 *   The weights decode with absmax' = fp32(c * s2).
 * MXFP4 (format MOEQ_FMT_MXFP4, blocksize 32; the microscaled 4-bit floating
 * point of the OCP Microscaling specification):
 *   qdata        uint8 [E][rows][cols/2]: E2M1 codes (sign, two exponent bits,
 *                one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 in magnitude);
 *                column 2m in the LOW nibble of byte m, column 2m+1 in the
 *                high nibble.
 *   scale_codes  uint8 [E][rows*cols/32]: one byte s per block of 32 columns,
 *                the scale 2^(s - 127); s = 255 makes the whole block NaN.
 *   scales       NULL.
 * FP8 (blocksize 128, cols % 16 == 0): E4M3 codes (OCP 8-bit floating point,
 * three fraction bits, 448 the largest, no infinities) with an fp32 scale for
 * each 128 columns of a row (format MOEQ_FMT_FP8_ROW, for activations) or each
 * 128 x 128 tile of an expert (MOEQ_FMT_FP8_TILE, for weights); last blocks and
 * tiles may be smaller:
 *   qdata        uint8 [E][rows][cols]: codes.
 *   scales       fp32 [E][rows][ceil(cols/128)], or
 *                fp32 [E][ceil(rows/128)][ceil(cols/128)].
 *   scale_codes  NULL.
 * Since blocks and groups never straddle an expert, &qdata[e] / &scales[e]
 * (and &scale_codes[e]) with num_experts = 1 describe expert e alone.
 * scale_codes must be NULL for plain NF4 and int8.
 * The experts and offload calls below take NF4, NF4_DQ and int8 tensors;
 * MXFP4 and FP8 tensors belong to the calls that name the format, and any other
 * call returns MOEQ_EFORMAT.  Those calls return MOEQ_ESHAPE for a tensor of
 * more than 2^40 blocks.
 */
typedef struct moeq_qweight {
  int32_t format;
  int32_t num_experts;
  int32_t rows;
  int32_t cols;
  int32_t blocksize;
  void *qdata;
  float *scales;
  uint8_t *scale_codes;
} moeq_qweight;

/* Version of this ABI (MOEQ_ABI_VERSION). */
int32_t moeq_abi_version(void);

/* Static, NUL-terminated description of a status code. */
const char *moeq_status_string(moeq_status status);

/*
 * Host copy of the 16 NF4 levels the kernels use (ascending, fp32), written
 * to out[0..15].  The pages name the NF4 format without printing it; the
 * levels are the QLoRA NormalFloat construction (evenly spaced standard-
 * normal quantiles, zero exactly representable, extremes -1 and +1).
 * Host-only; makes no HIP call.  MOEQ_EINVAL if out is NULL.
 */
moeq_status moeq_nf4_codebook(float *out);

/*
 * Quantize-on-load, 4-bit ("MoE Expert Quantization", intro and
 * Implementation details; bitsandbytes issue #1849, maintainer thread).
 * w_bf16: bf16 [E][rows][cols] (16-byte aligned); dst describes the output
 * and must have format MOEQ_FMT_NF4 or MOEQ_FMT_NF4_DQ, blocksize 64,
 * cols % 64 == 0, and 16-byte aligned qdata/scales/scale_codes.  For each
 * 64-block: absmax = max |w|; n = fp32(w / absmax) (IEEE division); code =
 * nearest NF4 level, an exact tie to the lower index; an all-zero block
 * stores absmax 0 and code 7.  With MOEQ_FMT_NF4_DQ the absmax is then
 * double-quantized in the same pass (as moeq_compress_absmax would); the
 * 4-bit codes are those of the plain format.
 * The source may be freed (stream-ordered) as soon as the call returns.
 * Preconditions not checked on device: finite weights.
 */
moeq_status moeq_quantize_nf4(const uint16_t *w_bf16, const moeq_qweight *dst, void *stream);

/*
 * Measurement reference, not part of the method: the launch shape, loads and
 * stores of moeq_quantize_nf4 on a plain NF4 tensor (every bf16 element read
 * once with the same 16-byte loads, 0.5 B of codes and 4/64 B of absmax
 * written per element) with the NF4 decision replaced by an XOR fold, so its
 * rate is the bandwidth attainable with the quantize kernel's byte mix and
 * access pattern.  Same arguments and checks as moeq_quantize_nf4 (format
 * MOEQ_FMT_NF4 only); the bytes it writes into dst are meaningless.
 */
moeq_status moeq_stream_reference(const uint16_t *w_bf16, const moeq_qweight *dst, void *stream);

/*
 * Quantize-on-load, 8-bit ("MoE Expert Quantization", Implementation
 * details: row-wise int8 parametrization).  dst: format
 * MOEQ_FMT_INT8_ROWWISE, blocksize == cols, cols % 8 == 0.  Per row:
 * absmax = max |w|; scale = fp32(absmax / 127); q = round-half-even of
 * fp32(fp32(127 w) / absmax); a zero row gives scale 0 and q 0.
 * Preconditions not checked on device: finite weights, |w| < 2^120.
 */
moeq_status moeq_quantize_int8_rowwise(const uint16_t *w_bf16, const moeq_qweight *dst, void *stream);

/*
 * Double-quantize the absmax of an NF4 tensor (bitsandbytes issue #1849,
 * Reproduction and maintainer thread: double quantization, the absmax
 * itself quantized).  src: MOEQ_FMT_NF4; dst: MOEQ_FMT_NF4_DQ of the same
 * shape.  dst->qdata may be src->qdata (the 4-bit codes are shared) or
 * another buffer (they are copied).  Codes and group scales as described
 * at moeq_qweight.  Preconditions not checked on device: finite absmax >= 0.
 */
moeq_status moeq_compress_absmax(const moeq_qweight *src, const moeq_qweight *dst, void *stream);

/*
 * Dequantize (bitsandbytes issue #1849, maintainer thread: the
 * correctness-first path dequantizes the experts; "MoE Expert
 * Quantization", Implementation details: int8 is dequantized for the
 * forward).  out_bf16: bf16 [E][rows][cols], 16-byte aligned.
 * NF4: out = bf16_rne(fp32(level[code] * absmax)); int8: out =
 * bf16_rne(fp32(q * scale)) -- the fp32 product first, then round to bf16.
 * NF4 with double-quantized absmax: as NF4 with absmax' = fp32(c * s2).
 */
moeq_status moeq_dequantize(const moeq_qweight *src, uint16_t *out_bf16, void *stream);

/*
 * Device workspace moeq_experts_forward needs for T tokens and top-K routing
 * over these weights (an upper bound independent of the routing); 0 if the
 * arguments are invalid.  Host-only.
 */
size_t moeq_experts_forward_workspace_bytes(int32_t T, int32_t K, const moeq_qweight *gate_up,
                                            const moeq_qweight *down);

/*
 * Routed experts forward from packed storage (unsloth-zoo issue #850,
 * Suggested fix: the (hidden_states, top_k_index, top_k_weights) interface
 * is uniform across fused-expert architectures; bitsandbytes issue #1849,
 * Description: gate_up_proj [E, 2I, H], down_proj [E, H, I], act_fn).
 *   hidden_bf16   bf16 [T][H]
 *   top_k_index   int32 [T][K]; entries outside [0, E) are not routed and
 *                 contribute nothing; a repeated expert counts per occurrence
 *   top_k_weights fp32 [T][K], used as given
 *   gate_up       [E][2I][H]: rows 0..I-1 are the gate, rows I..2I-1 the up
 *                 projection; down [E][H][I]; both of one format (NF4,
 *                 NF4 with double-quantized absmax, or int8)
 *   out_bf16      bf16 [T][H]:
 *                 out[t] = sum_k w[t,k] * down[e] @ (silu(gate[e] x_t) * up[e] x_t)
 *                 with the k terms added in order k = 0..K-1 in fp32
 *                 (deterministic, bit-identical run to run); above 512
 *                 assignments each weighted term is first rounded to bf16.
 *   workspace     device memory of at least
 *                 moeq_experts_forward_workspace_bytes(T, K, gate_up, down).
 * Weights are dequantized tile by tile inside the kernels (bf16 operands,
 * fp32 accumulation); no dequantized tensor is materialised.  T == 0 is a
 * valid no-op.  MOEQ_ESHAPE unless H and I are multiples of 64, T*K <= 2^24
 * and hidden_states is smaller than 4 GiB.
 */
moeq_status moeq_experts_forward(const uint16_t *hidden_bf16, const int32_t *top_k_index,
                                 const float *top_k_weights, int32_t T, int32_t K,
                                 const moeq_qweight *gate_up, const moeq_qweight *down,
                                 uint16_t *out_bf16, void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * moeq_experts_forward with stage timing: stage_events is NULL or an array of
 * 5 hipEvent_t (created by the caller) recorded on `stream` before routing,
 * after routing, after the gate_up GEMM, after the down GEMM and after the
 * combine, so the caller can time each stage with hipEventElapsedTime.
 * Otherwise identical to moeq_experts_forward.
 */
moeq_status moeq_experts_forward_timed(const uint16_t *hidden_bf16, const int32_t *top_k_index,
                                       const float *top_k_weights, int32_t T, int32_t K,
                                       const moeq_qweight *gate_up, const moeq_qweight *down,
                                       uint16_t *out_bf16, void *workspace, size_t workspace_bytes,
                                       void *stream, void *const *stage_events);

/*
 * moeq_experts_forward for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same arguments, kernels and results, without the
 * workspace argument.  The workspace is a device array inside the library of
 * MOEQ_NOALLOC_SCRATCH_BYTES (64 MiB), which each GPU the library runs on
 * holds until the process ends; its address on the current device is looked
 * up on the first call there (the stream must belong to the current device).
 * The call allocates nothing.  MOEQ_EWORKSPACE when
 * moeq_experts_forward_workspace_bytes(T, K, gate_up, down) exceeds the array
 * (the largest batches that fit: 818 tokens of an OLMoE-shaped layer at
 * top-8, 744 of a Mixtral-shaped one at top-2; every few-assignment batch
 * fits).  Every call on one GPU
 * shares that GPU's array: calls that overlap in time on one GPU (different
 * streams, or threads) race and must be serialised by the caller.  Nothing
 * in the array needs clearing between calls (every byte the forward reads is
 * written earlier in the same call).
 */
#define MOEQ_NOALLOC_SCRATCH_BYTES (64u << 20)
moeq_status moeq_experts_forward_noalloc(const uint16_t *hidden_bf16, const int32_t *top_k_index,
                                         const float *top_k_weights, int32_t T, int32_t K,
                                         const moeq_qweight *gate_up, const moeq_qweight *down,
                                         uint16_t *out_bf16, void *stream);

/*
 * Gradients of the routed experts block with respect to its inputs, the
 * packed weights frozen: the workload the quantized experts serve is adapter
 * training over frozen 4-bit/8-bit experts ("MoE Expert Quantization",
 * Axolotl docs, intro and Expert LoRA targeting; Axolotl issue #3787, Use
 * case).  With out = moeq_experts_forward(...) and the incoming gradient
 * grad_out = dL/dout (bf16 [T][H]):
 *   grad_hidden_bf16   bf16 [T][H]: dL/dhidden = sum_k (gate^T dg + up^T du),
 *                      added in k order, with dh = w * down^T grad_out_t,
 *                      dg = dh u s (1 + g (1 - s)), du = dh g s,
 *                      s = sigmoid(g), g / u the gate / up projections
 *   grad_weights       fp32 [T][K]: dL/dw[t,k] = grad_out_t . (down h),
 *                      formed as (down^T grad_out_t) . h from the down^T
 *                      product that dh needs; 0 for an unrouted assignment
 * Same arguments and rules as moeq_experts_forward otherwise; the forward's
 * gate_up GEMM is recomputed inside (g, u and h are not taken from a previous
 * call).  Roundings: h and dg/du feed bf16 MFMA operands; every sum is fp32;
 * deterministic (no float atomics).  workspace: at least
 * moeq_experts_backward_workspace_bytes(T, K, gate_up, down) bytes.
 * MOEQ_ESHAPE additionally unless T*K*2I*2 bytes < 4 GiB.
 */
size_t moeq_experts_backward_workspace_bytes(int32_t T, int32_t K, const moeq_qweight *gate_up,
                                             const moeq_qweight *down);
moeq_status moeq_experts_backward(const uint16_t *hidden_bf16, const int32_t *top_k_index,
                                  const float *top_k_weights, int32_t T, int32_t K,
                                  const moeq_qweight *gate_up, const moeq_qweight *down,
                                  const uint16_t *grad_out_bf16, uint16_t *grad_hidden_bf16,
                                  float *grad_weights, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * Training pair without the backward's recompute of the gate_up GEMM, for
 * adapter training over frozen quantized experts ("MoE Expert Quantization",
 * Axolotl docs, Expert LoRA targeting; Axolotl issue #3787, Use case) when
 * the memory for the pre-activations is there.  moeq_experts_forward_save is
 * moeq_experts_forward that also writes, for every routed assignment, the
 * fp32 g = gate[e] x_t and u = up[e] x_t; moeq_experts_backward_saved takes
 * them in place of its recompute.  The chain rule, roundings and order are
 * moeq_experts_backward's, and both calls group the assignments in the same
 * deterministic order, so the gradients equal moeq_experts_backward's bit
 * for bit.
 *   gu_saved  fp32 [T*K][2I], caller-owned, 16-byte aligned: row p holds g
 *             (columns 0..I-1) then u (I..2I-1) of the p-th assignment in
 *             the expert-major stable order of moeq_route_buckets' perm;
 *             rows past the routed count are not written.  It must come from
 *             moeq_experts_forward_save with the same top_k_index, hidden
 *             states and gate_up (not checked).
 * moeq_experts_forward_save takes the tiled path for every batch size (for
 * T*K <= 512 moeq_experts_forward takes the few-assignment path, whose
 * output then agrees within rounding, not bit for bit); its workspace is
 * moeq_experts_forward_workspace_bytes.  The backward needs no hidden
 * states; its workspace, moeq_experts_backward_saved_workspace_bytes, has
 * no g|u region.  Both return MOEQ_ESHAPE where moeq_experts_backward does.
 */
moeq_status moeq_experts_forward_save(const uint16_t *hidden_bf16, const int32_t *top_k_index,
                                      const float *top_k_weights, int32_t T, int32_t K,
                                      const moeq_qweight *gate_up, const moeq_qweight *down, uint16_t *out_bf16,
                                      float *gu_saved, void *workspace, size_t workspace_bytes, void *stream);
size_t moeq_experts_backward_saved_workspace_bytes(int32_t T, int32_t K, const moeq_qweight *gate_up,
                                                   const moeq_qweight *down);
moeq_status moeq_experts_backward_saved(const int32_t *top_k_index, const float *top_k_weights, int32_t T,
                                        int32_t K, const moeq_qweight *gate_up, const moeq_qweight *down,
                                        const float *gu_saved, const uint16_t *grad_out_bf16,
                                        uint16_t *grad_hidden_bf16, float *grad_weights, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * Router front-end producing the experts' (top_k_index, top_k_weights): the
 * gate weight mlp.gate.weight stays bf16 beside the quantized experts
 * ("MoE Expert Quantization", Axolotl docs, Expert LoRA targeting;
 * bitsandbytes issue #1849, maintainer thread: router-only training over
 * NF4 experts) and feeds the uniform experts interface (unsloth-zoo issue
 * #850, Suggested fix).
 *   hidden_bf16    bf16 [T][H], 16-byte aligned
 *   gate_bf16      bf16 [E][H] (one row per expert), 16-byte aligned
 *   logits         gate @ x_t: bf16 operands, fp32 accumulation
 *   top_k_index    int32 [T][K]: the K largest logits, largest first, equal
 *                  logits to the lower expert index
 *   top_k_weights  fp32 [T][K]: softmax over all E of the selected logits;
 *                  with renormalize != 0 divided by their sum (a softmax
 *                  over the K selected logits)
 * Deterministic.  MOEQ_ESHAPE unless H % 64 == 0 and 1 <= K <= E <=
 * MOEQ_MAX_EXPERTS; T == 0 is a valid no-op.
 */
moeq_status moeq_router_topk(const uint16_t *hidden_bf16, const uint16_t *gate_bf16, int32_t T, int32_t H,
                             int32_t E, int32_t K, int32_t renormalize, int32_t *top_k_index,
                             float *top_k_weights, void *stream);

/*
 * Router front-end fused with the routing stage: the same logits, top-K and
 * weights as moeq_router_topk, and from the same selections the grouping of
 * the T*K assignments a = t*K + k by expert that moeq_route_buckets computes
 * (unsloth-zoo issue #850, Suggested fix: one generic routing behind the
 * uniform (hidden_states, top_k_index, top_k_weights) interface; "MoE Expert
 * Quantization", Axolotl docs, Expert LoRA targeting: the router
 * mlp.gate.weight beside the quantized experts).  The router's workgroups
 * rank their own selections (stable, by assignment order) as they make them,
 * so top_k_index is not read back; a per-expert scan and a scatter follow.
 *   top_k_index, top_k_weights  as for moeq_router_topk ([T][K])
 *   counts  int32 [E], offsets int32 [E+1], perm int32 [T*K], slot int32 [T*K]:
 *           as for moeq_route_buckets (every selection is routed, so perm is
 *           a full permutation and no slot is -1)
 *   workspace  device memory of moeq_router_route_workspace_bytes(T, H, E, K)
 * Bit-identical to moeq_router_topk followed by moeq_route_buckets.
 * MOEQ_ESHAPE unless H % 64 == 0, 1 <= K <= min(E, 64), E <= MOEQ_MAX_EXPERTS
 * and T*K <= 2^24; T == 0 writes zero counts and offsets.
 */
size_t moeq_router_route_workspace_bytes(int32_t T, int32_t H, int32_t E, int32_t K);
moeq_status moeq_router_route(const uint16_t *hidden_bf16, const uint16_t *gate_bf16, int32_t T, int32_t H,
                              int32_t E, int32_t K, int32_t renormalize, int32_t *top_k_index,
                              float *top_k_weights, int32_t *counts, int32_t *offsets, int32_t *perm,
                              int32_t *slot, void *workspace, size_t workspace_bytes, void *stream);

/*
 * moeq_experts_forward with the routing already done: offsets, perm and slot
 * are the grouping of this top_k_index by expert (as moeq_router_route or
 * moeq_route_buckets wrote it), so the routing stage is skipped.  Same
 * arguments, workspace, rules and results as moeq_experts_forward (the
 * output is bit-identical).  Preconditions not checked on device: the
 * routing buffers belong to this top_k_index.
 */
moeq_status moeq_experts_forward_routed(const uint16_t *hidden_bf16, const int32_t *top_k_index,
                                        const float *top_k_weights, int32_t T, int32_t K,
                                        const moeq_qweight *gate_up, const moeq_qweight *down,
                                        const int32_t *offsets, const int32_t *perm, const int32_t *slot,
                                        uint16_t *out_bf16, void *workspace, size_t workspace_bytes,
                                        void *stream);

/*
 * Asynchronous copy of one packed expert tensor (codes and scales) between
 * host and device memory, in either direction, on `stream`: the building
 * block of expert-granularity offload, where every layer's packed experts
 * live in pinned host memory, one layer is resident and layer N+1 is
 * prefetched on a side stream during layer N (Axolotl issue #3787, Proposed
 * shape; Evidence: the forward is bit-identical with offload on or off).
 * src and dst must describe the same format and shape (codes, scales and,
 * for MOEQ_FMT_NF4_DQ, absmax codes are copied); their pointers may be
 * pinned host memory (allocated pinned, e.g. hipHostMalloc) or device
 * memory.  The copy is ordered on `stream` like any other call; the caller
 * makes the compute stream wait (an event) before using dst.
 */
moeq_status moeq_qweight_copy_async(const moeq_qweight *src, const moeq_qweight *dst, void *stream);

/*
 * The routing stage of moeq_experts_forward on its own (same kernels):
 * groups the T*K assignments a = t*K + k by expert (unsloth-zoo issue #850,
 * Suggested fix: one generic routing for every architecture).
 *   counts  int32 [E]    assignments per expert
 *   offsets int32 [E+1]  exclusive prefix sum of counts
 *   perm    int32 [T*K]  assignments sorted by expert, ascending a within an
 *                        expert; entries past offsets[E] are left untouched
 *   slot    int32 [T*K]  position of a in perm, -1 for an unrouted a
 * Needs T*K <= 2^24 and E <= MOEQ_MAX_EXPERTS; workspace as for the forward
 * (moeq_experts_forward_workspace_bytes with any weights of E experts) or
 * moeq_route_workspace_bytes(T, K, E).
 */
size_t moeq_route_workspace_bytes(int32_t T, int32_t K, int32_t E);
moeq_status moeq_route_buckets(const int32_t *top_k_index, int32_t T, int32_t K, int32_t E,
                               int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *slot,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * Quantize to MXFP4: w_bf16 bf16 [E][rows][cols] (16-byte aligned; weights,
 * or activations with E = 1); dst format MOEQ_FMT_MXFP4, blocksize 32,
 * cols % 32 == 0, 16-byte aligned qdata and scale_codes.  For each block of
 * 32 columns: s = max(floor(log2(max |w|)) - 2, -127) + 127, code = the E2M1
 * value nearest to w * 2^(127 - s), ties to the even code, at most 6 in
 * magnitude; an all-zero block stores s = 0 and zero codes.  A block with an
 * infinity or a NaN stores s = 255 (NaN) and zero codes.  MOEQ_EINVAL for
 * buffers that overlap, here and in moeq_dequantize_mxfp4.
 */
moeq_status moeq_quantize_mxfp4(const uint16_t *w_bf16, const moeq_qweight *dst, void *stream);

/*
 * MXFP4 -> bf16 [E][rows][cols], 16-byte aligned: E2M1 value * 2^(s - 127),
 * exact (s >= 253, which moeq_quantize_mxfp4 never writes, can overflow to
 * infinities); NaN for s = 255.
 */
moeq_status moeq_dequantize_mxfp4(const moeq_qweight *src, uint16_t *out_bf16, void *stream);

/*
 * Matrix products grouped by expert, for rows sorted by expert: what trains
 * or serves expert weights and per-expert adapters in bf16 beside the packed
 * ones ("MoE Expert Quantization", Axolotl docs, Expert LoRA targeting).
 * Rows p with offsets[e] <= p < offsets[e + 1] belong to expert e:
 *   moeq_grouped_mm              out[p] = w[e] x[p]
 *   moeq_grouped_mm_grad_input   grad_x[p] = w[e]^T grad_out[p]
 *   moeq_grouped_mm_grad_weight  grad_w[e] = sum over p of grad_out[p] x[p]^T
 *   x, grad_x      bf16 [M][K]
 *   w              bf16 [E][N][K]
 *   out, grad_out  bf16 [M][N]
 *   grad_w         fp32 (dtype MOEQ_DTYPE_FP32) or bf16 (MOEQ_DTYPE_BF16)
 *                  [E][N][K]; zeros for an expert without rows
 *   offsets        int32 [E+1] on the device, ascending, as
 *                  moeq_route_buckets and moeq_router_route write them
 *   workspace      of moeq_grouped_mm_grad_weight_workspace_bytes(M, E, N, K),
 *                  16-byte aligned: the rows of an expert that has many are
 *                  summed in segments (none, and NULL, where that is 0)
 * Products of bf16 values summed in fp32, rounded once at the end; the same
 * bits from run to run.  Rows of out and grad_x outside [offsets[0],
 * offsets[E]) are not written, and rows outside an expert's range never
 * reach its results (they may hold anything).  Offsets are clamped to
 * [0, M]; ones that do not ascend give undefined results, but no access
 * outside the arrays.  Every pointer 16-byte aligned, except offsets.
 * MOEQ_EINVAL for a result that overlaps an operand or the workspace.
 * MOEQ_ESHAPE unless N and K are multiples of 8 of at most 2^20, N*K*2 < 2^31,
 * E <= MOEQ_MAX_EXPERTS, M <= 2^28 and the tiles fit one launch:
 * (M/256 + E)(N/256 + 1) < 6.7e6, and for K <= 64 (M/64 + E)(N/128 + 1) <
 * 1.3e7 (N and K exchanged for the input gradient).  M == 0 is a valid no-op,
 * except that moeq_grouped_mm_grad_weight then writes zeros.
 */
moeq_status moeq_grouped_mm(const uint16_t *x_bf16, const uint16_t *w_bf16, const int32_t *offsets, int32_t M,
                            int32_t E, int32_t N, int32_t K, uint16_t *out_bf16, void *stream);
moeq_status moeq_grouped_mm_grad_input(const uint16_t *grad_out_bf16, const uint16_t *w_bf16, const int32_t *offsets,
                                       int32_t M, int32_t E, int32_t N, int32_t K, uint16_t *grad_x_bf16,
                                       void *stream);
moeq_status moeq_grouped_mm_grad_weight(const uint16_t *grad_out_bf16, const uint16_t *x_bf16, const int32_t *offsets,
                                        int32_t M, int32_t E, int32_t N, int32_t K, int32_t dtype, void *grad_w,
                                        void *workspace, size_t workspace_bytes, void *stream);
size_t moeq_grouped_mm_grad_weight_workspace_bytes(int32_t M, int32_t E, int32_t N, int32_t K);

/*
 * moeq_grouped_mm with both operands in MXFP4: x one "expert" of M rows
 * ([1][M][K], activations quantized with moeq_quantize_mxfp4), w [E][N][K].
 * The block scales are applied inside the matrix instructions; products are
 * summed in fp32 and rounded once to bf16.  A NaN block makes the outputs
 * that it enters NaN.  Otherwise as moeq_grouped_mm, with K % 32 == 0; x with
 * rows == 0 (its data pointers may then be NULL) is a valid no-op.
 */
moeq_status moeq_grouped_mm_mxfp4(const moeq_qweight *x, const moeq_qweight *w, const int32_t *offsets,
                                  uint16_t *out_bf16, void *stream);

/*
 * Quantize to FP8: w_bf16 bf16 [E][rows][cols] (16-byte aligned; weights, or
 * activations with E = 1); dst of format MOEQ_FMT_FP8_ROW or MOEQ_FMT_FP8_TILE
 * says what shares a scale, 16-byte aligned qdata.  For each block, amax its
 * largest magnitude: scale = fp32(amax / 448), code = the E4M3 value nearest to
 * 448 w / amax, ties to the even code; a block of zeros stores scale 0 and zero
 * codes (of either sign).  A block with an infinity or a NaN stores a NaN scale and
 * zero codes.  (Below amax = 2^-117 the scale is subnormal and loses bits.)
 * MOEQ_EINVAL for buffers that overlap, here and in moeq_dequantize_fp8.
 */
moeq_status moeq_quantize_fp8(const uint16_t *w_bf16, const moeq_qweight *dst, void *stream);

/* FP8 -> bf16 [E][rows][cols], 16-byte aligned: bf16_rne(fp32(code * scale)). */
moeq_status moeq_dequantize_fp8(const moeq_qweight *src, uint16_t *out_bf16, void *stream);

/*
 * moeq_grouped_mm with both operands in FP8: x one "expert" of M rows
 * ([1][M][K], MOEQ_FMT_FP8_ROW), w [E][N][K] of MOEQ_FMT_FP8_TILE.  The codes'
 * products are summed over each block of 128 columns, multiplied by fp32(x's
 * scale * w's scale) and added in fp32; the result is rounded once to bf16.
 * The sums are fp32 ones, but for the 8-bit matrix instructions' alignment:
 * eight consecutive products are cut off at 2^-13 of the largest one's power of
 * two.  A block with a NaN scale makes the outputs that it enters NaN.
 * Otherwise as moeq_grouped_mm; x with rows == 0 (its data pointers may then be
 * NULL) is a valid no-op.
 */
moeq_status moeq_grouped_mm_fp8(const moeq_qweight *x, const moeq_qweight *w, const int32_t *offsets,
                                uint16_t *out_bf16, void *stream);

/*
 * The gated feed-forward block of experts over rows sorted by expert, in bf16:
 * moeq_experts_forward's block for experts that are trained rather than frozen
 * and packed ("MoE Expert Quantization", Axolotl docs, Expert LoRA targeting).
 * For rows p with offsets[e] <= p < offsets[e + 1]:
 *   g | u   = gate_up[e] x[p]          out[p] = down[e] h,  h = silu(g) * u
 *   x, out    bf16 [M][H]
 *   gate_up   bf16 [E][2I][H]: rows 0..I-1 the gate, I..2I-1 the up projection
 *   down      bf16 [E][H][I]
 *   offsets   int32 [E+1] on the device, as for moeq_grouped_mm
 *   gu_saved  NULL, or fp32 [M][2I] for g | u, which the backward pass takes
 *   workspace of moeq_grouped_ffn_workspace_bytes(M, E, H, I), 16-byte aligned
 * g, u and the sums are fp32; h is rounded to bf16 for the down product.  The
 * same bits from run to run.  Rows of out and gu_saved outside [offsets[0],
 * offsets[E]) are not written, and such rows of x never reach a result.
 * Alignment, overlaps and offsets that do not ascend as for moeq_grouped_mm.
 * MOEQ_ESHAPE unless moeq_grouped_mm and moeq_grouped_mm_grad_input take both
 * products (H and I multiples of 8, 4*I*H < 2^31).  M == 0 is a valid no-op.
 */
size_t moeq_grouped_ffn_workspace_bytes(int32_t M, int32_t E, int32_t H, int32_t I);
moeq_status moeq_grouped_ffn(const uint16_t *x_bf16, const uint16_t *gate_up_bf16, const uint16_t *down_bf16,
                             const int32_t *offsets, int32_t M, int32_t E, int32_t H, int32_t I, float *gu_saved,
                             uint16_t *out_bf16, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Its gradients for the incoming grad_out = dL/dout, bf16 [M][H], from the same
 * x, gate_up, down and offsets and the forward's gu_saved:
 *   dh = down[e]^T grad_out[p]    s = 1 / (1 + exp(-g))
 *   dg = dh u s (1 + g (1 - s))   du = dh g s
 *   grad_x        bf16 [M][H]: gate_up[e]^T (dg | du)
 *   grad_gate_up  [E][2I][H]: sum over the expert's rows of (dg | du) x[p]^T
 *   grad_down     [E][H][I]: sum of grad_out[p] h^T, h from the saved g and u
 *                 both fp32 (dtype MOEQ_DTYPE_FP32) or bf16 (MOEQ_DTYPE_BF16);
 *                 zeros for an expert without rows
 *   workspace     of moeq_grouped_ffn_backward_workspace_bytes(M, E, H, I)
 * dh and every sum are fp32; h, dg and du are rounded to bf16 for the products
 * that take them, so fp32 weight gradients carry that rounding.  Rows outside
 * [offsets[0], offsets[E]) as above; M == 0 writes zero weight gradients.
 * Otherwise as moeq_grouped_ffn.
 */
size_t moeq_grouped_ffn_backward_workspace_bytes(int32_t M, int32_t E, int32_t H, int32_t I);
moeq_status moeq_grouped_ffn_backward(const uint16_t *grad_out_bf16, const uint16_t *x_bf16,
                                      const uint16_t *gate_up_bf16, const uint16_t *down_bf16, const int32_t *offsets,
                                      const float *gu_saved, int32_t M, int32_t E, int32_t H, int32_t I,
                                      int32_t dtype, uint16_t *grad_x_bf16, void *grad_gate_up, void *grad_down,
                                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * The norm of all gradients of a training step, and their clipping:
 *   *norm = sqrt(sum of squares over every tensor)
 *   dst   = src * min(1, max_norm / *norm), in the tensor's own type
 * grads is a HOST array of `count` descriptors (read before the call
 * returns; src and dst are device memory).  dst == src clips in place; a dst
 * elsewhere must overlap no src and no other dst, nor any of them norm or the
 * workspace (MOEQ_EINVAL).  src and dst are aligned to their type.  norm: one fp32 on the device.  The sum is
 * formed in fp64 in a fixed order: the same bits from run to run, and no
 * overflow.  A gradient that is an infinity or a NaN makes the norm one, and
 * nothing is scaled (dst becomes src).  A norm of finite gradients past fp32's
 * range reads as an infinity in *norm, but they are scaled by its fp64 value
 * as any others.  Either way the caller can skip the step on *norm alone.
 * Empty tensors are allowed; count == 0 gives a norm of 0.  MOEQ_EINVAL for a
 * max_norm that is negative or NaN.  Workspace of
 * moeq_clip_grad_norm_workspace_bytes(count), 16-byte aligned.
 */
typedef struct moeq_grad {
  const void *src;
  void *dst;
  int64_t numel;
  int32_t dtype; /* MOEQ_DTYPE_BF16 or MOEQ_DTYPE_FP32 */
} moeq_grad;
size_t moeq_clip_grad_norm_workspace_bytes(int32_t count);
moeq_status moeq_clip_grad_norm(const moeq_grad *grads, int32_t count, double max_norm, float *norm, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * Orthogonalised updates, for trained expert weights: each matrix G of a batch
 * [E][N][K] goes through `steps` Newton-Schulz steps, which move its singular
 * values towards 1 and keep its singular vectors.  From X = G / |G| (the root of
 * the sum of squares; a matrix of zeros stays one), step i takes
 *   A = X X^T,   X <- a X + (b A + c A A) X,   (a, b, c) = coefficients[i]
 *   g             bf16 (dtype MOEQ_DTYPE_BF16) or fp32 (MOEQ_DTYPE_FP32)
 *                 [E][N][K], aligned to its type
 *   coefficients  fp32 [steps][3] in HOST memory, read before the call returns
 *   out_bf16      bf16 [E][N][K], 16-byte aligned
 *   workspace     of moeq_orthogonalize_workspace_bytes(E, N, K), 16-byte aligned
 * The norm is summed in fp64; X, A and the polynomial are kept in fp16, scaled by
 * powers of two, with fp32 sums, and the result is rounded to bf16.  The
 * coefficients may have any size (the polynomial's entries are kept to 2^-11 of
 * themselves, or to 2^-39 (|a| + |b| + |c|) where that is more), but have to keep
 * every singular value below 15.9 from step to step, or the result overflows.
 * Directions that G lacks pick up fp16's rounding, which the steps raise with the
 * small singular values: with the usual coefficients and five steps, a [512, 1024]
 * matrix of rank one is 15 % off, of rank 4 7 %, 16 4.4 %, 64 2.2 %, 256 0.75 %, of
 * full rank 0.2 %, and other shapes alike.  The same bits from run to run.  An
 * infinity or a NaN makes its own matrix NaN.  MOEQ_EINVAL for buffers that
 * overlap, coefficients that are not finite and steps outside 1..64; MOEQ_ESHAPE
 * unless N and K are at most 2^20, the smaller at most 2^15, E <= 65535 and
 * E (N/256 + 1)(K/256 + 1) < 2^18.
 */
size_t moeq_orthogonalize_workspace_bytes(int32_t E, int32_t N, int32_t K);
moeq_status moeq_orthogonalize(const void *g, int32_t dtype, int32_t E, int32_t N, int32_t K,
                               const float *coefficients, int32_t steps, uint16_t *out_bf16, void *workspace,
                               size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOEQ_H */

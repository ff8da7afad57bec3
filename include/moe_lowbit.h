/*
 * moe_lowbit.h -- C ABI of the block-scaled storage forms of the MoE FFN
 * layer (the layer itself: moe_native.h, whose conventions hold here: device
 * pointers owned by the caller, 16-byte aligned, row-major and contiguous; a
 * call only enqueues kernels on `stream`, never allocates, synchronises or
 * reads device memory on the host; arguments are validated on the host from
 * scalars and fail closed; device data is range-checked in the kernels).
 *
 * Two forms, for the two ends of a layer's life:
 *
 *   w4  expert weights in 4 bits, for serving: with few tokens a forward
 *       reads whole experts for a handful of rows, so the weights' bytes are
 *       its time.
 *   q8  the training forward's pre-activation in 8 bits: the one large
 *       tensor that lives from the forward to the backward.
 *
 * Both store groups of 32 consecutive columns with one scale byte b, the
 * power of two 2^(b - 127):
 *
 *   q8  codes int8 c in [-127, 127];                        value c * 2^(b-127)
 *   w4  codes of 4 bits s|ee|m (sign, 2-bit exponent, 1-bit mantissa), the
 *       magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6, two a byte, the even column
 *       in the low half;                                    value c * 2^(b-127)
 *
 * (w4 is laid out like the OCP microscaling format MXFP4, so a checkpoint in
 * that format, codes [rows, K/2] and scales [rows, K/32], is used as it is:
 * every byte from 0 to 254 counts exactly, except that the magnitudes that no
 * float32 or bf16 holds, 2^128 and more (codes 4 and 6 at b = 253, 2 to 6 at
 * 254), are infinite.)
 * The quantizers pick the smallest b >= 1 with which no element of the group
 * is off by more than half a step of its codes, and round to nearest, ties
 * to the even code; a group of zeros has b = 1 and codes 0.  b = 255 stands
 * for NaN in the whole group (codes then mean nothing); the quantizers write
 * it, with codes 0, for a group that holds a NaN, an infinity or a magnitude
 * that would round to 2^128 (from 255 * 2^120 on in q8, 7 * 2^125 in w4).
 * Every value of b up to 248 (q8) or 252 (w4), all that the quantizers write,
 * is a bf16 number exactly, so dequantizing rounds nothing.
 */
#ifndef MOE_LOWBIT_H
#define MOE_LOWBIT_H

#include "moe_native.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bf16 [rows, K] -> 4-bit codes [rows, K/2] and scales [rows, K/32].  Any
 * stack of matrices is one call (an expert tensor [E, r, K]: rows = E*r).
 * rows >= 0 (0: no-op), K a multiple of 64 in [64, 32768], and rows * K at
 * most 2^34 (MOE_ERR_UNSUPPORTED otherwise). */
int moe_w4_quantize(const uint16_t* w, int64_t rows, int32_t K, uint8_t* codes, uint8_t* scales,
                    hipStream_t stream);

/* The bf16 values that 4-bit codes stand for (exact; the inverse layout of
 * moe_w4_quantize, same limits). */
int moe_w4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K,
                      uint16_t* w, hipStream_t stream);

/* bf16 [rows, D] -> int8 codes [rows, D] and scales [rows, D/32]; limits as
 * moe_w4_quantize with D for K. */
int moe_q8_quantize(const uint16_t* v, int64_t rows, int32_t D, int8_t* codes, uint8_t* scales,
                    hipStream_t stream);

/* The bf16 values that 8-bit codes stand for (exact). */
int moe_q8_dequantize(const int8_t* codes, const uint8_t* scales, int64_t rows, int32_t D,
                      uint16_t* v, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Steps 4-5 of the dropless form on 4-bit weights.
 *
 * The route list is moe_route_dropless's (or moe_route_dropless_live's), with
 * R = moe_dropless_bound(N, K, E) slots; N, K, E are the sizes it was built
 * with.  Expert e's routes are the slots block_start[e]*BM + (0 ..
 * route_counts[e]-1).
 *
 *   x          in  bf16 [N, H]
 *   w1_codes   in  [E, 2I, H/2], w1_scales [E, 2I, H/32]  rows 0..I-1 gate, I..2I-1 up
 *   w2_codes   in  [E, H, I/2],  w2_scales [E, H, I/32]
 *   act        out bf16  [R, I]  silu(x_r W1g^T) * (x_r W1u^T) * prob, rounded
 *                                once from float32; a transient FC2 consumes
 *   route_out  out float32 [R, H]  act W2^T per slot, not rounded: the token's
 *                                sum rounds once
 *   y          out bf16  [N, H]  float32 sum over k of the token's routes, in
 *                                k order from +0.0 (zeros for a token without routes)
 *
 * Only the routes' rows of act and route_out are written: pad slots and the
 * tail past the extent stay as they were, and nothing reads them.  A route's
 * result depends on its own row and expert alone, bit for bit: not on N, on
 * the other tokens, or on its slot.  Any N of the routing envelope is served;
 * the kernels are made for few routes per expert (up to about 64), where the
 * weights' bytes decide.  An expert's weights are read and converted once for
 * every 32 of its routes, so with hundreds of them the bf16 layer is faster
 * (128 experts of 2048 x 768: 64 routes an expert 182 us against 235 in bf16,
 * 128 314 against 282; 8 of 4096 x 1792: 256 158 against 209, 512 282 against
 * 271; 64 of 7168 x 2048: 128 1126 against 1181).
 *
 * H and I multiples of 64 in [64, 16384]; (N + 1)*H*2, (N + BM)*max(H, I)*4
 * and one expert's codes I*H below 2^31. */
int moe_grouped_fc1_swiglu_w4(const uint16_t* x, const uint8_t* w1_codes, const uint8_t* w1_scales,
                              const int32_t* sorted_slot_ids, const float* slot_probs,
                              const int32_t* expert_ids, const int32_t* block_start,
                              const int32_t* route_counts, int64_t N, int32_t H, int32_t I,
                              int32_t E, int32_t K, uint16_t* act, hipStream_t stream);
int moe_grouped_fc2_w4(const uint16_t* act, const uint8_t* w2_codes, const uint8_t* w2_scales,
                       const int32_t* expert_ids, const int32_t* block_start,
                       const int32_t* route_counts, int64_t N, int32_t H, int32_t I, int32_t E,
                       int32_t K, float* route_out, hipStream_t stream);

/* moe_gather_combine over float32 rows: y[t] = bf16( float32 sum over k with
 * 0 <= token_routes[t,k] < R of route_out[token_routes[t,k]] ).  Limits as
 * moe_gather_combine. */
int moe_gather_combine_f32(const float* route_out, const int32_t* token_routes, int64_t N,
                           int32_t K, int32_t H, int64_t R, uint16_t* y, hipStream_t stream);

/* The three calls above, in order, on one stream: the same y, bit for bit.
 * act and route_out are scratch here: what they hold afterwards is unspecified
 * (for a few tokens FC2 and the sum run as one kernel, which leaves route_out
 * alone), and calls that share them must not overlap. */
int moe_grouped_ffn_w4(const uint16_t* x, const uint8_t* w1_codes, const uint8_t* w1_scales,
                       const uint8_t* w2_codes, const uint8_t* w2_scales,
                       const int32_t* sorted_slot_ids, const float* slot_probs,
                       const int32_t* expert_ids, const int32_t* block_start,
                       const int32_t* route_counts, const int32_t* token_routes, int64_t N,
                       int32_t H, int32_t I, int32_t E, int32_t K, uint16_t* act, float* route_out,
                       uint16_t* y, hipStream_t stream);

/* ------------------------------------------------------------------------
 * The training step with its pre-activation kept in 8 bits: in place of
 * moe_grouped_fc1_swiglu_save and moe_swiglu_bwd, everything else as there.
 * ------------------------------------------------------------------------ */

/* moe_grouped_fc1_swiglu that also stores the raw FC1 product
 * h = x[row(s)] @ W1[e]^T in 8 bits, quantized from its float32 sums:
 *   codes  out int8  [R, 2I]     row s = [gate (I) | up (I)]
 *   scales out uint8 [R, 2I/32]
 * act is the same as moe_grouped_fc1_swiglu's.  Pad slots: codes 0.
 * Arguments and limits as moe_grouped_fc1_swiglu_save. */
int moe_grouped_fc1_swiglu_save_q8(const uint16_t* x, const uint16_t* w1,
                                   const int32_t* sorted_slot_ids, const float* slot_probs,
                                   int64_t N, int32_t H, int32_t I, int32_t E, int64_t C,
                                   uint16_t* act, int8_t* codes, uint8_t* scales,
                                   hipStream_t stream);

/* moe_swiglu_bwd with the pre-activation read from its 8-bit form:
 *   codes in int8 [R, 2I], scales in uint8 [R, 2I/32], d_act in bf16 [R, I],
 *   slot_probs in f32 [R]; act out bf16 [R, I], d_preact out bf16 [R, 2I],
 *   d_prob out f32 [R].
 * act and d_preact are bit for bit those of moe_swiglu_bwd on the dequantized
 * pre-activation; d_prob is the same sum in another order. */
int moe_swiglu_bwd_q8(const int8_t* codes, const uint8_t* scales, const uint16_t* d_act,
                      const float* slot_probs, int64_t R, int32_t I, uint16_t* act,
                      uint16_t* d_preact, float* d_prob, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LOWBIT_H */

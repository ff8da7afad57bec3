/*
 * moe_block.h -- C ABI of the operators around the MoE FFN layer (the layer
 * itself: moe_native.h, whose conventions hold here: device pointers owned by
 * the caller, 16-byte aligned, row-major and contiguous; a call only enqueues
 * kernels on `stream`, never allocates, synchronises or reads device memory on
 * the host; arguments are validated on the host from scalars and fail closed;
 * device data is range-checked in the kernels).
 *
 * A transformer block's feed-forward half, from residual stream to residual
 * stream:
 *
 *   h = x + r;  u = norm(h);  y = h + MoE(u)
 *
 *   moe_layer_norm_fwd, moe_layer_norm_bwd   the norm and the addition in
 *                         front of it, and their backward
 *   moe_ffn_decode        the whole layer for the few tokens of a decode step,
 *                         router logits in, residual stream out, in two kernels
 *   moe_grad_norm, moe_adamw_step            the gradients' global norm, and
 *                         the clipped AdamW step over many tensors, its
 *                         moments in 32 bits or in 8
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_native.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The layer for a few tokens
 * ------------------------------------------------------------------------ */

/* Most tokens of a moe_ffn_decode call: 64. */
int32_t moe_ffn_decode_max_tokens(void);

/* Bytes of moe_ffn_decode's workspace: the activation between its kernels,
 * bf16 [N*K, I], and the batch's routes by expert.  0 when the arguments fall outside the call's limits.
 * Host-only.  Contents between calls mean nothing; calls that share a
 * workspace must not overlap. */
size_t moe_ffn_decode_workspace_bytes(int64_t N, int32_t H, int32_t I, int32_t E, int32_t K);

/* Steps 1-5 of the dropless form for 1 <= N <= 64 tokens (N == 0: no-op), in
 * two kernels that read a chosen expert's weights once for every block of its
 * routes: of up to 8, 16 or 32 in the first and 4, 8 or 16 in the second, by the
 * routes an expert on average, so once where the batch is spread out:
 *
 *   logits      in  float32 [N, E]
 *   x           in  bf16 [N, H]
 *   w1          in  bf16 [E, 2I, H], w2 in bf16 [E, H, I]
 *   residual    in  bf16 [N, H], added to each token's sum; may be null
 *   n_live      in  int32 [1], device scalar clamped to [0, N]; may be null (N).
 *                   Tokens at or past it route nowhere (ids -1, probabilities
 *                   0) and their rows of y are left as they were
 *   topk_ids    out int32 [N, K], topk_probs out float32 [N, K]: bit for bit
 *                   moe_route_dropless's
 *   y           out bf16 [N, H] = bf16( sum_k act_k W2[e_k]^T + residual ),
 *                   act_k = bf16( silu(x Wg^T) * (x Wu^T) * prob_k ); may be
 *                   residual or x
 *
 * Outputs (the workspace's bytes among them) that share memory with another
 * buffer in any other way are refused.
 *
 * Sums are float32 and rounded once; between the products only the activation
 * is rounded, as everywhere in the layer.  The same inputs give the same bits;
 * the order of a token's sums depends on the call's sizes and on which experts
 * the batch uses, so a token's last bits can differ from one batch to another.
 * H, I multiples of 64 in [64, 16384], 1 <= K <= min(E, 32), E <= 1024. */
int moe_ffn_decode(const float* logits, const uint16_t* x, const uint16_t* w1, const uint16_t* w2,
                   const uint16_t* residual, const int32_t* n_live, int64_t N, int32_t H, int32_t I,
                   int32_t E, int32_t K, int32_t* topk_ids, float* topk_probs, void* workspace,
                   size_t workspace_bytes, uint16_t* y, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm and RMS norm
 * ------------------------------------------------------------------------ */

/* Types of a norm's tensors. */
typedef enum { MOE_BF16 = 0, MOE_F32 = 1 } moe_dtype;

/* One row of D values:
 *   h    = x + residual, rounded to x's type      (x itself without residual)
 *   mean = sum h / D, rstd = 1 / sqrt( sum (h - mean)^2 / D + eps )
 *   y    = (h - mean) * rstd * weight + bias
 * RMS norm: mean null, and 0 in the formulas.
 *
 *   x, residual  in  [rows, D] of x_type; residual may be null
 *   weight       in  float32 [D]; bias in float32 [D], may be null (0)
 *   total        out h, [rows, D] of x_type: given if and only if residual is;
 *                    may be x or residual
 *   y            out [rows, D] of y_type (x bf16: bf16; x float32: either);
 *                    may be x or residual if the types are equal and total is not it
 *   mean, rstd   out float32 [rows]; mean may be null (RMS norm)
 *
 * Outputs that share memory with another buffer in any other way are refused.
 *
 * 1 <= D <= 16384, any rows * D < 2^40; rows == 0: no-op.  Sums are float32;
 * the variance is the second pass's, over the row in registers. */
int moe_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias,
                       int64_t rows, int32_t D, double eps, int32_t x_type, int32_t y_type,
                       void* total, void* y, float* mean, float* rstd, hipStream_t stream);

/* Bytes of moe_layer_norm_bwd's workspace (0 outside its limits).  Host-only.
 * Calls that share a workspace must not overlap. */
size_t moe_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t D);

/* The backward, with xhat = (h - mean) * rstd and g = dy * weight:
 *   dx      = rstd * ( g - mean_D(g) - xhat * mean_D(g * xhat) ) + dtotal
 *   dweight = sum over rows of dy * xhat,   dbias = sum over rows of dy
 * RMS norm (mean null): without mean_D(g).
 *
 *   dy       in  [rows, D] of y_type
 *   h        in  [rows, D] of x_type: what was normalised (total, or x)
 *   mean, rstd in float32 [rows] of the forward
 *   dtotal   in  [rows, D] of x_type, the gradient that reaches h past the
 *                norm (through total); may be null
 *   dx       out [rows, D] of x_type: the gradient of x and of residual alike;
 *                may be h or dtotal, or dy if the types are equal
 *   dweight  out float32 [D]; dbias out float32 [D], may be null
 *   accumulate   0: the weight gradients are written; 1: added to what is there
 *
 * Outputs (workspace_bytes as asked for among them) that share memory with another
 * buffer in any other way are refused.
 *
 * Sums are float32, rows in a fixed order, no atomics: the same bits from the
 * same inputs.  Limits as the forward; rows == 0 writes zero weight gradients
 * (or adds nothing). */
int moe_layer_norm_bwd(const void* dy, const void* h, const float* weight, const float* mean,
                       const float* rstd, const void* dtotal, int64_t rows, int32_t D,
                       int32_t x_type, int32_t y_type, int32_t accumulate, void* dx, float* dweight,
                       float* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Gradient norm and AdamW over many tensors
 * ------------------------------------------------------------------------ */

/* One tensor of n elements.  Pointers are device pointers; an array of these is
 * read on the host during a call and not kept. */
typedef struct {
    void* param;            /* bf16 or float32 [n], updated                         */
    float* master;          /* float32 [n], updated, param then its rounding; null:
                             * param itself is read and updated                     */
    const void* grad;       /* bf16 or float32 [n]                                  */
    void* m;                /* first moment: float32 [n], or codes uint8 [n]        */
    void* v;                /* second moment: float32 [n], or codes uint8 [n]       */
    uint8_t* m_scales;      /* codes: ceil(n / 32) scale bytes each, of any         */
    uint8_t* v_scales;      /* alignment; null for float32 moments                  */
    int64_t n;              /* elements, 0 to 2^34                                  */
    float weight_decay;
    int32_t param_type;     /* moe_dtype                                            */
    int32_t grad_type;      /* moe_dtype                                            */
    int32_t reserved;       /* 0                                                    */
} moe_adamw_tensor;

/* Moments in 8 bits: groups of 32 consecutive elements of a tensor share a
 * scale byte b, the power of two 2^(b - 127); b = 255 stands for NaN in the
 * whole group (codes then mean nothing).
 *   m   OCP e4m3 codes (sign, 4-bit exponent, 3-bit mantissa, largest 448),
 *       value code * 2^(b-127), to nearest, ties to even: the layout of MXFP8
 *   v   held by its root: code c stands for root (1 + (c%16)/16) *
 *       2^(c/16 - 15) * 2^(b-127), c = 0 for 0; to nearest, ties to even, and a
 *       root that is not 0 never becomes 0 (nothing is ever divided by a
 *       vanished moment)
 * The scale is the smallest b >= 1 with which no magnitude of the group rounds
 * past the largest code (464 and 1.96875 times 2^(b-127) go to the next b). */

/* A plan: a device buffer that holds the list of tensors for the kernels, and
 * their partial sums and counters.  moe_adamw_plan writes it (with kernels, no
 * copy); moe_grad_norm and moe_adamw_step take the same list again, on the
 * host, and the plan written for it: as long as the tensors stay where they
 * are, one plan serves every step.  Calls that share a plan must not overlap.
 * All tensors of a list have moments of the same kind; together at most 2^40
 * elements.  No two of a list's buffers may overlap if a step writes one of them
 * (gradients may).  0 bytes: bad arguments. */
size_t moe_adamw_plan_bytes(const moe_adamw_tensor* tensors, int32_t count);
int moe_adamw_plan(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                   hipStream_t stream);

/* norm[0] = float32( sqrt( sum over all tensors of grad^2 ) ): eight neighbours'
 * squares in float32 (in float64 where their sum leaves 1e-25 .. 1e38), the sums
 * of eight in float64, in a fixed order. */
int moe_grad_norm(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                  float* norm, hipStream_t stream);

/* One AdamW step of every tensor:
 *   c = max_norm / norm where norm > max_norm, else 1 (and 1 without grad_norm)
 *   g = c * grad;  t = step + 1
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / ( sqrt(v) / sqrt(1 - beta2^t) + eps )
 * in float32; roots and the division are the hardware's, good to 1 ulp (8-bit
 * moments: p moves by the moments before they are rounded).
 * 8-bit moments are rounded to the nearest code, which loses moves of less than half
 * a code: right for a step or a few, but over a training run the moments do not
 * follow the gradients (moe_moments.h has figures, and the step for that).
 *
 *   lr         in  float32 [1], device scalar
 *   grad_norm  in  float32 [1], device scalar (moe_grad_norm's); may be null.
 *                  Not finite: the call leaves everything as it was, step included
 *   max_norm   > 0, used with grad_norm only
 *   step       in/out int32 [1], device scalar: steps taken so far (clamped to
 *                  [0, 2^31 - 2]); becomes t
 *
 * 0 <= beta < 1; eps 0 (an element that has had no gradient then becomes NaN, 0 / 0)
 * or 2^-126 and more. */
int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                   const float* lr, double beta1, double beta2, double eps, const float* grad_norm,
                   double max_norm, int32_t* step, hipStream_t stream);

/* What 8-bit moments stand for: m and the root of v, both bf16 [n] (exact from
 * b = 13 on; below, where bf16 ends, rounded to its subnormals).
 * 0 <= n <= 2^34. */
int moe_moment_values(const uint8_t* m, const uint8_t* m_scales, const uint8_t* v,
                      const uint8_t* v_scales, int64_t n, uint16_t* m_values, uint16_t* root_values,
                      hipStream_t stream);

/* 8-bit moments from float32 ones (v: the moment itself, not its root). */
int moe_moment_codes(const float* m, const float* v, int64_t n, uint8_t* m_codes, uint8_t* m_scales,
                     uint8_t* v_codes, uint8_t* v_scales, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */

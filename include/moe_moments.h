/*
 * moe_moments.h -- C ABI of the AdamW step whose 8-bit moments follow their
 * gradients over a training run (lists, plans, formats and the step itself:
 * moe_block.h, whose conventions hold here).
 *
 * A step moves a moment by a small part of itself: a second moment by 1 - beta2
 * of it at most downwards, its root by half that.  Codes are 1/32 to 1/16 of a
 * root and 1/16 to 1/8 of a first moment apart, so rounding to the nearest code
 * after every step loses the move, and the moment stays where it is: with
 * moe_adamw_step the root of v after 2000 steps is 0.74 of the true one
 * (constant gradients, beta2 0.95; 0.16 with 0.999), 1.2 (normal ones, 0.95), and
 * 11 where the gradients became ten times smaller half-way.  Here a moment is
 * rounded up or down at random such that its mean over the steps is kept; of the
 * same runs the median root is within 3% of the true one, the mean of v within 0.5%.
 */
#ifndef MOE_MOMENTS_H
#define MOE_MOMENTS_H

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* moe_adamw_step for a list of 8-bit moments, which it rounds stochastically:
 *
 *   m   to the e4m3 code below or above its magnitude, up with probability
 *       (|m| - below) / (above - below)
 *   v   its root r to the code below or above, up with probability
 *       (r^2 - below^2) / (above^2 - below^2), so that the mean of v is kept;
 *       a root that is not 0 and lies below code 1 becomes code 1
 *
 * The scale is the smallest b >= 1 with which no magnitude of the group exceeds
 * the largest code (448 and 1.9375 times 2^(b-127)).  Parameters move by the
 * moments before they are rounded, as in moe_adamw_step.
 *
 * The chance comes from a hash, with the same seed, step and list always the same:
 * with t = step + 1 and an element at place j of chunk c (chunks of 4096
 * elements are counted through the list, each tensor of n > 0 begins one)
 *
 *   mix(x):  x ^= x >> 16; x *= 0x6A09E667; x ^= x >> 15; x *= 0xBB67AE85; x ^= x >> 16
 *   h = mix( mix( mix(seed + 0x9E3779B9 t) + c ) + 0x9E3779B9 j )       in 32 bits
 *
 * m goes up where h >> 12 reaches 2^20 (1 - its fraction), the root where
 * (h & 0xFFFFFF) / 2^24 is below its own.  A captured step draws anew in every
 * replay, since the step is a device scalar.  Lists of 32-bit moments are refused. */
int moe_adamw_step_stochastic(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                              const float* lr, double beta1, double beta2, double eps, const float* grad_norm,
                              double max_norm, int32_t* step, uint32_t seed, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MOMENTS_H */

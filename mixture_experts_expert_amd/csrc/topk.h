// Top-K of a token's router logits by a group of LPT lanes (internal): the order
// of logits, the selection rounds and the softmax over the picks.  The routing
// calls use all of it; the forward for a few tokens shares the order, and the
// rounds above 256 experts, and has rounds and a softmax of its own beside them,
// of the same operations, so that picks and probabilities agree bit for bit.
#pragma once

#include <math.h>

#include "moe_common.h"

namespace moe {
namespace {

// DPP lane exchanges inside a 16-lane row (no LDS round trip).
constexpr int kDppXor1 = 0xB1;        // quad_perm [1,0,3,2]
constexpr int kDppXor2 = 0x4E;        // quad_perm [2,3,0,1]
constexpr int kDppHalfMirror = 0x141; // lane i <-> 7-i within each half row
constexpr int kDppMirror = 0x140;     // lane i <-> 15-i within the row
constexpr int kDppShr1 = 0x111;       // lane i <- lane i-1 within the row

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(dpp<CTRL>(__float_as_int(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const long long b = __double_as_longlong(v);
    const int lo = dpp<CTRL>(static_cast<int>(b)), hi = dpp<CTRL>(static_cast<int>(b >> 32));
    return __longlong_as_double((static_cast<long long>(hi) << 32) | static_cast<uint32_t>(lo));
}

// Arg-max key of (logit, expert): the float's bits made monotonic as an
// unsigned integer in the high word (with -0 folded onto +0 first, so equal
// logits stay equal), and ~expert in the low word, so the larger key is the
// larger logit and, between equal logits, the lower expert -- the order the
// routing defines, decided by one unsigned comparison with no branches.  Any
// real logit's key exceeds 2^32; a key with a zero high word has been picked.
__device__ __forceinline__ uint64_t topk_key(float v, int e) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t u = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return (static_cast<uint64_t>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(e));
}
__device__ __forceinline__ float key_logit(uint64_t key) {
    const uint32_t u = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
    const int lo = dpp<CTRL>(static_cast<int>(v)), hi = dpp<CTRL>(static_cast<int>(v >> 32));
    return (static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) | static_cast<uint32_t>(lo);
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int off, int width) {
    const int lo = __shfl_xor(static_cast<int>(v), off, width);
    const int hi = __shfl_xor(static_cast<int>(v >> 32), off, width);
    return (static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) | static_cast<uint32_t>(lo);
}

// K rounds of a group-wide arg-max over the lanes' keys (0: no expert there).
// Lane k of the group keeps round k's winner.
template <int LPT, int VPL>
__device__ __forceinline__ void topk_rounds(uint64_t (&key)[VPL], int K, int g, int& my_id, float& my_logit) {
    for (int k = 0; k < K; ++k) {
        // the lane's best remaining key (a tree for independent comparisons),
        // then the group's, by DPP inside 16-lane rows and shuffles across them
        uint64_t m[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) m[j] = key[j];
#pragma unroll
        for (int w = 1; w < VPL; w <<= 1)
#pragma unroll
            for (int j = 0; j + w < VPL; j += 2 * w) m[j] = umax64(m[j], m[j + w]);
        uint64_t best = m[0];
        best = umax64(best, dpp64<kDppXor1>(best));
        best = umax64(best, dpp64<kDppXor2>(best));
        best = umax64(best, dpp64<kDppHalfMirror>(best));
        best = umax64(best, dpp64<kDppMirror>(best));
#pragma unroll
        for (int off = 16; off < LPT; off <<= 1) best = umax64(best, shfl_xor64(best, off, LPT));
        // the winner leaves the running: its key keeps only the low word
        const uint32_t won = static_cast<uint32_t>(best);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (static_cast<uint32_t>(key[j]) == won) key[j] = won;
        if (g == k) { my_logit = key_logit(best); my_id = static_cast<int>(0xFFFFFFFFu - won); }
    }
}

// The K-way softmax of the picks, lane k's probability (0 past K): float64
// exp(l_k - l_0), summed in k order, one division, one rounding.
template <int LPT>
__device__ __forceinline__ float topk_prob(float my_logit, int K, int g) {
    const double top = static_cast<double>(__shfl(my_logit, 0, LPT));
    const double ex = g < K ? exp(static_cast<double>(my_logit) - top) : 0.0;
    // denominator: e_0 + e_1 + ... + e_{K-1} in k order.  In a 16-lane row,
    // K-1 rounds of s <- s(lane-1) + e leave lane K-1 holding the ordered sum.
    double denom;
    if (LPT == 16) {
        double s = ex;
        for (int it = 1; it < K; ++it) {
            const double prev = dpp<kDppShr1>(s);
            s = g == 0 ? ex : prev + ex;
        }
        denom = __shfl(s, K - 1, LPT);
    } else {
        denom = 0.0;
        for (int k = 0; k < K; ++k) denom += __shfl(ex, k, LPT);
    }
    return static_cast<float>(ex / denom);
}

}  // namespace
}  // namespace moe

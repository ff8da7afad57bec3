// Conversions between bf16 tensors and their block-scaled forms, and the
// SwiGLU backward that reads the 8-bit pre-activation.
//
// All are HBM-bound passes: every input is read once and every output written
// once, 8 columns a lane (16 bytes of bf16), so a group of 32 columns is four
// neighbouring lanes, which share its largest magnitude in two lane swaps.
// 8192 rows of 7168, three tensors in turn: 32 us each way in 8 bits, 5.5 TB/s,
// what a plain copy reaches (two pieces a lane the same, four 33 and 35 us); one
// after the other, the second from the caches, 37 and 27.  In 4 bits, once in a
// checkpoint's life, 41 and 37 us (4.0 TB/s: more of it is arithmetic); the
// weights of 128 experts of 2048 x 768, 1.2 GB, 395 and 354 us.
#include <algorithm>
#include <initializer_list>

#include "lowbit.h"

namespace moe {
namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t group_amax(const u16x8& v) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, static_cast<uint32_t>(v[j]) << 16 & 0x7FFF0000u);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1)));
    return max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2)));
}

// One lane: 8 columns.  `items` (a multiple of 8) counts lanes' pieces.
__global__ __launch_bounds__(256) void q8_quantize_kernel(const uint16_t* __restrict__ v, int64_t items,
                                                          int8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= items) return;
    const u16x8 x = reinterpret_cast<const u16x8*>(v)[i];
    const int b = q8_scale_byte(group_amax(x));
    const float inv = inv_scale(b);
    u32x2 c;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        c[h] = q8_pack4(bf16_to_f32(x[4 * h]), bf16_to_f32(x[4 * h + 1]), bf16_to_f32(x[4 * h + 2]),
                        bf16_to_f32(x[4 * h + 3]), inv);
    if (b == kScaleNaN) c = 0;
    reinterpret_cast<u32x2*>(codes)[i] = c;
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(b);
}

__global__ __launch_bounds__(256) void q8_dequantize_kernel(const int8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t items,
                                                            uint16_t* __restrict__ v) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= items) return;
    const u32x2 c = reinterpret_cast<const u32x2*>(codes)[i];
    const float s = scale_value(scales[i >> 2]);
    u16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = f32_to_bf16(q8_float(c[j >> 2], j & 3) * s);
    reinterpret_cast<u16x8*>(v)[i] = o;
}

// The code nearest to a = |v| / scale, ties to the even mantissa (the code's
// low bit): the middles 0.25, 1.25, 2.5 and 5 round down, 0.75, 1.75 and 3.5 up.
__device__ __forceinline__ uint32_t w4_code(float v, float inv) {
    const float a = __builtin_fabsf(v) * inv;
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return c | (v < 0.0f ? 8u : 0u);
}

__global__ __launch_bounds__(256) void w4_quantize_kernel(const uint16_t* __restrict__ w, int64_t items,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= items) return;
    const u16x8 x = reinterpret_cast<const u16x8*>(w)[i];
    const int b = w4_scale_byte(group_amax(x));
    const float inv = inv_scale(b);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) c |= w4_code(bf16_to_f32(x[j]), inv) << (4 * j);
    if (b == kScaleNaN) c = 0;
    reinterpret_cast<uint32_t*>(codes)[i] = c;
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(b);
}

__global__ __launch_bounds__(256) void w4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t items,
                                                            uint16_t* __restrict__ w) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= items) return;
    const uint32_t c = reinterpret_cast<const uint32_t*>(codes)[i];
    const float s = scale_value(scales[i >> 2]);
    u16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t k = c >> (4 * j), e = k >> 1 & 3u, m = k & 1u;
        const float mag = e == 0 ? 0.5f * m : __uint_as_float((126u + e) << 23 | m << 22);
        o[j] = f32_to_bf16((k & 8u ? -mag : mag) * s);
    }
    reinterpret_cast<u16x8*>(w)[i] = o;
}

// With g, u = the pre-activation's values, sig = sigmoid(g):
//   act    = silu(g) * u * p
//   d_gate = d_act * p * u * sig * (1 + g * (1 - sig))
//   d_up   = d_act * p * silu(g)
//   d_prob = sum over the row of d_act * silu(g) * u
// A workgroup takes the rows, one at least, whose 8-column pieces its threads
// hold at once: lanes have work whatever I is (with a wave a row, I = 64 used
// one lane in eight: 60000 rows 29 us, 8.8 now), and a thread's loads are all on
// their way together (32768 rows of 768, three sets in turn: 47 us, 5.4 TB/s; 53
// a wave a row, 48.6 with two pieces a thread).  A row is a multiple of 8 pieces: 8
// neighbouring lanes hold 64 columns of one row, their sum goes to LDS, and 8
// lanes add a row's sums.  The stores are of the default policy: non-temporal
// they take this kernel to 42.6 us, but the GEMMs that read d_preact and act
// next then find them in memory instead of the caches, and the backward as a
// whole takes 829 us against 820.
constexpr int kBwdThreads = 256;

__global__ __launch_bounds__(kBwdThreads) void swiglu_bwd_q8_kernel(const int8_t* __restrict__ codes,
                                                                    const uint8_t* __restrict__ scales,
                                                                    const uint16_t* __restrict__ d_act,
                                                                    const float* __restrict__ probs, int R, int I,
                                                                    int per, uint16_t* __restrict__ act,
                                                                    uint16_t* __restrict__ d_pre,
                                                                    float* __restrict__ d_prob) {
    __shared__ float s_dp[kMaxDim / 64];                 // of `per` rows: 256 pieces, or one row's
    const int pieces = I / 8;                            // of a row
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * per;
    const int rows = static_cast<int>(min(static_cast<int64_t>(per), R - row0));
    for (int i = threadIdx.x; i < rows * pieces; i += kBwdThreads) {
        const int r = i / pieces, c = (i - r * pieces) * 8;
        const int64_t s = row0 + r;
        const int8_t* row = codes + s * 2 * I;
        const uint8_t* srow = scales + s * (2 * I / kGroup);
        const u32x2 cg = *reinterpret_cast<const u32x2*>(row + c);
        const u32x2 cu = *reinterpret_cast<const u32x2*>(row + I + c);
        const float fg = scale_value(srow[c / kGroup]), fu = scale_value(srow[(I + c) / kGroup]);
        const u16x8 d8 = *reinterpret_cast<const u16x8*>(d_act + s * I + c);
        const float p = probs[s];
        u16x8 a8, dg8, du8;
        float dp = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = q8_float(cg[j >> 2], j & 3) * fg, u = q8_float(cu[j >> 2], j & 3) * fu;
            const float d = bf16_to_f32(d8[j]);
            const float sg = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
            const float sl = g * sg;
            a8[j] = f32_to_bf16(sl * u * p);
            dg8[j] = f32_to_bf16(d * p * u * (sg * (1.0f + g * (1.0f - sg))));
            du8[j] = f32_to_bf16(d * p * sl);
            dp += d * sl * u;
        }
        *reinterpret_cast<u16x8*>(act + s * I + c) = a8;
        *reinterpret_cast<u16x8*>(d_pre + s * 2 * I + c) = dg8;
        *reinterpret_cast<u16x8*>(d_pre + s * 2 * I + I + c) = du8;
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) dp += __shfl_xor(dp, o);
        if ((threadIdx.x & 7) == 0) s_dp[i / 8] = dp;
    }
    __syncthreads();
    const int r = threadIdx.x / 8, n = pieces / 8;
    if (r < rows) {
        float dp = 0.0f;
        for (int j = threadIdx.x & 7; j < n; j += 8) dp += s_dp[r * n + j];
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) dp += __shfl_xor(dp, o);
        if ((threadIdx.x & 7) == 0) d_prob[row0 + r] = dp;
    }
}

int check_pieces(int64_t rows, int32_t cols, std::initializer_list<const void*> ptrs, int64_t* items) {
    if (rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
    // the widest rows are a pre-activation's, 2I; a grid holds fewer than 2^32 lanes
    if (cols % 64 || cols > 2 * kMaxDim || rows > (static_cast<int64_t>(1) << 34) / cols) return MOE_ERR_UNSUPPORTED;
    *items = rows * (cols / 8);
    if (rows == 0) return MOE_OK;
    for (const void* q : ptrs) {
        if (!q) return MOE_ERR_INVALID_ARG;
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    }
    return MOE_OK;
}

unsigned piece_blocks(int64_t items) { return static_cast<unsigned>((items + 255) / 256); }

}  // namespace
}  // namespace moe

extern "C" int moe_q8_quantize(const uint16_t* v, int64_t rows, int32_t D, int8_t* codes, uint8_t* scales,
                               hipStream_t stream) {
    using namespace moe;
    int64_t items = 0;
    const int st = check_pieces(rows, D, {v, codes, scales}, &items);
    if (st != MOE_OK || rows == 0) return st;
    q8_quantize_kernel<<<piece_blocks(items), 256, 0, stream>>>(v, items, codes, scales);
    return launch_status();
}

extern "C" int moe_q8_dequantize(const int8_t* codes, const uint8_t* scales, int64_t rows, int32_t D,
                                 uint16_t* v, hipStream_t stream) {
    using namespace moe;
    int64_t items = 0;
    const int st = check_pieces(rows, D, {codes, scales, v}, &items);
    if (st != MOE_OK || rows == 0) return st;
    q8_dequantize_kernel<<<piece_blocks(items), 256, 0, stream>>>(codes, scales, items, v);
    return launch_status();
}

extern "C" int moe_w4_quantize(const uint16_t* w, int64_t rows, int32_t K, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream) {
    using namespace moe;
    int64_t items = 0;
    const int st = check_pieces(rows, K, {w, codes, scales}, &items);
    if (st != MOE_OK || rows == 0) return st;
    w4_quantize_kernel<<<piece_blocks(items), 256, 0, stream>>>(w, items, codes, scales);
    return launch_status();
}

extern "C" int moe_w4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K,
                                 uint16_t* w, hipStream_t stream) {
    using namespace moe;
    int64_t items = 0;
    const int st = check_pieces(rows, K, {codes, scales, w}, &items);
    if (st != MOE_OK || rows == 0) return st;
    w4_dequantize_kernel<<<piece_blocks(items), 256, 0, stream>>>(codes, scales, items, w);
    return launch_status();
}

extern "C" int moe_swiglu_bwd_q8(const int8_t* codes, const uint8_t* scales, const uint16_t* d_act,
                                 const float* slot_probs, int64_t R, int32_t I, uint16_t* act,
                                 uint16_t* d_preact, float* d_prob, hipStream_t stream) {
    using namespace moe;
    if (R < 0 || I < 1) return MOE_ERR_INVALID_ARG;
    if (I % 64 || I > kMaxDim || R > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    for (const void* q : {static_cast<const void*>(codes), static_cast<const void*>(scales),
                          static_cast<const void*>(d_act), static_cast<const void*>(slot_probs),
                          static_cast<const void*>(act), static_cast<const void*>(d_preact),
                          static_cast<const void*>(d_prob)}) {
        if (!q) return MOE_ERR_INVALID_ARG;
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    }
    const int per = std::max(1, kBwdThreads / (I / 8));
    // a grid of 2^32 threads or more wraps without an error: at most 2^23 workgroups a launch
    const int64_t most = static_cast<int64_t>(per) << 23;
    for (int64_t r = 0; r < R; r += most) {
        const int n = static_cast<int>(std::min(most, R - r));
        swiglu_bwd_q8_kernel<<<static_cast<unsigned>((n + per - 1) / per), kBwdThreads, 0, stream>>>(
            codes + r * 2 * I, scales + r * (2 * I / kGroup), d_act + r * I, slot_probs + r, n, I, per,
            act + r * I, d_preact + r * 2 * I, d_prob + r);
    }
    return launch_status();
}

// Steps 4-5 of the dropless MoE FFN forward on 4-bit expert weights, for the
// few tokens of a decode step.
//
//   act[s]       = silu(x_r W1g^T) * (x_r W1u^T) * p_s     r = sorted_slot_ids[s]
//   route_out[s] = act[s] W2^T                             (float32)
//   y[t]         = bf16( sum_k route_out[token_routes[t, k]] )
//
// With a handful of rows per expert the weights' bytes are the time: every
// byte of an expert in use is read once, for all of its rows, and everything
// else is kept out of the way of that stream.
//   * A lane's 16-byte load of codes is one group of 32 columns, so it takes
//     one scale byte, and the codes go from memory to registers without LDS.
//     gfx950's v_cvt_scalef32_pk_bf16_fp4 turns two codes into two scaled bf16
//     (exact: a 2-bit significand times a power of two) in one instruction:
//     half a vector instruction per weight.
//   * The products are 16x16x32 bf16 MFMAs with the weight rows as the first
//     operand and up to 16 routes as the second.  A contraction may run over
//     its columns in any order that both operands share: lane group q takes
//     columns 32q .. 32q+31 of a 128-wide step, which four MFMAs consume 8 at
//     a time, so both operands load straight from their rows.
//   * The workgroup's four waves split the contraction in 128-wide steps and
//     add their sums in wave order through LDS.  The split depends on the
//     contraction's length alone, so a route's result is the same, bit for
//     bit, whatever else is in the batch.
//   * FC1 pairs gate and up rows in one workgroup, so the SwiGLU and the
//     route's probability are applied to the sums in registers.
#include <algorithm>
#include <initializer_list>

#include "gemm_common.h"
#include "lowbit.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kW4Waves = 4;      // waves of a workgroup; they split the contraction
constexpr int kW4Step = 128;     // columns of a step: four lane groups of one scale group each

struct W4Args {
    const uint16_t* a;           // FC1: x [N, H]; FC2: act [R, I]
    const uint8_t* codes;        // [E, wrows, Kdim/2]
    const uint8_t* scales;       // [E, wrows, Kdim/32]
    const int* sorted_slot_ids;  // FC1 only
    const float* slot_probs;     // FC1 only
    const int* expert_ids;       // [R/BM]
    const int* block_start;      // [E]
    const int* route_counts;     // [E]
    void* out;                   // FC1: act bf16 [R, I]; FC2: route_out f32 [R, H]
    int N, Kdim, ncols, wrows, E, R;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                             static_cast<int>(bytes), kRsrcWord3);
}

// 8 codes (one word) as 8 bf16 times 2^(exponent of scale).
__device__ __forceinline__ bf16x8 w4_values(uint32_t word, float scale) {
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 0);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 1);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 2);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(word, scale, 3);
    bf16x8 r;
    r[0] = v0[0]; r[1] = v0[1]; r[2] = v1[0]; r[3] = v1[1];
    r[4] = v2[0]; r[5] = v2[1]; r[6] = v3[0]; r[7] = v3[1];
    return r;
}

// One workgroup: output columns 16*RT * blockIdx.x .. of the routes
// [rel*BM, rel*BM + 16*CT) of one expert, rel the layout block's place in the
// expert's segment.  WT weight tiles of 16 rows: FC1 has a gate and an up
// tile for each of its RT column tiles.
template <bool FC1, int RT, int CT>
__global__ __launch_bounds__(kW4Waves * kWave) void w4_gemm_kernel(W4Args p) {
    constexpr int WT = FC1 ? 2 * RT : RT;
    constexpr int U = CT == 1 ? 4 : 2;                  // steps whose loads are in flight together
    static_assert(CT <= 2 || CT % 2 == 0, "whole layout blocks");
    __shared__ floatx4 s_acc[kW4Waves][WT * CT][kWave];

    // the layout block's expert and rows: device data, range-checked
    const int b = blockIdx.y;
    const int e = p.expert_ids[b];
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.E)) return;      // past the extent
    const int rel = b - p.block_start[e];
    if (rel < 0 || rel % ((16 * CT + kBlockM - 1) / kBlockM) != 0) return;   // another workgroup's rows
    const int slot0 = b * kBlockM;
    const int n = min(min(p.route_counts[e] - rel * kBlockM, 16 * CT), p.R - slot0);
    if (n <= 0) return;

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int r16 = lane & 15, q = lane >> 4;
    const int col0 = blockIdx.x * (16 * RT);            // first output column

    // per-lane byte offsets of the weight rows (out-of-range rows read zeros)
    const int64_t base = static_cast<int64_t>(e) * p.wrows;
    const __amdgpu_buffer_rsrc_t crs = buffer(p.codes + base * (p.Kdim / 2), static_cast<uint32_t>(p.wrows) * (p.Kdim / 2));
    const __amdgpu_buffer_rsrc_t srs = buffer(p.scales + base * (p.Kdim / kGroup), static_cast<uint32_t>(p.wrows) * (p.Kdim / kGroup));
    uint32_t coff[WT], soff[WT];
#pragma unroll
    for (int t = 0; t < WT; ++t) {
        const int col = col0 + (FC1 ? t / 2 : t) * 16 + r16;
        const int row = FC1 && (t & 1) ? p.ncols + col : col;
        coff[t] = col < p.ncols ? static_cast<uint32_t>(row) * (p.Kdim / 2) + q * 16 : kOob;
        soff[t] = col < p.ncols ? static_cast<uint32_t>(row) * (p.Kdim / kGroup) + q : kOob;
    }
    // and of the routes' rows
    const __amdgpu_buffer_rsrc_t ars = FC1
        ? buffer(p.a, static_cast<uint32_t>(p.N) * p.Kdim * 2u)
        : buffer(p.a + static_cast<int64_t>(slot0) * p.Kdim, static_cast<uint32_t>(n) * p.Kdim * 2u);
    uint32_t aoff[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int i = c * 16 + r16;
        int row = i < n ? i : -1;
        if (FC1 && i < n) row = p.sorted_slot_ids[slot0 + i];
        const int rows = FC1 ? p.N : n;
        aoff[c] = static_cast<unsigned>(row) < static_cast<unsigned>(rows)
            ? static_cast<uint32_t>(row) * p.Kdim * 2u + q * 64 : kOob;
    }

    floatx4 acc[WT][CT];
#pragma unroll
    for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    // this wave's steps
    const int steps = (p.Kdim + kW4Step - 1) / kW4Step;
    const int lo = steps * wave / kW4Waves, hi = steps * (wave + 1) / kW4Waves;
    for (int k0 = lo; k0 < hi; k0 += U) {
        u32x4 cw[U][WT], xw[U][CT][4];
        uint32_t sb[U][WT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            // a lane group past the row's end, or a step past the wave's, reads zeros
            const bool live = k < hi && k * kW4Step + q * 32 < p.Kdim;
#pragma unroll
            for (int t = 0; t < WT; ++t) {
                cw[u][t] = __builtin_amdgcn_raw_buffer_load_b128(crs, live ? coff[t] + k * (kW4Step / 2) : kOob, 0, kStoreNT);
                sb[u][t] = __builtin_amdgcn_raw_buffer_load_b8(srs, live ? soff[t] + k * (kW4Step / kGroup) : kOob, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    xw[u][c][j] = __builtin_amdgcn_raw_buffer_load_b128(ars, live ? aoff[c] + k * (kW4Step * 2) + j * 16 : kOob, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < WT; ++t) {
                const float scale = __uint_as_float(sb[u][t] << 23);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 w = w4_values(cw[u][t][j], scale);
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            w, __builtin_bit_cast(bf16x8, xw[u][c][j]), acc[t][c], 0, 0, 0);
                }
            }
    }

    // the waves' sums, added in wave order
#pragma unroll
    for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) s_acc[wave][t * CT + c][lane] = acc[t][c];
    __syncthreads();
    auto sum = [&](int t, int c) {
        floatx4 v = s_acc[0][t * CT + c][lane];
#pragma unroll
        for (int w = 1; w < kW4Waves; ++w) v += s_acc[w][t * CT + c][lane];
        return v;
    };
    // lane: route c*16 + r16, output columns col0 + 16t + 4q .. +3
    for (int i = wave; i < RT * CT; i += kW4Waves) {
        const int t = i / CT, c = i % CT;
        const int route = c * 16 + r16, col = col0 + 16 * t + 4 * q;
        if (route >= n || col >= p.ncols) continue;
        const int64_t at = static_cast<int64_t>(slot0 + route) * p.ncols + col;
        if (FC1) {
            const floatx4 g = sum(2 * t, c), u = sum(2 * t + 1, c);
            const float pr = p.slot_probs[slot0 + route];
            uint2 o;
            o.x = pack_bf16x2(silu(g[0]) * u[0] * pr, silu(g[1]) * u[1] * pr);
            o.y = pack_bf16x2(silu(g[2]) * u[2] * pr, silu(g[3]) * u[3] * pr);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = o;
        } else {
            *reinterpret_cast<floatx4*>(static_cast<float*>(p.out) + at) = sum(t, c);
        }
    }
}

// y[t] = bf16( sum over k, from +0.0 in k order, of the token's routes ).
// One thread: 4 columns of one token.
template <int KMAX>
__global__ __launch_bounds__(256) void combine_f32_kernel(const float* __restrict__ route_out,
                                                          const int* __restrict__ token_routes, int N, int K,
                                                          int H, int R, uint16_t* __restrict__ y) {
    const int chunks = H / 4;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (item >= static_cast<int64_t>(N) * chunks) return;
    const int t = static_cast<int>(item / chunks);
    const int c = static_cast<int>(item - static_cast<int64_t>(t) * chunks);
    floatx4 v[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        const int r = k < K ? token_routes[static_cast<int64_t>(t) * K + k] : -1;
        v[k] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        if (r >= 0 && r < R)   // device data is range-checked, never trusted
            v[k] = *reinterpret_cast<const floatx4*>(route_out + static_cast<int64_t>(r) * H + c * 4);
    }
    floatx4 s = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < KMAX; ++k) s += v[k];
    uint2 o;
    o.x = pack_bf16x2(s[0], s[1]);
    o.y = pack_bf16x2(s[2], s[3]);
    *reinterpret_cast<uint2*>(y + static_cast<int64_t>(t) * H + c * 4) = o;
}

template <int KMAX>
void launch_combine_f32(const float* ro, const int* tr, int N, int K, int H, int R, uint16_t* y, hipStream_t s) {
    const int64_t items = static_cast<int64_t>(N) * (H / 4);
    combine_f32_kernel<KMAX><<<static_cast<unsigned>((items + 255) / 256), 256, 0, s>>>(ro, tr, N, K, H, R, y);
}

// Layout blocks that can hold routes: at most one partly filled block per
// expert in use beside the full ones.
int w4_blocks(int64_t N, int32_t E, int32_t K, int64_t R) {
    const int64_t routes = N * K;
    return static_cast<int>(std::min<int64_t>(R, routes + (kBlockM - 1) * std::min<int64_t>(E, routes)) / kBlockM);
}

int check_w4(int64_t N, int32_t H, int32_t I, int32_t E, int32_t K, int64_t* R) {
    if (N < 0 || E < 1 || K < 1 || K > E) return MOE_ERR_INVALID_ARG;
    const int st = check_dims(H, I);
    if (st != MOE_OK) return st;
    *R = moe_dropless_bound(N, K, E);
    if (*R < 0) return static_cast<int>(*R);
    const int64_t big = static_cast<int64_t>(1) << 31;
    if (*R > INT32_MAX || (N + 1) * H * 2 >= big || (N + kBlockM) * std::max(H, I) * 4 >= big ||
        static_cast<int64_t>(I) * H >= big)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_ptrs(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs) {
        if (!q) return MOE_ERR_INVALID_ARG;
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    }
    return MOE_OK;
}

template <bool FC1>
void launch_w4(W4Args& a, int blocks, double mean, hipStream_t s) {
    constexpr int RT = FC1 ? 2 : 4;
    const dim3 grid((a.ncols + 16 * RT - 1) / (16 * RT), blocks);
    if (mean > 32) w4_gemm_kernel<FC1, RT, 4><<<grid, kW4Waves * kWave, 0, s>>>(a);
    else w4_gemm_kernel<FC1, RT, 2><<<grid, kW4Waves * kWave, 0, s>>>(a);
}

int ffn_w4(int which, const uint16_t* x, const uint8_t* w1_codes, const uint8_t* w1_scales,
           const uint8_t* w2_codes, const uint8_t* w2_scales, const int32_t* ssi, const float* probs,
           const int32_t* expert_ids, const int32_t* block_start, const int32_t* route_counts,
           const int32_t* token_routes, int64_t N, int32_t H, int32_t I, int32_t E, int32_t K,
           uint16_t* act, float* route_out, uint16_t* y, hipStream_t stream) {
    int64_t R = 0;
    int st = check_w4(N, H, I, E, K, &R);
    if (st != MOE_OK) return st;
    if (N == 0) return MOE_OK;
    st = check_ptrs({expert_ids, block_start, route_counts, act});
    if (st == MOE_OK && (which & 1)) st = check_ptrs({x, w1_codes, w1_scales, ssi, probs});
    if (st == MOE_OK && (which & 2)) st = check_ptrs({w2_codes, w2_scales, route_out});
    if (st == MOE_OK && (which & 4)) st = check_ptrs({token_routes, y});
    if (st != MOE_OK) return st;
    const int blocks = w4_blocks(N, E, K, R);
    const double mean = static_cast<double>(N) * K / E;
    W4Args a{};
    a.expert_ids = expert_ids; a.block_start = block_start; a.route_counts = route_counts;
    a.N = static_cast<int>(N); a.E = E; a.R = static_cast<int>(R);
    if (which & 1) {
        a.a = x; a.codes = w1_codes; a.scales = w1_scales; a.sorted_slot_ids = ssi; a.slot_probs = probs;
        a.out = act; a.Kdim = H; a.ncols = I; a.wrows = 2 * I;
        launch_w4<true>(a, blocks, mean, stream);
    }
    if (which & 2) {
        a.a = act; a.codes = w2_codes; a.scales = w2_scales;
        a.out = route_out; a.Kdim = I; a.ncols = H; a.wrows = H;
        launch_w4<false>(a, blocks, mean, stream);
    }
    if (which & 4) return moe_gather_combine_f32(route_out, token_routes, N, K, H, R, y, stream);
    return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" int moe_gather_combine_f32(const float* route_out, const int32_t* token_routes, int64_t N,
                                      int32_t K, int32_t H, int64_t R, uint16_t* y, hipStream_t stream) {
    using namespace moe;
    if (N < 0 || K < 1 || H < 1 || R < 0) return MOE_ERR_INVALID_ARG;
    if (N > kMaxN || K > kMaxK || H % 64 || H > kMaxDim || R > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (N == 0) return MOE_OK;
    const int st = check_ptrs({route_out, token_routes, y});
    if (st != MOE_OK) return st;
    const int n = static_cast<int>(N), r = static_cast<int>(R);
    if (K <= 2) launch_combine_f32<2>(route_out, token_routes, n, K, H, r, y, stream);
    else if (K <= 4) launch_combine_f32<4>(route_out, token_routes, n, K, H, r, y, stream);
    else if (K <= 8) launch_combine_f32<8>(route_out, token_routes, n, K, H, r, y, stream);
    else if (K <= 16) launch_combine_f32<16>(route_out, token_routes, n, K, H, r, y, stream);
    else launch_combine_f32<32>(route_out, token_routes, n, K, H, r, y, stream);
    return launch_status();
}

extern "C" int moe_grouped_fc1_swiglu_w4(const uint16_t* x, const uint8_t* w1_codes, const uint8_t* w1_scales,
                                         const int32_t* sorted_slot_ids, const float* slot_probs,
                                         const int32_t* expert_ids, const int32_t* block_start,
                                         const int32_t* route_counts, int64_t N, int32_t H, int32_t I,
                                         int32_t E, int32_t K, uint16_t* act, hipStream_t stream) {
    return moe::ffn_w4(1, x, w1_codes, w1_scales, nullptr, nullptr, sorted_slot_ids, slot_probs, expert_ids,
                       block_start, route_counts, nullptr, N, H, I, E, K, act, nullptr, nullptr, stream);
}

extern "C" int moe_grouped_fc2_w4(const uint16_t* act, const uint8_t* w2_codes, const uint8_t* w2_scales,
                                  const int32_t* expert_ids, const int32_t* block_start,
                                  const int32_t* route_counts, int64_t N, int32_t H, int32_t I, int32_t E,
                                  int32_t K, float* route_out, hipStream_t stream) {
    return moe::ffn_w4(2, nullptr, nullptr, nullptr, w2_codes, w2_scales, nullptr, nullptr, expert_ids,
                       block_start, route_counts, nullptr, N, H, I, E, K, const_cast<uint16_t*>(act), route_out,
                       nullptr, stream);
}

extern "C" int moe_grouped_ffn_w4(const uint16_t* x, const uint8_t* w1_codes, const uint8_t* w1_scales,
                                  const uint8_t* w2_codes, const uint8_t* w2_scales,
                                  const int32_t* sorted_slot_ids, const float* slot_probs,
                                  const int32_t* expert_ids, const int32_t* block_start,
                                  const int32_t* route_counts, const int32_t* token_routes, int64_t N,
                                  int32_t H, int32_t I, int32_t E, int32_t K, uint16_t* act, float* route_out,
                                  uint16_t* y, hipStream_t stream) {
    return moe::ffn_w4(7, x, w1_codes, w1_scales, w2_codes, w2_scales, sorted_slot_ids, slot_probs, expert_ids,
                       block_start, route_counts, token_routes, N, H, I, E, K, act, route_out, y, stream);
}

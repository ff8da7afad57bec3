// The gradients' global norm and the AdamW step over many tensors.
//
//   norm = sqrt(sum g^2);  c = min(1, max_norm / norm);  t = step + 1
//   m = b1 m + (1 - b1) c g;  v = b2 v + (1 - b2) (c g)^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// HBM-bound: every byte of state is read and written once.  Tensors are cut
// into chunks of a fixed length, a workgroup a chunk, and a launch takes up to
// kBatch tensors, whose table travels in the kernel's arguments: no table to
// upload, nothing to keep, and a captured call replays what it was given.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "gemm_common.h"
#include "lowbit.h"
#include "../../include/moe_block.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kEach = 4;                             // elements of a lane's piece
constexpr int kPieces = 4;                           // pieces of a lane
constexpr int kChunk = kThreads * kEach * kPieces;   // elements of a workgroup
constexpr int kNormPieces = 16;
constexpr int kNormChunk = kThreads * kEach * kNormPieces;
constexpr int kBatch = 44;                           // tensors of a launch (the arguments hold 4 KB)
constexpr int64_t kMaxBlocks = int64_t(1) << 23;     // workgroups of a launch: a grid holds under 2^32 threads
constexpr int64_t kMaxElements = int64_t(1) << 34;

struct AdamWEntry {
    void* param;
    float* master;
    const void* grad;
    void *m, *v;
    uint8_t *m_scales, *v_scales;
    int64_t n;
    float weight_decay;
    int32_t types;                                   // bit 0: float32 param, bit 1: float32 gradient
};

struct AdamWBatch {
    AdamWEntry e[kBatch];
    int32_t first[kBatch];                           // first workgroup of each tensor; INT32_MAX past the last
    const float* lr;
    const float* grad_norm;
    int32_t* step;
    uint32_t* ticket;                                // null: not the last launch
    double log2_beta1, log2_beta2;                   // -inf for beta 0
    float beta1, beta2, one_less_beta1, one_less_beta2, eps, max_norm;
};
static_assert(sizeof(AdamWBatch) <= 4096, "kernel arguments");

struct GradBatch {
    const void* grad[kBatch];
    int64_t n[kBatch];
    int32_t first[kBatch];
    int32_t f32[kBatch];
    double* part;                                    // of this launch's first workgroup
};

// The tensor of a workgroup: the last one that begins at or before it.
__device__ __forceinline__ int find_tensor(const int32_t* first) {
    const int lane = lane_id();
    const int f = lane < kBatch ? first[lane] : INT32_MAX;
    const uint64_t begun = __ballot(f <= static_cast<int>(blockIdx.x));
    return __builtin_amdgcn_readfirstlane(static_cast<int>(__popcll(begun)) - 1);
}

// Elements i .. i+3 of a tensor of n; those past the end are 0.
__device__ __forceinline__ floatx4 load4(const float* p, int64_t i, int64_t n) {
    if (i + kEach <= n) return *reinterpret_cast<const floatx4*>(p + i);
    floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) v[j] = p[i + j];
    return v;
}
__device__ __forceinline__ floatx4 load4(const uint16_t* p, int64_t i, int64_t n) {
    floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (i + kEach <= n) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p + i);
#pragma unroll
        for (int j = 0; j < kEach; ++j) v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
        return v;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) v[j] = bf16_to_f32(p[i + j]);
    return v;
}
__device__ __forceinline__ uint32_t load4(const uint8_t* p, int64_t i, int64_t n) {
    if (i + kEach <= n) return *reinterpret_cast<const uint32_t*>(p + i);
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) v |= static_cast<uint32_t>(p[i + j]) << (8 * j);
    return v;
}
__device__ __forceinline__ floatx4 load4_as(const void* p, bool f32, int64_t i, int64_t n) {
    return f32 ? load4(static_cast<const float*>(p), i, n) : load4(static_cast<const uint16_t*>(p), i, n);
}
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, floatx4 v) {
    if (i + kEach <= n) {
        *reinterpret_cast<floatx4*>(p + i) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) p[i + j] = v[j];
}
__device__ __forceinline__ void store4(uint16_t* p, int64_t i, int64_t n, floatx4 v) {
    if (i + kEach <= n) {
        u32x2 w;
        w[0] = pack_bf16x2(v[0], v[1]);
        w[1] = pack_bf16x2(v[2], v[3]);
        *reinterpret_cast<u32x2*>(p + i) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) p[i + j] = f32_to_bf16(v[j]);
}
__device__ __forceinline__ void store4(uint8_t* p, int64_t i, int64_t n, uint32_t v) {
    if (i + kEach <= n) {
        *reinterpret_cast<uint32_t*>(p + i) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) p[i + j] = static_cast<uint8_t>(v >> (8 * j));
}

// ---------------------------------------------------------------- moments in 8 bits
// A group of 32 elements is 8 neighbouring lanes' pieces.

// The largest magnitude's bits over a group (NaN above infinity above numbers).
__device__ __forceinline__ uint32_t group_max(floatx4 v) {
    uint32_t m = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
#pragma unroll
    for (int o = 1; o < kGroup / kEach; o <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o)));
    return m;
}

// e4m3: 448 = 1.75 * 2^8 is the largest, 464 = 1.8125 * 2^8 would round past it.
__device__ __forceinline__ int first_scale(uint32_t amax) { return scale_byte<0x180000u, 8>(amax); }
__device__ __forceinline__ uint32_t first_codes(floatx4 v, int b) {
    const float inv = inv_scale(b);
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, w, true);
    return b == kScaleNaN ? 0u : static_cast<uint32_t>(w);
}
__device__ __forceinline__ floatx4 first_values(uint32_t w, uint32_t b) {
    const float s = scale_value(b);
    floatx4 v;
    v[0] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 0) * s;
    v[1] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 1) * s;
    v[2] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 2) * s;
    v[3] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 3) * s;
    return v;
}

// Unsigned e4m4 without subnormals: the exponent and the upper four bits of the
// mantissa of a float in [2^-15, 2), counted from 2^-15 on; code 0 is 0.
__device__ __forceinline__ int root_scale(uint32_t amax) { return scale_byte<0x40000u, 0>(amax); }
__device__ __forceinline__ uint32_t root_code(float r, float inv) {
    const int bits = __float_as_int(r * inv);
    const int c = ((bits + 0x3FFFF + (bits >> 19 & 1)) >> 19) - 112 * 16;
    return r > 0.0f ? static_cast<uint32_t>(max(c, 1)) : 0u;
}
__device__ __forceinline__ uint32_t root_codes(floatx4 r, int b) {
    const float inv = inv_scale(b);
    const uint32_t w = root_code(r[0], inv) | root_code(r[1], inv) << 8 | root_code(r[2], inv) << 16 | root_code(r[3], inv) << 24;
    return b == kScaleNaN ? 0u : w;
}
__device__ __forceinline__ floatx4 root_values(uint32_t w, uint32_t b) {
    const float s = scale_value(b);
    floatx4 v;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const uint32_t c = w >> (8 * j) & 255u;
        v[j] = (c ? __uint_as_float((c << 19) + (112u << 23)) : 0.0f) * s;
    }
    return v;
}

// ---------------------------------------------------------------- gradient norm

__device__ __forceinline__ double block_sum(double v, double* s_part) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    if (lane_id() == 0) s_part[threadIdx.x / kWave] = v;
    __syncthreads();
    double t = 0.0;
    for (unsigned i = 0; i < blockDim.x / kWave; ++i) t += s_part[i];
    return t;
}

__global__ __launch_bounds__(kThreads) void grad_square_kernel(GradBatch b) {
    __shared__ double s_part[kThreads / kWave];
    const int k = find_tensor(b.first);
    const int64_t n = b.n[k], base = static_cast<int64_t>(static_cast<int>(blockIdx.x) - b.first[k]) * kNormChunk;
    const bool f32 = b.f32[k] != 0;
    const void* g = b.grad[k];
    double s[kEach] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
    for (int i = 0; i < kNormPieces; ++i) {
        const floatx4 v = load4_as(g, f32, base + (i * kThreads + static_cast<int>(threadIdx.x)) * kEach, n);
#pragma unroll
        for (int j = 0; j < kEach; ++j) s[j] += static_cast<double>(v[j]) * static_cast<double>(v[j]);
    }
    const double t = block_sum((s[0] + s[1]) + (s[2] + s[3]), s_part);
    if (threadIdx.x == 0) b.part[blockIdx.x] = t;
}

constexpr int kFinishThreads = 1024;
__global__ __launch_bounds__(kFinishThreads) void grad_norm_kernel(const double* __restrict__ part, int64_t n,
                                                                   float* __restrict__ norm) {
    __shared__ double s_part[kFinishThreads / kWave];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kFinishThreads) s += part[i];
    s = block_sum(s, s_part);
    if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(s));
}

// ---------------------------------------------------------------- AdamW

// One piece: the moments and the parameter's new value.
struct AdamWScalars {
    float clip, beta1, beta2, one_less_beta1, one_less_beta2, eps, keep, rate, inv_root_bc2;
    __device__ __forceinline__ void update(floatx4 g, floatx4& m, floatx4& v, floatx4& root, floatx4& p) const {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const float x = g[j] * clip;
            m[j] = beta1 * m[j] + one_less_beta1 * x;
            v[j] = beta2 * v[j] + one_less_beta2 * x * x;
            root[j] = __builtin_sqrtf(v[j]);
            p[j] = p[j] * keep - rate * (m[j] / (root[j] * inv_root_bc2 + eps));
        }
    }
};

template <bool Q8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamWBatch b) {
    const float norm = b.grad_norm ? b.grad_norm[0] : 0.0f;
    // infinite or NaN: nothing is written, the step is not taken
    if ((__float_as_uint(norm) & 0x7F800000u) == 0x7F800000u) return;
    const int t = __builtin_amdgcn_readfirstlane(b.step[0]) + 1;
    const int k = find_tensor(b.first);
    if (k >= 0) {                                    // (a launch of empty tensors alone has none)
        const AdamWEntry& e = b.e[k];
        const int64_t n = e.n, base = static_cast<int64_t>(static_cast<int>(blockIdx.x) - b.first[k]) * kChunk;
        const bool f32 = (e.types & 1) != 0, g32 = (e.types & 2) != 0;
        floatx4 g[kPieces], p[kPieces], m[kPieces], v[kPieces];
        uint32_t mc[kPieces], vc[kPieces], mb[kPieces], vb[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int64_t at = base + (i * kThreads + static_cast<int>(threadIdx.x)) * kEach;
            g[i] = load4_as(e.grad, g32, at, n);
            p[i] = e.master ? load4(e.master, at, n) : load4_as(e.param, f32, at, n);
            if (Q8) {
                mc[i] = load4(static_cast<const uint8_t*>(e.m), at, n);
                vc[i] = load4(static_cast<const uint8_t*>(e.v), at, n);
                mb[i] = at < n ? e.m_scales[at / kGroup] : 1;
                vb[i] = at < n ? e.v_scales[at / kGroup] : 1;
            } else {
                m[i] = load4(static_cast<const float*>(e.m), at, n);
                v[i] = load4(static_cast<const float*>(e.v), at, n);
            }
        }
        AdamWScalars s;
        const float lr = b.lr[0];
        const double bc1 = 1.0 - exp2(t * b.log2_beta1), bc2 = 1.0 - exp2(t * b.log2_beta2);
        s.clip = norm > b.max_norm ? b.max_norm / norm : 1.0f;
        s.beta1 = b.beta1; s.beta2 = b.beta2;
        s.one_less_beta1 = b.one_less_beta1; s.one_less_beta2 = b.one_less_beta2;
        s.eps = b.eps;
        s.keep = 1.0f - lr * e.weight_decay;
        s.rate = static_cast<float>(lr / bc1);
        s.inv_root_bc2 = static_cast<float>(1.0 / sqrt(bc2));
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int64_t at = base + (i * kThreads + static_cast<int>(threadIdx.x)) * kEach;
            if (Q8) {
                m[i] = first_values(mc[i], mb[i]);
                v[i] = root_values(vc[i], vb[i]);
                v[i] *= v[i];
            }
            floatx4 root;
            s.update(g[i], m[i], v[i], root, p[i]);
            if (Q8) {
                // elements past the end are zeros and take no part in the scale
                const int bm = first_scale(group_max(m[i])), br = root_scale(group_max(root));
                store4(static_cast<uint8_t*>(e.m), at, n, first_codes(m[i], bm));
                store4(static_cast<uint8_t*>(e.v), at, n, root_codes(root, br));
                if (at < n && at % kGroup == 0) {
                    e.m_scales[at / kGroup] = static_cast<uint8_t>(bm);
                    e.v_scales[at / kGroup] = static_cast<uint8_t>(br);
                }
            } else {
                store4(static_cast<float*>(e.m), at, n, m[i]);
                store4(static_cast<float*>(e.v), at, n, v[i]);
            }
            if (e.master) store4(e.master, at, n, p[i]);
            if (f32) store4(static_cast<float*>(e.param), at, n, p[i]);
            else store4(static_cast<uint16_t*>(e.param), at, n, p[i]);
        }
    }
    // all waves of a workgroup have read the step when it counts itself; the last
    // one to do so moves it
    if (!b.ticket) return;
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(b.ticket, 1u) == gridDim.x - 1) {
        b.step[0] = t;
        b.ticket[0] = 0u;
    }
}

__global__ __launch_bounds__(kThreads) void moment_values_kernel(const uint8_t* __restrict__ m, const uint8_t* __restrict__ ms,
                                                                 const uint8_t* __restrict__ v, const uint8_t* __restrict__ vs,
                                                                 int64_t n, uint16_t* __restrict__ mo, uint16_t* __restrict__ ro) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * kEach;
    if (at >= n) return;
    store4(mo, at, n, first_values(load4(m, at, n), ms[at / kGroup]));
    store4(ro, at, n, root_values(load4(v, at, n), vs[at / kGroup]));
}

__global__ __launch_bounds__(kThreads) void moment_codes_kernel(const float* __restrict__ m, const float* __restrict__ v,
                                                                int64_t n, uint8_t* __restrict__ mc, uint8_t* __restrict__ ms,
                                                                uint8_t* __restrict__ vc, uint8_t* __restrict__ vs) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * kEach;
    const floatx4 a = load4(m, at, n);
    floatx4 r = load4(v, at, n);
#pragma unroll
    for (int j = 0; j < kEach; ++j) r[j] = __builtin_sqrtf(r[j]);
    const int bm = first_scale(group_max(a)), br = root_scale(group_max(r));
    store4(mc, at, n, first_codes(a, bm));
    store4(vc, at, n, root_codes(r, br));
    if (at < n && at % kGroup == 0) {
        ms[at / kGroup] = static_cast<uint8_t>(bm);
        vs[at / kGroup] = static_cast<uint8_t>(br);
    }
}

// ---------------------------------------------------------------- host side

bool is_type(int32_t t) { return t == MOE_BF16 || t == MOE_F32; }
int64_t chunks(int64_t n, int chunk) { return (n + chunk - 1) / chunk; }

int check_list(const moe_adamw_tensor* t, int32_t count) {
    if (count < 0 || (count > 0 && !t)) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        if (t[i].n < 0 || !is_type(t[i].grad_type) || t[i].reserved != 0) return MOE_ERR_INVALID_ARG;
        if (t[i].n > kMaxElements) return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

int check_pointers(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs)
        if (!q) return MOE_ERR_INVALID_ARG;
    for (const void* q : ptrs)
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace moe

extern "C" size_t moe_grad_norm_workspace_bytes(const moe_adamw_tensor* tensors, int32_t count) {
    if (moe::check_list(tensors, count) != MOE_OK) return 0;
    int64_t n = 0;
    for (int i = 0; i < count; ++i) n += moe::chunks(tensors[i].n, moe::kNormChunk);
    return static_cast<size_t>(std::max<int64_t>(n, 2)) * sizeof(double);
}

extern "C" int moe_grad_norm(const moe_adamw_tensor* tensors, int32_t count, void* workspace,
                             size_t workspace_bytes, float* norm, hipStream_t stream) {
    using namespace moe;
    int st = check_list(tensors, count);
    if (st != MOE_OK) return st;
    for (int i = 0; i < count; ++i)
        if (tensors[i].n > 0 && (st = check_pointers({tensors[i].grad})) != MOE_OK) return st;
    st = check_pointers({workspace});
    if (st != MOE_OK) return st;
    if (!norm || workspace_bytes < moe_grad_norm_workspace_bytes(tensors, count)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(norm)) return MOE_ERR_MISALIGNED;
    int64_t total = 0;
    GradBatch b;
    int used = 0;
    int64_t blocks = 0;
    auto flush = [&]() {
        if (!used) return;
        for (int i = used; i < kBatch; ++i) b.first[i] = INT32_MAX;
        b.part = static_cast<double*>(workspace) + total;
        grad_square_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(b);
        total += blocks;
        used = 0;
        blocks = 0;
    };
    for (int i = 0; i < count; ++i) {
        const int64_t c = chunks(tensors[i].n, kNormChunk);
        if (c == 0) continue;
        if (used == kBatch || blocks + c > kMaxBlocks) flush();
        b.grad[used] = tensors[i].grad;
        b.n[used] = tensors[i].n;
        b.f32[used] = tensors[i].grad_type;
        b.first[used++] = static_cast<int32_t>(blocks);
        blocks += c;
    }
    flush();
    grad_norm_kernel<<<1, kFinishThreads, 0, stream>>>(static_cast<const double*>(workspace), total, norm);
    return launch_status();
}

extern "C" int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, int32_t state, const float* lr,
                              double beta1, double beta2, double eps, const float* grad_norm, double max_norm,
                              int32_t* step, uint32_t* ticket, hipStream_t stream) {
    using namespace moe;
    int st = check_list(tensors, count);
    if (st != MOE_OK) return st;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
        (grad_norm && !(max_norm > 0.0)))
        return MOE_ERR_INVALID_ARG;
    if (state != 32 && state != 8) return MOE_ERR_INVALID_ARG;
    if (!lr || !step || !ticket) return MOE_ERR_INVALID_ARG;
    if (!aligned4(lr) || !aligned4(step) || !aligned4(ticket) || !aligned4(grad_norm)) return MOE_ERR_MISALIGNED;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (!is_type(t.param_type) || !std::isfinite(t.weight_decay)) return MOE_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if ((st = check_pointers({t.param, t.grad, t.m, t.v})) != MOE_OK) return st;
        if (t.master && !aligned16(t.master)) return MOE_ERR_MISALIGNED;
        if (state == 8 ? !t.m_scales || !t.v_scales : t.m_scales || t.v_scales) return MOE_ERR_INVALID_ARG;
    }
    AdamWBatch b;
    b.lr = lr; b.grad_norm = grad_norm; b.step = step;
    b.log2_beta1 = std::log2(beta1); b.log2_beta2 = std::log2(beta2);
    b.beta1 = static_cast<float>(beta1); b.beta2 = static_cast<float>(beta2);
    b.one_less_beta1 = static_cast<float>(1.0 - beta1); b.one_less_beta2 = static_cast<float>(1.0 - beta2);
    b.eps = static_cast<float>(eps);
    b.max_norm = grad_norm ? static_cast<float>(max_norm) : 0.0f;
    int used = 0;
    int64_t blocks = 0;
    auto flush = [&](bool last) {
        if (!used && !last) return;
        for (int i = used; i < kBatch; ++i) b.first[i] = INT32_MAX;
        b.ticket = last ? ticket : nullptr;
        const unsigned g = static_cast<unsigned>(std::max<int64_t>(blocks, 1));
        if (state == 8) adamw_kernel<true><<<g, kThreads, 0, stream>>>(b);
        else adamw_kernel<false><<<g, kThreads, 0, stream>>>(b);
        used = 0;
        blocks = 0;
    };
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        const int64_t c = chunks(t.n, kChunk);
        if (c == 0) continue;
        if (used == kBatch || blocks + c > kMaxBlocks) flush(false);
        b.e[used] = AdamWEntry{t.param, t.master, t.grad, t.m, t.v, t.m_scales, t.v_scales, t.n, t.weight_decay,
                               (t.param_type == MOE_F32 ? 1 : 0) | (t.grad_type == MOE_F32 ? 2 : 0)};
        b.first[used++] = static_cast<int32_t>(blocks);
        blocks += c;
    }
    flush(true);
    return launch_status();
}

namespace moe {
namespace {
int check_moments(int64_t n, std::initializer_list<const void*> ptrs, const uint8_t* ms, const uint8_t* vs) {
    if (n < 0) return MOE_ERR_INVALID_ARG;
    if (n > kMaxElements) return MOE_ERR_UNSUPPORTED;
    if (n == 0) return MOE_OK;
    const int st = check_pointers(ptrs);
    return st != MOE_OK ? st : ms && vs ? MOE_OK : MOE_ERR_INVALID_ARG;
}
unsigned moment_blocks(int64_t n) { return static_cast<unsigned>((n + kThreads * kEach - 1) / (kThreads * kEach)); }
}  // namespace
}  // namespace moe

extern "C" int moe_moment_values(const uint8_t* m, const uint8_t* m_scales, const uint8_t* v,
                                 const uint8_t* v_scales, int64_t n, uint16_t* m_values, uint16_t* root_values,
                                 hipStream_t stream) {
    using namespace moe;
    const int st = check_moments(n, {m, v, m_values, root_values}, m_scales, v_scales);
    if (st != MOE_OK || n == 0) return st;
    moment_values_kernel<<<moment_blocks(n), kThreads, 0, stream>>>(m, m_scales, v, v_scales, n, m_values, root_values);
    return launch_status();
}

extern "C" int moe_moment_codes(const float* m, const float* v, int64_t n, uint8_t* m_codes, uint8_t* m_scales,
                                uint8_t* v_codes, uint8_t* v_scales, hipStream_t stream) {
    using namespace moe;
    const int st = check_moments(n, {m, v, m_codes, v_codes}, m_scales, v_scales);
    if (st != MOE_OK || n == 0) return st;
    moment_codes_kernel<<<moment_blocks(n), kThreads, 0, stream>>>(m, v, n, m_codes, m_scales, v_codes, v_scales);
    return launch_status();
}

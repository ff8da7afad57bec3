// The gradients' global norm and the AdamW step over many tensors.
//
//   norm = sqrt(sum g^2);  c = min(1, max_norm / norm);  t = step + 1
//   m = b1 m + (1 - b1) c g;  v = b2 v + (1 - b2) (c g)^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// HBM-bound: every byte of state is read and written once.  Tensors are cut
// into chunks, a workgroup a chunk, and one launch takes all of them whatever
// their sizes: a plan in device memory names each chunk's tensor, so a
// workgroup finds its work in two dependent loads.  (A table in the kernel's
// arguments takes 44 tensors a launch and is read from host memory: 300 small
// tensors 14 launches, 104 us.)
//
// Measured: 75.5 M elements with bf16 parameters, float32 master copies and
// gradients: norm 41 to 55 us (5.5 to 7.4 TB/s; behind a step that has just written
// everything, its reads compete with the write-back), step 390 with moments in 32
// bits (6.2 TB/s), in 8 222 rounded to nearest (6.2), 227 at random; 300 tensors of
// 2.9 M elements in all: 6.7 + 14.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <utility>
#include <vector>

#include "gemm_common.h"
#include "lowbit.h"
#include "../../include/moe_moments.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kEach = 8;                             // elements of a lane's piece
constexpr int kPieces = 2;                           // pieces of a lane
constexpr int kChunk = kThreads * kEach * kPieces;   // elements of a workgroup
constexpr int kBatch = 44;                           // entries of a launch that writes a plan (arguments hold 4 KB)
constexpr int kNormBlocks = 2048;                    // workgroups of the norm, at most: eight a compute unit
constexpr int64_t kMaxBlocks = int64_t(1) << 23;     // workgroups of a launch: a grid holds under 2^32 threads
constexpr int64_t kMaxElements = int64_t(1) << 34;   // of a tensor
constexpr int64_t kMaxChunks = int64_t(1) << 28;     // of all

// A chunk: its pieces of a tensor.
struct Chunk {
    void* param;
    float* master;
    const void* grad;
    void *m, *v;
    uint8_t *m_scales, *v_scales;
    int32_t n;                                       // elements, up to kChunk
    int32_t types;                                   // bit 0: float32 param, bit 1: float32 gradient
    float weight_decay;
    int32_t pad;
};
static_assert(sizeof(Chunk) == 72, "layout");

// Counts the workgroups of a launch that are done.  Atomics on one address take
// turns, so workgroups count in kGroups groups, and the last of a group counts
// for it.  Every counter has its cache lines to itself: with the chunks beside it
// each atomic took them from the other XCDs' caches (75 M elements 1590 us
// against 390).
struct Line {
    uint32_t n, pad[31];
};
constexpr uint32_t kGroups = 32;
struct Counter {
    Line group[kGroups], all;
    __device__ __forceinline__ void reset() {
        for (uint32_t i = 0; i < kGroups; ++i) group[i].n = 0u;
        all.n = 0u;
    }
    // Whether this workgroup is the last of `total` to come here; leaves zeros then.
    __device__ __forceinline__ bool last(uint32_t me, uint32_t total) {
        const uint32_t g = me % kGroups, members = (total - g + kGroups - 1) / kGroups;
        if (count(&group[g].n) != members - 1) return false;
        clear(&group[g].n);
        if (count(&all.n) != min(total, kGroups) - 1) return false;
        clear(&all.n);
        return true;
    }
    static __device__ __forceinline__ uint32_t count(uint32_t* p) {
        return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    static __device__ __forceinline__ void clear(uint32_t* p) {
        __hip_atomic_store(p, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

// A plan: the norm's partial sums, the counters, then the chunks.
struct PlanHead {
    double part[kNormBlocks];
    Counter norm_done, step_done;
};
static_assert(sizeof(PlanHead) % 128 == 0, "whole lines");
struct Plan {
    PlanHead* head;
    __host__ __device__ Chunk* chunk() const { return reinterpret_cast<Chunk*>(head + 1); }
};

// Writing it: up to kBatch tensors a launch, a workgroup each.
struct Entry {
    Chunk all;                                       // (all.n is not used)
    int64_t n;
    int32_t first;                                   // chunk
    int32_t state;
};
struct PlanBatch {
    Entry e[kBatch];
};
static_assert(sizeof(PlanBatch) + 8 <= 4096, "kernel arguments");

__global__ void plan_reset_kernel(PlanHead* head) {
    head->norm_done.reset();
    head->step_done.reset();
}

__global__ __launch_bounds__(kThreads) void plan_kernel(PlanBatch b, Plan plan) {
    const Entry e = b.e[blockIdx.x];
    const int32_t chunks = static_cast<int32_t>((e.n + kChunk - 1) / kChunk);
    for (int32_t i = threadIdx.x; i < chunks; i += kThreads) {
        const int64_t at = static_cast<int64_t>(i) * kChunk;
        auto bytes_on = [&](auto* p, int size) {
            return reinterpret_cast<decltype(p)>(reinterpret_cast<uintptr_t>(p) + (p ? at * size : 0));
        };
        const int state = e.state == 8 ? 1 : 4;
        Chunk c = e.all;
        c.param = bytes_on(c.param, c.types & 1 ? 4 : 2);
        c.master = bytes_on(c.master, 4);
        c.grad = bytes_on(c.grad, c.types & 2 ? 4 : 2);
        c.m = bytes_on(c.m, state);
        c.v = bytes_on(c.v, state);
        if (c.m_scales) c.m_scales += at / kGroup;
        if (c.v_scales) c.v_scales += at / kGroup;
        c.n = static_cast<int32_t>(e.n - at < kChunk ? e.n - at : kChunk);
        plan.chunk()[e.first + i] = c;
    }
}

// Elements i .. i+7 of n, as two halves; those past the end are 0.
struct Eight {
    floatx4 h[2];
    __device__ __forceinline__ float& operator[](int j) { return reinterpret_cast<float*>(h)[j]; }
    __device__ __forceinline__ float operator[](int j) const { return reinterpret_cast<const float*>(h)[j]; }
};
__device__ __forceinline__ Eight load8(const float* p, int i, int n) {
    Eight v;
    if (i + kEach <= n) {
        v.h[0] = reinterpret_cast<const floatx4*>(p + i)[0];
        v.h[1] = reinterpret_cast<const floatx4*>(p + i)[1];
        return v;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = i + j < n ? p[i + j] : 0.0f;
    return v;
}
__device__ __forceinline__ Eight load8(const uint16_t* p, int i, int n) {
    Eight v;
    if (i + kEach <= n) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
        for (int j = 0; j < kEach; ++j) v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
        return v;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.0f;
    return v;
}
__device__ __forceinline__ u32x2 load8(const uint8_t* p, int i, int n) {
    if (i + kEach <= n) return *reinterpret_cast<const u32x2*>(p + i);
    u32x2 v = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) v[j / 4] |= static_cast<uint32_t>(p[i + j]) << (8 * (j % 4));
    return v;
}
__device__ __forceinline__ Eight load8_as(const void* p, bool f32, int i, int n) {
    return f32 ? load8(static_cast<const float*>(p), i, n) : load8(static_cast<const uint16_t*>(p), i, n);
}
__device__ __forceinline__ void store8(float* p, int i, int n, const Eight& v) {
    if (i + kEach <= n) {
        reinterpret_cast<floatx4*>(p + i)[0] = v.h[0];
        reinterpret_cast<floatx4*>(p + i)[1] = v.h[1];
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) p[i + j] = v[j];
}
__device__ __forceinline__ void store8(uint16_t* p, int i, int n, const Eight& v) {
    if (i + kEach <= n) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < kEach; j += 2) w[j / 2] = pack_bf16x2(v[j], v[j + 1]);
        *reinterpret_cast<u32x4*>(p + i) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) p[i + j] = f32_to_bf16(v[j]);
}
__device__ __forceinline__ void store8(uint8_t* p, int i, int n, u32x2 v) {
    if (i + kEach <= n) {
        *reinterpret_cast<u32x2*>(p + i) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (i + j < n) p[i + j] = static_cast<uint8_t>(v[j / 4] >> (8 * (j % 4)));
}

// ---------------------------------------------------------------- moments in 8 bits
// A group of 32 elements is 4 neighbouring lanes' pieces.

// The largest magnitude's bits over a group (NaN above infinity above numbers).
__device__ __forceinline__ uint32_t group_max(const Eight& v) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) m = max(m, abs_bits(v[j]));
#pragma unroll
    for (int o = 1; o < kGroup / kEach; o <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o)));
    return m;
}

// e4m3: 448 = 1.75 * 2^8 is the largest, 464 = 1.8125 * 2^8 would round past it.
__device__ __forceinline__ int first_scale(uint32_t amax) { return scale_byte<0x180000u, 8>(amax); }
__device__ __forceinline__ u32x2 first_codes(const Eight& v, int b) {
    const float inv = inv_scale(b);
    u32x2 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, w, true);
        o[i] = b == kScaleNaN ? 0u : static_cast<uint32_t>(w);
    }
    return o;
}
__device__ __forceinline__ Eight first_values(u32x2 w, uint32_t b) {
    const float s = scale_value(b);
    Eight v;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = static_cast<int>(w[i]);
        v[4 * i] = __builtin_amdgcn_cvt_f32_fp8(c, 0) * s;
        v[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(c, 1) * s;
        v[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(c, 2) * s;
        v[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(c, 3) * s;
    }
    return v;
}

// Both scales without room for rounding past the largest code: a magnitude above
// 448, 1.9375 for a root, goes to the next.
__device__ __forceinline__ int first_scale_above(uint32_t amax) { return scale_byte<0x1FFFFFu, 8>(amax); }
__device__ __forceinline__ int root_scale_above(uint32_t amax) { return scale_byte<0x7FFFFu, 0>(amax); }

// Unsigned e4m4 without subnormals: the exponent and the upper four bits of the
// mantissa of a float in [2^-15, 2), counted from 2^-15 on; code 0 is 0.
__device__ __forceinline__ int root_scale(uint32_t amax) { return scale_byte<0x40000u, 0>(amax); }
__device__ __forceinline__ u32x2 root_codes(const Eight& r, int b) {
    const float inv = inv_scale(b);
    u32x2 o = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int bits = __float_as_int(r[j] * inv);
        const int c = ((bits + 0x3FFFF + (bits >> 19 & 1)) >> 19) - 112 * 16;
        o[j / 4] |= (r[j] > 0.0f ? static_cast<uint32_t>(max(c, 1)) : 0u) << (8 * (j % 4));
    }
    return b == kScaleNaN ? u32x2{0u, 0u} : o;
}
__device__ __forceinline__ Eight root_values(u32x2 w, uint32_t b) {
    const float s = scale_value(b);
    Eight v;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const uint32_t c = w[j / 4] >> (8 * (j % 4)) & 255u;
        v[j] = (c ? __uint_as_float((c << 19) + (112u << 23)) : 0.0f) * s;
    }
    return v;
}

// Stochastic rounding.  32 random bits serve both moments: the upper 20 the first
// one, the lower 24 the root, each of which decides by its own upper bits but once
// in 256 times (their decisions' correlation is 0.004).  A bijection whose results'
// bits all depend on all of x; the constants are 2^32 times the fractions of the
// roots of 2 and 3 and of the golden ratio.
constexpr uint32_t kGolden = 0x9E3779B9u;
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ x >> 16;
}
__device__ __forceinline__ uint32_t chunk_key(uint32_t seed, uint32_t t, uint32_t chunk) {
    return mix(mix(seed + kGolden * t) + chunk);
}

// e4m3 keeps 20 bits less of the mantissa, from 2^-6 on; below, 2^-6 is added, which
// brings the values to where the codes are as far apart.  Random bits are added to
// the bits that go, and carry with the probability of what those are worth.
__device__ __forceinline__ float first_random(float a, uint32_t h) {
    const float m = __builtin_fabsf(a), shift = m < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t bits = (__float_as_uint(m + shift) + (h >> 12)) & 0xFFF00000u;
    return __builtin_copysignf(__uint_as_float(bits) - shift, a);
}
__device__ __forceinline__ u32x2 first_codes_random(const Eight& v, int b, uint32_t key, int at) {
    const float inv = inv_scale(b);
    Eight r;
#pragma unroll
    for (int j = 0; j < kEach; ++j) r[j] = first_random(v[j] * inv, mix(key + kGolden * static_cast<uint32_t>(at + j)));
    u32x2 o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {                        // exact: they are codes' values
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(r[4 * i], r[4 * i + 1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(r[4 * i + 2], r[4 * i + 3], w, true);
        o[i] = b == kScaleNaN ? 0u : static_cast<uint32_t>(w);
    }
    return o;
}
// The root's code below and the one above, which is taken where the random fraction
// of the way between their squares has not reached the root's square.
__device__ __forceinline__ u32x2 root_codes_random(const Eight& r, int b, uint32_t key, int at) {
    const float inv = inv_scale(b);
    u32x2 o = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const uint32_t h = mix(key + kGolden * static_cast<uint32_t>(at + j)) & 0xFFFFFFu;
        const float x = r[j] * inv;
        const uint32_t below = __float_as_uint(x) & 0xFFF80000u;
        const float lo = __uint_as_float(below), hi = __uint_as_float(below + 0x80000u);
        const bool up = static_cast<float>(h) * 0x1p-24f * ((hi - lo) * (hi + lo)) < (x - lo) * (x + lo);
        const int c = static_cast<int>(below >> 19) - 112 * 16;
        // a root below code 1 becomes that
        o[j / 4] |= (r[j] > 0.0f ? static_cast<uint32_t>(c < 1 ? 1 : c + up) : 0u) << (8 * (j % 4));
    }
    return b == kScaleNaN ? u32x2{0u, 0u} : o;
}

// The hardware's root (1 ulp), which takes no subnormals: those are scaled up first.
__device__ __forceinline__ float root_of(float v) {
    const bool low = v < 0x1p-96f;
    return __builtin_amdgcn_sqrtf(low ? v * 0x1p64f : v) * (low ? 0x1p-32f : 1.0f);
}

// ---------------------------------------------------------------- gradient norm

__device__ __forceinline__ double block_sum(double v, double* s_part) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if (lane_id() == 0) s_part[threadIdx.x / kWave] = v;
    __syncthreads();
    double t = 0.0;
    for (unsigned i = 0; i < blockDim.x / kWave; ++i) t += s_part[i];
    return t;
}

// Waits until the wave's memory operations have been performed.
__device__ __forceinline__ void wait_memory() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

// Eight squares are added in float32 and their sum in float64, unless it leaves
// float32's range: conversions and float64 products of every element would take
// longer than a bf16 gradient's bytes.
__device__ __forceinline__ double squares(const float (&v)[8]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[j] * v[j];
    if (s > 1e-25f && s < 1e38f) return static_cast<double>(s);
    double d = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) d += static_cast<double>(v[j]) * static_cast<double>(v[j]);
    return d;
}

// A workgroup squares the gradients of a run of chunks, 16 bytes a lane and load,
// the next chunk on its way; the last workgroup to finish adds the sums of all in
// their order.  The sums pass between the XCDs' caches as device-scope atomics,
// which are performed in memory: a sum is there before its workgroup counts
// itself, and is read there.
__global__ __launch_bounds__(kThreads) void grad_norm_kernel(Plan plan, int chunks, float* __restrict__ norm) {
    __shared__ double s_part[kThreads / kWave];
    __shared__ bool s_last;
    constexpr int PIECES = kChunk * 4 / (kThreads * 16);          // of a float32 chunk, 16 bytes each; half of them in bf16
    const int G = gridDim.x, t = threadIdx.x;
    const int share = chunks / G, over = chunks - share * G, b0 = blockIdx.x;
    const int lo = b0 * share + min(b0, over), hi = lo + share + (b0 < over ? 1 : 0);
    u32x4 next[PIECES], now[PIECES];
    bool f32 = false;
    auto load = [&](int c) {
        const Chunk& k = plan.chunk()[c];
        f32 = (k.types & 2) != 0;
        const uint8_t* g = static_cast<const uint8_t*>(k.grad);
        const int bytes = k.n * (f32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int at = (i * kThreads + t) * 16;
            next[i] = u32x4{0u, 0u, 0u, 0u};
            if (at + 16 <= bytes) {
                next[i] = *reinterpret_cast<const u32x4*>(g + at);
            } else if (at < bytes) {                              // the last piece of a tensor, by its elements
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at + 2 * j < bytes)
                        next[i][j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(g + at + 2 * j)) << (16 * (j % 2));
            }
        }
    };
    double s = 0.0;
    if (lo < hi) load(lo);
    for (int c = lo; c < hi; ++c) {
        const bool wide = f32;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) now[i] = next[i];
        if (c + 1 < hi) load(c + 1);
#pragma unroll
        for (int i = 0; i < PIECES; i += 2) {
            float v[8];
            if (wide) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(now[i + j / 4][j % 4]);
                s += squares(v);
            } else if (i < PIECES / 2) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = __uint_as_float(j & 1 ? now[i + h][j / 2] & 0xFFFF0000u : now[i + h][j / 2] << 16);
                    s += squares(v);
                }
            }
        }
    }
    const double sum = block_sum(s, s_part);
    if (t == 0) {
        __hip_atomic_store(&plan.head->part[blockIdx.x], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        wait_memory();
        s_last = plan.head->norm_done.last(blockIdx.x, G);
    }
    __syncthreads();
    if (!s_last) return;
    double all = 0.0;
    for (int i = t; i < G; i += kThreads)
        all += __hip_atomic_load(&plan.head->part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    all = block_sum(all, s_part);
    if (t == 0) norm[0] = static_cast<float>(sqrt(all));
}

// ---------------------------------------------------------------- AdamW

struct AdamWArgs {
    Plan plan;
    const float* lr;
    const float* grad_norm;
    int32_t* step;
    double log2_beta1, log2_beta2;                   // -inf for beta 0
    float beta1, beta2, one_less_beta1, one_less_beta2, eps, max_norm;
    uint32_t seed;                                   // of stochastic rounding
    int chunk0, chunks;                              // this launch's first chunk, all launches' chunks
};

struct AdamWScalars {
    float clip, beta1, beta2, one_less_beta1, one_less_beta2, eps, keep, rate, inv_root_bc2;
    // One piece: the moments, the second one's root and the parameter's new value.
    __device__ __forceinline__ void update(const Eight& g, Eight& m, Eight& v, Eight& root, Eight& p) const {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const float x = g[j] * clip;
            m[j] = beta1 * m[j] + one_less_beta1 * x;
            v[j] = beta2 * v[j] + one_less_beta2 * x * x;
            root[j] = root_of(v[j]);
            p[j] = p[j] * keep - rate * m[j] * __builtin_amdgcn_rcpf(root[j] * inv_root_bc2 + eps);
        }
    }
};

// How moments are held: in 32 bits, or in 8, rounded to nearest or at random.
enum State { kFloats, kNearest, kRandom };

// A workgroup a chunk: all its loads are issued before the scalars are looked at.
// With 8-bit moments six waves a SIMD (80 registers; at 81 five: 231 us instead of
// 222 for 75 M elements).
template <State STATE>
__global__ __launch_bounds__(kThreads, STATE == kFloats ? 1 : 6) void adamw_kernel(AdamWArgs b) {
    constexpr bool Q8 = STATE != kFloats;
    const int c = b.chunk0 + static_cast<int>(blockIdx.x);
    const bool there = c < b.chunks;                 // (without any element one workgroup moves the step alone)
    const Chunk& e = b.plan.chunk()[there ? c : 0];
    const int n = there ? e.n : 0;
    const bool f32 = there && (e.types & 1) != 0, g32 = there && (e.types & 2) != 0;
    Eight g[kPieces], p[kPieces], m[kPieces], v[kPieces];
    u32x2 mc[kPieces], vc[kPieces];
    uint32_t mb[kPieces], vb[kPieces];
    if (there) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int at = (i * kThreads + static_cast<int>(threadIdx.x)) * kEach;
            g[i] = load8_as(e.grad, g32, at, n);
            p[i] = e.master ? load8(e.master, at, n) : load8_as(e.param, f32, at, n);
            if (Q8) {
                mc[i] = load8(static_cast<const uint8_t*>(e.m), at, n);
                vc[i] = load8(static_cast<const uint8_t*>(e.v), at, n);
                mb[i] = at < n ? e.m_scales[at / kGroup] : 1;
                vb[i] = at < n ? e.v_scales[at / kGroup] : 1;
            } else {
                m[i] = load8(static_cast<const float*>(e.m), at, n);
                v[i] = load8(static_cast<const float*>(e.v), at, n);
            }
        }
    }
    const float norm = b.grad_norm ? b.grad_norm[0] : 0.0f;
    const float lr = b.lr[0];
    const int t = min(max(__builtin_amdgcn_readfirstlane(b.step[0]), 0), INT32_MAX - 1) + 1;
    // infinite or NaN: nothing is written, the step is not taken
    if ((__float_as_uint(norm) & 0x7F800000u) == 0x7F800000u) return;
    if (there) {
        AdamWScalars s;
        const double bc1 = 1.0 - exp2(t * b.log2_beta1), bc2 = 1.0 - exp2(t * b.log2_beta2);
        s.clip = norm > b.max_norm ? b.max_norm / norm : 1.0f;
        s.beta1 = b.beta1; s.beta2 = b.beta2;
        s.one_less_beta1 = b.one_less_beta1; s.one_less_beta2 = b.one_less_beta2;
        s.eps = b.eps;
        s.keep = 1.0f - lr * e.weight_decay;
        s.rate = static_cast<float>(lr / bc1);
        s.inv_root_bc2 = static_cast<float>(1.0 / sqrt(bc2));
        const uint32_t key = STATE == kRandom ? chunk_key(b.seed, static_cast<uint32_t>(t), static_cast<uint32_t>(c)) : 0u;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int at = (i * kThreads + static_cast<int>(threadIdx.x)) * kEach;
            if (Q8) {
                m[i] = first_values(mc[i], mb[i]);
                v[i] = root_values(vc[i], vb[i]);
#pragma unroll
                for (int j = 0; j < kEach; ++j) v[i][j] *= v[i][j];
            }
            Eight root;
            s.update(g[i], m[i], v[i], root, p[i]);
            if (Q8) {
                // elements past the end are zeros and take no part in the scale
                int bm, br;
                if constexpr (STATE == kRandom) {
                    bm = first_scale_above(group_max(m[i]));
                    br = root_scale_above(group_max(root));
                    store8(static_cast<uint8_t*>(e.m), at, n, first_codes_random(m[i], bm, key, at));
                    store8(static_cast<uint8_t*>(e.v), at, n, root_codes_random(root, br, key, at));
                } else {
                    bm = first_scale(group_max(m[i]));
                    br = root_scale(group_max(root));
                    store8(static_cast<uint8_t*>(e.m), at, n, first_codes(m[i], bm));
                    store8(static_cast<uint8_t*>(e.v), at, n, root_codes(root, br));
                }
                if (at < n && at % kGroup == 0) {
                    e.m_scales[at / kGroup] = static_cast<uint8_t>(bm);
                    e.v_scales[at / kGroup] = static_cast<uint8_t>(br);
                }
            } else {
                store8(static_cast<float*>(e.m), at, n, m[i]);
                store8(static_cast<float*>(e.v), at, n, v[i]);
            }
            if (e.master) store8(e.master, at, n, p[i]);
            if (f32) store8(static_cast<float*>(e.param), at, n, p[i]);
            else store8(static_cast<uint16_t*>(e.param), at, n, p[i]);
        }
    }
    // All waves of a workgroup have read the step when it counts itself; the last
    // one of the last launch moves it.
    if (b.chunk0 + static_cast<int>(gridDim.x) < b.chunks) return;
    __syncthreads();
    if (threadIdx.x == 0 && b.plan.head->step_done.last(blockIdx.x, gridDim.x)) b.step[0] = t;
}

// Workgroup x: elements from x * kThreads * kEach on.
constexpr int kSpan = kThreads * kEach;
__global__ __launch_bounds__(kThreads) void moment_values_kernel(const uint8_t* __restrict__ m, const uint8_t* __restrict__ ms,
                                                                 const uint8_t* __restrict__ v, const uint8_t* __restrict__ vs,
                                                                 int64_t n, uint16_t* __restrict__ mo, uint16_t* __restrict__ ro) {
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSpan;
    const int at = threadIdx.x * kEach, left = static_cast<int>(min(n - base, static_cast<int64_t>(kSpan)));
    if (at >= left) return;
    const u32x2 a = load8(m + base, at, left), c = load8(v + base, at, left);
    const int64_t group = (base + at) / kGroup;
    store8(mo + base, at, left, first_values(a, ms[group]));
    store8(ro + base, at, left, root_values(c, vs[group]));
}

__global__ __launch_bounds__(kThreads) void moment_codes_kernel(const float* __restrict__ m, const float* __restrict__ v,
                                                                int64_t n, uint8_t* __restrict__ mc, uint8_t* __restrict__ ms,
                                                                uint8_t* __restrict__ vc, uint8_t* __restrict__ vs) {
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSpan;
    const int at = threadIdx.x * kEach, left = static_cast<int>(min(n - base, static_cast<int64_t>(kSpan)));
    const Eight a = load8(m + base, at, left);
    Eight r = load8(v + base, at, left);
#pragma unroll
    for (int j = 0; j < kEach; ++j) r[j] = root_of(r[j]);
    const int bm = first_scale(group_max(a)), br = root_scale(group_max(r));
    store8(mc + base, at, left, first_codes(a, bm));
    store8(vc + base, at, left, root_codes(r, br));
    if (at < left && at % kGroup == 0) {
        ms[(base + at) / kGroup] = static_cast<uint8_t>(bm);
        vs[(base + at) / kGroup] = static_cast<uint8_t>(br);
    }
}

// ---------------------------------------------------------------- host side

bool is_type(int32_t t) { return t == MOE_BF16 || t == MOE_F32; }

int check_pointers(std::initializer_list<const void*> ptrs) {
    for (const void* q : ptrs)
        if (!q) return MOE_ERR_INVALID_ARG;
    for (const void* q : ptrs)
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What a list comes to: chunks, tensors that hold something, bits of their moments.
struct ListShape {
    int64_t chunks = 0;
    int entries = 0, state = 32;
    size_t bytes() const { return sizeof(PlanHead) + static_cast<size_t>(std::max<int64_t>(chunks, 1)) * sizeof(Chunk); }
};

int check_list(const moe_adamw_tensor* t, int32_t count, ListShape* s) {
    if (count < 0 || (count > 0 && !t)) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        if (t[i].n < 0) return MOE_ERR_INVALID_ARG;
        if (t[i].n > kMaxElements) return MOE_ERR_UNSUPPORTED;
        if (t[i].n == 0) continue;
        const int state = t[i].m_scales ? 8 : 32;
        if (!t[i].m_scales != !t[i].v_scales || (s->entries > 0 && state != s->state)) return MOE_ERR_INVALID_ARG;
        s->state = state;
        s->chunks += (t[i].n + kChunk - 1) / kChunk;
        ++s->entries;
        if (s->chunks > kMaxChunks) return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

// Whether memory that a step writes belongs to two of its tensors, or holds a
// gradient as well: workgroups would then change each other's elements.
bool shares_memory(const moe_adamw_tensor* tensors, int32_t count) {
    typedef std::pair<uintptr_t, uintptr_t> Range;
    std::vector<Range> written, read;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        const uintptr_t n = static_cast<uintptr_t>(t.n), groups = (n + kGroup - 1) / kGroup, state = t.m_scales ? 1 : 4;
        auto add = [](std::vector<Range>& to, const void* p, uintptr_t bytes) {
            if (p && bytes) to.emplace_back(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes);
        };
        add(written, t.param, n * (t.param_type == MOE_F32 ? 4 : 2));
        add(written, t.master, n * 4);
        add(written, t.m, n * state);
        add(written, t.v, n * state);
        add(written, t.m_scales, groups);
        add(written, t.v_scales, groups);
        add(read, t.grad, n * (t.grad_type == MOE_F32 ? 4 : 2));
    }
    std::sort(written.begin(), written.end());
    for (size_t i = 1; i < written.size(); ++i)
        if (written[i].first < written[i - 1].second) return true;
    for (const Range& r : read) {                    // the first written range that ends behind its beginning
        const auto at = std::upper_bound(written.begin(), written.end(), r.first,
                                         [](uintptr_t a, const Range& w) { return a < w.second; });
        if (at != written.end() && at->first < r.second) return true;
    }
    return false;
}

// The plan that goes with a list.
int check_plan(const moe_adamw_tensor* t, int32_t count, const void* plan, size_t bytes, ListShape* s) {
    const int st = check_list(t, count, s);
    if (st != MOE_OK) return st;
    if (!plan || bytes < s->bytes()) return MOE_ERR_INVALID_ARG;
    return aligned16(plan) ? MOE_OK : MOE_ERR_MISALIGNED;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_adamw_plan_bytes(const moe_adamw_tensor* tensors, int32_t count) {
    moe::ListShape s;
    return moe::check_list(tensors, count, &s) == MOE_OK ? s.bytes() : 0;
}

extern "C" int moe_adamw_plan(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                              hipStream_t stream) {
    using namespace moe;
    ListShape s;
    int st = check_plan(tensors, count, plan, plan_bytes, &s);
    if (st != MOE_OK) return st;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (!is_type(t.param_type) || !is_type(t.grad_type) || t.reserved != 0 || !std::isfinite(t.weight_decay))
            return MOE_ERR_INVALID_ARG;
        if (t.n == 0) continue;
        if ((st = check_pointers({t.param, t.grad, t.m, t.v})) != MOE_OK) return st;
        if (!aligned16(t.master)) return MOE_ERR_MISALIGNED;
    }
    try {
        if (shares_memory(tensors, count)) return MOE_ERR_INVALID_ARG;
    } catch (...) {                                  // no host memory for a list of this length
        return MOE_ERR_UNSUPPORTED;
    }
    const Plan p = Plan{static_cast<PlanHead*>(plan)};
    PlanBatch b{};
    int used = 0;
    int32_t chunk = 0;
    plan_reset_kernel<<<1, 1, 0, stream>>>(p.head);
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n > 0) {
            b.e[used++] = Entry{Chunk{t.param, t.master, t.grad, t.m, t.v, t.m_scales, t.v_scales, 0,
                                      (t.param_type == MOE_F32 ? 1 : 0) | (t.grad_type == MOE_F32 ? 2 : 0), t.weight_decay, 0},
                                t.n, chunk, s.state};
            chunk += static_cast<int32_t>((t.n + kChunk - 1) / kChunk);
        }
        if (used == kBatch || (i == count - 1 && used > 0)) {
            plan_kernel<<<used, kThreads, 0, stream>>>(b, p);
            used = 0;
        }
    }
    return launch_status();
}

extern "C" int moe_grad_norm(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                             float* norm, hipStream_t stream) {
    using namespace moe;
    ListShape s;
    const int st = check_plan(tensors, count, plan, plan_bytes, &s);
    if (st != MOE_OK) return st;
    if (!norm) return MOE_ERR_INVALID_ARG;
    if (!aligned4(norm)) return MOE_ERR_MISALIGNED;
    const int grid = static_cast<int>(std::min<int64_t>(std::max<int64_t>(s.chunks, 1), kNormBlocks));
    grad_norm_kernel<<<grid, kThreads, 0, stream>>>(Plan{static_cast<PlanHead*>(plan)}, static_cast<int>(s.chunks), norm);
    return launch_status();
}

namespace moe {
namespace {

// `random`: 8-bit moments are rounded stochastically, with `seed`.
int adamw_step(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes, const float* lr, double beta1,
               double beta2, double eps, const float* grad_norm, double max_norm, int32_t* step, bool random, uint32_t seed,
               hipStream_t stream) {
    ListShape s;
    const int st = check_plan(tensors, count, plan, plan_bytes, &s);
    if (st != MOE_OK) return st;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
        (grad_norm && !(max_norm > 0.0)))
        return MOE_ERR_INVALID_ARG;
    // v_rcp_f32 takes a subnormal denominator for 0, which eps alone can be (a root is not: 2^-75 at least, or 0)
    if (eps > 0.0 && static_cast<float>(eps) < 0x1p-126f) return MOE_ERR_UNSUPPORTED;
    if (!lr || !step || (random && s.entries > 0 && s.state != 8)) return MOE_ERR_INVALID_ARG;
    if (!aligned4(lr) || !aligned4(step) || !aligned4(grad_norm)) return MOE_ERR_MISALIGNED;
    AdamWArgs a;
    a.plan = Plan{static_cast<PlanHead*>(plan)};
    a.lr = lr; a.grad_norm = grad_norm; a.step = step;
    a.log2_beta1 = std::log2(beta1); a.log2_beta2 = std::log2(beta2);
    a.beta1 = static_cast<float>(beta1); a.beta2 = static_cast<float>(beta2);
    a.one_less_beta1 = static_cast<float>(1.0 - beta1); a.one_less_beta2 = static_cast<float>(1.0 - beta2);
    a.eps = static_cast<float>(eps);
    a.max_norm = grad_norm ? static_cast<float>(max_norm) : 0.0f;
    a.seed = seed;
    a.chunks = static_cast<int>(s.chunks);
    int64_t at = 0;
    do {
        const unsigned grid = static_cast<unsigned>(std::min(std::max<int64_t>(s.chunks - at, 1), kMaxBlocks));
        a.chunk0 = static_cast<int>(at);
        if (s.state != 8) adamw_kernel<kFloats><<<grid, kThreads, 0, stream>>>(a);
        else if (random) adamw_kernel<kRandom><<<grid, kThreads, 0, stream>>>(a);
        else adamw_kernel<kNearest><<<grid, kThreads, 0, stream>>>(a);
        at += grid;
    } while (at < s.chunks);
    return launch_status();
}

}  // namespace
}  // namespace moe

extern "C" int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                              const float* lr, double beta1, double beta2, double eps, const float* grad_norm,
                              double max_norm, int32_t* step, hipStream_t stream) {
    return moe::adamw_step(tensors, count, plan, plan_bytes, lr, beta1, beta2, eps, grad_norm, max_norm, step, false, 0u, stream);
}

extern "C" int moe_adamw_step_stochastic(const moe_adamw_tensor* tensors, int32_t count, void* plan, size_t plan_bytes,
                                         const float* lr, double beta1, double beta2, double eps, const float* grad_norm,
                                         double max_norm, int32_t* step, uint32_t seed, hipStream_t stream) {
    return moe::adamw_step(tensors, count, plan, plan_bytes, lr, beta1, beta2, eps, grad_norm, max_norm, step, true, seed, stream);
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

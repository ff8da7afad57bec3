// Layer norm and RMS norm of the residual stream, with the addition in front,
// and their backward.
//
//   h = T(x + r);  mean = sum h / D;  rstd = 1/sqrt(sum (h - mean)^2 / D + eps)
//   y = (h - mean) rstd w + b
//   dx = rstd (g - mean_D(g) - xhat mean_D(g xhat)) + dtotal,  g = dy w
//   dw = sum_rows dy xhat,  db = sum_rows dy
//
// Both are HBM-bound passes: a row is read once, kept in registers as float32
// through its sums, and written once.  TL lanes share a row, V pieces of 8
// columns each, so a lane holds at most 32 columns, and the weights of its
// columns stay in registers from row to row.  Rows need not begin on a 16-byte
// boundary (D is any number): pieces are loaded whole at any alignment, the
// last one of a row by elements.
#include <algorithm>
#include <initializer_list>

#include "gemm_common.h"
#include "../../include/moe_block.h"

namespace moe {
namespace {

constexpr int kPiece = 8;            // columns a lane holds together
constexpr int kNormThreads = 256;

struct Bf16 { uint16_t bits; };

__device__ __forceinline__ float widen(Bf16 v) { return bf16_to_f32(v.bits); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void narrow(float f, Bf16* o) { o->bits = f32_to_bf16(f); }
__device__ __forceinline__ void narrow(float f, float* o) { *o = f; }

// Eight columns as they are in memory.
template <class T>
struct Piece;
template <>
struct Piece<Bf16> {
    u32x4 w;
    __device__ __forceinline__ float operator[](int j) const {
        return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
    __device__ __forceinline__ void set(int j, Bf16 v) {
        w[j / 2] = j & 1 ? (w[j / 2] & 0xFFFFu) | static_cast<uint32_t>(v.bits) << 16 : (w[j / 2] & 0xFFFF0000u) | v.bits;
    }
    __device__ __forceinline__ void from(const float (&v)[kPiece]) {
#pragma unroll
        for (int j = 0; j < kPiece; j += 2) w[j / 2] = pack_bf16x2(v[j], v[j + 1]);
    }
};
template <>
struct Piece<float> {
    float w[kPiece];
    __device__ __forceinline__ float operator[](int j) const { return w[j]; }
    __device__ __forceinline__ void set(int j, float v) { w[j] = v; }
    __device__ __forceinline__ void from(const float (&v)[kPiece]) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) w[j] = v[j];
    }
};

// A lane's piece of a row: columns c .. c+7.  The last piece of a row whose D is
// no multiple of 8 begins early, so that it can be loaded whole: its first
// `skip` columns are another lane's, count as 0 and are not stored.  A lane
// without a piece skips all 8.
struct Place {
    int c, skip;
    __device__ __forceinline__ Place(int piece, int D) {
        c = max(min(piece * kPiece, D - kPiece), 0);
        skip = min(piece * kPiece - c, kPiece);
    }
};

// FEW: rows of under 8 columns, by elements.
template <bool FEW, class T>
__device__ __forceinline__ Piece<T> load8(const T* row, Place at, int D) {
    Piece<T> p{};
    if (FEW) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (at.skip == 0 && j < D) p.set(j, row[j]);
        return p;
    }
    __builtin_memcpy(&p.w, row + at.c, kPiece * sizeof(T));
    return p;
}
template <bool FEW, class T>
__device__ __forceinline__ void store8(T* row, Place at, int D, const float (&v)[kPiece]) {
    if (!FEW && at.skip == 0) {
        Piece<T> p;
        p.from(v);
        __builtin_memcpy(row + at.c, &p.w, kPiece * sizeof(T));
    } else if (at.skip < kPiece) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (j >= at.skip && (!FEW || j < D)) narrow(v[j], &row[at.c + j]);
    }
}
// Another lane's columns become 0 (and those past the end of few).
template <bool FEW>
__device__ __forceinline__ void clear_skipped(float (&v)[kPiece], Place at, int D) {
    if (FEW || at.skip > 0) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (j < at.skip || (FEW && j >= D)) v[j] = 0.0f;
    }
}

// Sums over the TL lanes that share a row, the same in each of them.
// `scratch`: 2 * TL / 64 floats of the row's own in LDS, used in turn.
template <int TL>
__device__ __forceinline__ float row_total(float v, float* scratch, int turn) {
#pragma unroll
    for (int o = (TL < kWave ? TL : kWave) / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    if (TL <= kWave) return v;
    constexpr int WAVES = TL / kWave > 0 ? TL / kWave : 1;
    float* s = scratch + (turn & 1) * WAVES;
    if (lane_id() == 0) s[threadIdx.x % TL / kWave] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) t += s[i];
    return t;
}

struct NormArgs {
    const void *x, *residual, *dy, *dtotal;
    const float *weight, *bias;
    void *total, *y, *dx;
    float *mean, *rstd, *part;
    int64_t rows;
    int D, centre;
    float eps;
};

template <class TX, class TY, int TL, int V, bool FEW>
__global__ __launch_bounds__(TL > kNormThreads ? TL : kNormThreads) void norm_fwd_kernel(NormArgs p) {
    constexpr int THREADS = TL > kNormThreads ? TL : kNormThreads;
    constexpr int ROWS = THREADS / TL;                   // rows of a workgroup at once
    static_assert(TL <= kWave || ROWS == 1, "a workgroup's barriers are one row's");
    __shared__ float s_sum[2 * (TL / kWave > 0 ? TL / kWave : 1)];
    const int t = threadIdx.x % TL, D = p.D;
    const float inv = 1.0f / static_cast<float>(D);
    float w[V][kPiece], b[V][kPiece];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const Place at(i * TL + t, D);
        const Piece<float> pw = load8<FEW>(p.weight, at, D);
        Piece<float> pb{};
        if (p.bias) pb = load8<FEW>(p.bias, at, D);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) w[i][j] = pw[j], b[i][j] = pb[j];
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    int turn = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TL; r < p.rows; r += step) {
        const TX* x = static_cast<const TX*>(p.x) + r * D;
        float h[V][kPiece];
        Piece<TX> in[V], add[V];
#pragma unroll
        for (int i = 0; i < V; ++i) in[i] = load8<FEW>(x, Place(i * TL + t, D), D);
        if (p.residual) {
            const TX* res = static_cast<const TX*>(p.residual) + r * D;
#pragma unroll
            for (int i = 0; i < V; ++i) add[i] = load8<FEW>(res, Place(i * TL + t, D), D);
            // (a lane's columns that are another's may be overwritten from here on: they are cleared)
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {       // what is stored is what is normalised
                    TX o;
                    narrow(in[i][j] + add[i][j], &o);
                    h[i][j] = widen(o);
                }
                store8<FEW>(static_cast<TX*>(p.total) + r * D, Place(i * TL + t, D), D, h[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) h[i][j] = in[i][j];
        }
        float mean = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) clear_skipped<FEW>(h[i], Place(i * TL + t, D), D);
        if (p.centre) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) s += h[i][j];
            mean = row_total<TL>(s, s_sum, turn++) * inv;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < kPiece; ++j) h[i][j] -= mean;
                clear_skipped<FEW>(h[i], Place(i * TL + t, D), D);
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) s += h[i][j] * h[i][j];
        const float rstd = 1.0f / __builtin_sqrtf(row_total<TL>(s, s_sum, turn++) * inv + p.eps);
        TY* y = static_cast<TY*>(p.y) + r * D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) h[i][j] = h[i][j] * rstd * w[i][j] + b[i][j];
            store8<FEW>(y, Place(i * TL + t, D), D, h[i]);
        }
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

// The backward: dx of each row, and each workgroup's sums of the weights'
// gradients over its rows, in `part` [2][G][D].  The next row is on its way
// while one is worked on and the weights stay in registers, where there are
// enough of them (not with 16 waves a workgroup).
constexpr int kBwdThreads = 512;

template <class TX, class TY, int TL, int V, bool FEW>
__global__ __launch_bounds__(TL > kBwdThreads ? TL : kBwdThreads) void norm_bwd_kernel(NormArgs p) {
    constexpr int ROWS = TL > kBwdThreads ? 1 : kBwdThreads / TL;
    constexpr bool AHEAD = TL <= kBwdThreads;
    __shared__ float s_sum[ROWS][2 * (TL / kWave > 0 ? TL / kWave : 1)];
    __shared__ float s_part[ROWS > 1 ? ROWS - 1 : 1][ROWS > 1 ? V * TL * kPiece : 1];
    const int t = threadIdx.x % TL, team = threadIdx.x / TL, D = p.D;
    const float inv = 1.0f / static_cast<float>(D);
    float w[V][kPiece], dw[V][kPiece], db[V][kPiece];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const Piece<float> pw = load8<FEW>(p.weight, Place(i * TL + t, D), D);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) w[i][j] = AHEAD ? pw[j] : 0.0f, dw[i][j] = db[i][j] = 0.0f;
    }
    struct Row {
        Piece<TX> h[V];
        Piece<TY> dy[V];
        float mean, rstd;
    };
    auto load = [&](int64_t r) {
        Row o{};
        if (r >= p.rows) return o;                       // a team without a row keeps the others' barriers company
#pragma unroll
        for (int i = 0; i < V; ++i) {
            o.h[i] = load8<FEW>(static_cast<const TX*>(p.x) + r * D, Place(i * TL + t, D), D);
            o.dy[i] = load8<FEW>(static_cast<const TY*>(p.dy) + r * D, Place(i * TL + t, D), D);
        }
        o.mean = p.centre ? p.mean[r] : 0.0f;
        o.rstd = p.rstd[r];
        return o;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    int turn = 0;
    Row next{};
    if (AHEAD) next = load(static_cast<int64_t>(blockIdx.x) * ROWS + team);
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * ROWS; r0 < p.rows; r0 += step) {
        const int64_t r = r0 + team;
        const Row now = AHEAD ? next : load(r);
        if (AHEAD && r0 + step < p.rows) next = load(r + step);
        float c1 = 0.0f, c2 = 0.0f, xh[V][kPiece], g[V][kPiece];
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) xh[i][j] = (now.h[i][j] - now.mean) * now.rstd, g[i][j] = now.dy[i][j];
            clear_skipped<FEW>(xh[i], Place(i * TL + t, D), D);
            clear_skipped<FEW>(g[i], Place(i * TL + t, D), D);
            Piece<float> pw{};
            if (!AHEAD) pw = load8<FEW>(p.weight, Place(i * TL + t, D), D);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                dw[i][j] += g[i][j] * xh[i][j];
                db[i][j] += g[i][j];
                g[i][j] *= AHEAD ? w[i][j] : pw[j];
                c1 += g[i][j] * xh[i][j];
                c2 += g[i][j];
            }
        }
        c1 = row_total<TL>(c1, s_sum[team], turn++) * inv;
        c2 = p.centre ? row_total<TL>(c2, s_sum[team], turn++) * inv : 0.0f;
        if (r >= p.rows) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Place at(i * TL + t, D);
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) o[j] = (g[i][j] - c2 - xh[i][j] * c1) * now.rstd;
            if (p.dtotal) {
                const Piece<TX> a = load8<FEW>(static_cast<const TX*>(p.dtotal) + r * D, at, D);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) o[j] += a[j];
            }
            store8<FEW>(static_cast<TX*>(p.dx) + r * D, at, D, o);
        }
    }
    // the teams of the workgroup add theirs in order
#pragma unroll 1
    for (int half = 0; half < (p.bias ? 2 : 1); ++half) {
        __syncthreads();
        if (team > 0) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    s_part[ROWS > 1 ? team - 1 : 0][ROWS > 1 ? (i * kPiece + j) * TL + t : 0] = half ? db[i][j] : dw[i][j];
        }
        __syncthreads();
        if (team == 0) {
            float* part = p.part + (static_cast<int64_t>(half) * gridDim.x + blockIdx.x) * D;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float o[kPiece];
#pragma unroll
                for (int j = 0; j < kPiece; ++j) o[j] = half ? db[i][j] : dw[i][j];
#pragma unroll 1
                for (int k = 0; k < ROWS - 1; ++k)
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) o[j] += s_part[k][ROWS > 1 ? (i * kPiece + j) * TL + t : 0];
                store8<FEW>(part, Place(i * TL + t, D), D, o);
            }
        }
    }
}

// dweight and dbias: the workgroups' sums, in order.  Workgroup (x, y): 64
// columns of gradient y, 16 lanes with 4 each; its 64 groups of lanes take the
// sums in turn, and theirs are added in order.
constexpr int kFinishThreads = 1024, kFinishGroups = kFinishThreads / 16;
__global__ __launch_bounds__(kFinishThreads) void norm_finish_kernel(const float* __restrict__ part, int G, int D,
                                                                     int accumulate, float* __restrict__ dweight,
                                                                     float* __restrict__ dbias) {
    __shared__ float s_part[kFinishGroups][kWave];
    const int q = threadIdx.x % 16, group = threadIdx.x / 16, c = blockIdx.x * kWave + q * 4;
    const float* mine = part + static_cast<int64_t>(blockIdx.y) * G * D;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int g = group; g < G; g += kFinishGroups) {
        const float* at = mine + static_cast<int64_t>(g) * D;
        if (c + 4 <= D) {
            float v[4];
            __builtin_memcpy(v, at + c, sizeof(v));
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < D) s[j] += at[c + j];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s_part[group][q * 4 + j] = s[j];
    __syncthreads();
    // eight waves add eight groups each, then the first one the eight
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    float v = 0.0f;
    if (wave < 8) {
#pragma unroll
        for (int i = 0; i < kFinishGroups / 8; ++i) v += s_part[wave * (kFinishGroups / 8) + i][lane];
    }
    __syncthreads();
    if (wave < 8) s_part[wave][lane] = v;
    __syncthreads();
    const int col = blockIdx.x * kWave + lane;
    if (wave == 0 && col < D) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s_part[i][lane];
        float* out = blockIdx.y ? dbias : dweight;
        out[col] = accumulate ? out[col] + t : t;
    }
}

constexpr int kMaxNormDim = 16384;

template <class TX, class TY, int TL, int V, bool FEW = false>
void launch_fwd(const NormArgs& a, hipStream_t s) {
    constexpr int THREADS = std::max(TL, kNormThreads), ROWS = THREADS / TL;
    const int64_t blocks = std::min<int64_t>((a.rows + ROWS - 1) / ROWS, 2048);
    norm_fwd_kernel<TX, TY, TL, V, FEW><<<static_cast<unsigned>(blocks), THREADS, 0, s>>>(a);
}

// Lanes a row and pieces a lane for D columns.  The backward's sums take twice
// the registers: at most two pieces a lane.
constexpr int bwd_lanes(int pieces) {
    return pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 128 ? 64 : pieces <= 256 ? 128
           : pieces <= 512 ? 256 : pieces <= 1024 ? 512 : 1024;
}
template <class TX, class TY>
void by_width_fwd(const NormArgs& a, hipStream_t s) {
    const int pieces = (a.D + kPiece - 1) / kPiece;
    if (a.D < kPiece) launch_fwd<TX, TY, 8, 1, true>(a, s);
    else if (pieces <= 8) launch_fwd<TX, TY, 8, 1>(a, s);
    else if (pieces <= 16) launch_fwd<TX, TY, 16, 1>(a, s);
    else if (pieces <= 32) launch_fwd<TX, TY, 32, 1>(a, s);
    else if (pieces <= 64) launch_fwd<TX, TY, 64, 1>(a, s);
    else if (pieces <= 128) launch_fwd<TX, TY, 64, 2>(a, s);
    else if (pieces <= 256) launch_fwd<TX, TY, 64, 4>(a, s);
    else if (pieces <= 512) launch_fwd<TX, TY, 256, 2>(a, s);
    else if (pieces <= 1024) launch_fwd<TX, TY, 256, 4>(a, s);
    else launch_fwd<TX, TY, 512, 4>(a, s);
}
template <class TX, class TY>
void by_width_bwd(const NormArgs& a, int G, hipStream_t s) {
    const int pieces = (a.D + kPiece - 1) / kPiece;
    switch (bwd_lanes(pieces)) {
        case 8:
            if (a.D < kPiece) norm_bwd_kernel<TX, TY, 8, 1, true><<<G, kBwdThreads, 0, s>>>(a);
            else norm_bwd_kernel<TX, TY, 8, 1, false><<<G, kBwdThreads, 0, s>>>(a);
            return;
        case 16: norm_bwd_kernel<TX, TY, 16, 1, false><<<G, kBwdThreads, 0, s>>>(a); return;
        case 32: norm_bwd_kernel<TX, TY, 32, 1, false><<<G, kBwdThreads, 0, s>>>(a); return;
        case 64:
            if (pieces <= 64) norm_bwd_kernel<TX, TY, 64, 1, false><<<G, kBwdThreads, 0, s>>>(a);
            else norm_bwd_kernel<TX, TY, 64, 2, false><<<G, kBwdThreads, 0, s>>>(a);
            return;
        case 128: norm_bwd_kernel<TX, TY, 128, 2, false><<<G, kBwdThreads, 0, s>>>(a); return;
        case 256: norm_bwd_kernel<TX, TY, 256, 2, false><<<G, kBwdThreads, 0, s>>>(a); return;
        case 512: norm_bwd_kernel<TX, TY, 512, 2, false><<<G, kBwdThreads, 0, s>>>(a); return;
        default: norm_bwd_kernel<TX, TY, 1024, 2, false><<<G, 1024, 0, s>>>(a);
    }
}

// Workgroups of the backward: one a compute unit, since their sums, 8 * D bytes
// each, are written and read once more, and no more than have a row.
int bwd_groups(int64_t rows, int D) {
    const int teams = std::max(1, kBwdThreads / bwd_lanes((D + kPiece - 1) / kPiece));
    return static_cast<int>(std::min<int64_t>(std::max<int64_t>((rows + teams - 1) / teams, 1), 256));
}

int check_norm(int64_t rows, int32_t D, int32_t x_type, int32_t y_type) {
    if (rows < 0 || D < 1 || (x_type != MOE_BF16 && x_type != MOE_F32) || (y_type != MOE_BF16 && y_type != MOE_F32))
        return MOE_ERR_INVALID_ARG;
    if (D > kMaxNormDim || rows > (static_cast<int64_t>(1) << 40) / D || (x_type == MOE_BF16 && y_type == MOE_F32))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Null pointers that must be there, then the alignment of all that are.
int check_given(std::initializer_list<const void*> needed, std::initializer_list<const void*> optional) {
    for (const void* q : needed)
        if (!q) return MOE_ERR_INVALID_ARG;
    for (const void* q : needed)
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    for (const void* q : optional)
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias,
                                  int64_t rows, int32_t D, double eps, int32_t x_type, int32_t y_type,
                                  void* total, void* y, float* mean, float* rstd, hipStream_t stream) {
    using namespace moe;
    int st = check_norm(rows, D, x_type, y_type);
    if (st != MOE_OK) return st;
    if (!(eps >= 0.0) || !(eps <= 1.0) || !residual != !total) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    st = check_given({x, weight, y, rstd}, {residual, bias, total, mean});
    if (st != MOE_OK) return st;
    // a row's total is stored before its y: one of them would be lost
    if (y == total) return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.total = total; a.y = y;
    a.mean = mean; a.rstd = rstd; a.rows = rows; a.D = D; a.centre = mean != nullptr;
    a.eps = static_cast<float>(eps);
    if (x_type == MOE_BF16) by_width_fwd<Bf16, Bf16>(a, stream);
    else if (y_type == MOE_BF16) by_width_fwd<float, Bf16>(a, stream);
    else by_width_fwd<float, float>(a, stream);
    return launch_status();
}

extern "C" size_t moe_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t D) {
    if (moe::check_norm(rows, D, MOE_F32, MOE_F32) != MOE_OK) return 0;
    return static_cast<size_t>(moe::bwd_groups(rows, D)) * D * 2 * sizeof(float);
}

extern "C" int moe_layer_norm_bwd(const void* dy, const void* h, const float* weight, const float* mean,
                                  const float* rstd, const void* dtotal, int64_t rows, int32_t D,
                                  int32_t x_type, int32_t y_type, int32_t accumulate, void* dx, float* dweight,
                                  float* dbias, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace moe;
    int st = check_norm(rows, D, x_type, y_type);
    if (st != MOE_OK) return st;
    if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
    st = rows ? check_given({dy, h, weight, rstd, dx, dweight, workspace}, {mean, dtotal, dbias})
              : check_given({dweight, workspace}, {dbias});
    if (st != MOE_OK) return st;
    const int G = bwd_groups(rows, D);
    if (workspace_bytes < moe_layer_norm_bwd_workspace_bytes(rows, D)) return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = h; a.dy = dy; a.dtotal = dtotal; a.weight = weight; a.bias = dbias; a.dx = dx;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.part = static_cast<float*>(workspace); a.rows = rows; a.D = D; a.centre = mean != nullptr;
    if (rows) {
        if (x_type == MOE_BF16) by_width_bwd<Bf16, Bf16>(a, G, stream);
        else if (y_type == MOE_BF16) by_width_bwd<float, Bf16>(a, G, stream);
        else by_width_bwd<float, float>(a, G, stream);
    }
    norm_finish_kernel<<<dim3((D + kWave - 1) / kWave, dbias ? 2 : 1), kFinishThreads, 0, stream>>>(
        a.part, rows ? G : 0, D, accumulate, dweight, dbias);
    return launch_status();
}

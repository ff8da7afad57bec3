// Layer norm and RMS norm of the residual stream, with the addition in front,
// and their backward.
//
//   h = T(x + r);  mean = sum h / D;  rstd = 1/sqrt(sum (h - mean)^2 / D + eps)
//   y = (h - mean) rstd w + b
//   dx = rstd (g - mean_D(g) - xhat mean_D(g xhat)) + dtotal,  g = dy w
//   dw = sum_rows dy xhat,  db = sum_rows dy
//
// Both are HBM-bound passes: a row is read once, kept in registers as float32
// through its sums, and written once.  WPR waves share a row, V pieces of 8
// columns a lane, so a lane holds at most 32 columns and the weights of its
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

// Columns c .. c+7 of a row of D as float32; columns past the end are 0.
template <class T>
__device__ __forceinline__ void load8(const T* row, int c, int D, float (&v)[kPiece]) {
    if (c + kPiece <= D) {
        T t[kPiece];
        __builtin_memcpy(t, row + c, sizeof(t));
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = widen(t[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = c + j < D ? widen(row[c + j]) : 0.0f;
    }
}
template <class T>
__device__ __forceinline__ void store8(T* row, int c, int D, const float (&v)[kPiece]) {
    if (c + kPiece <= D) {
        T t[kPiece];
#pragma unroll
        for (int j = 0; j < kPiece; ++j) narrow(v[j], &t[j]);
        __builtin_memcpy(row + c, t, sizeof(t));
    } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (c + j < D) narrow(v[j], &row[c + j]);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sums over the WPR waves that share a row, the same in every lane.
// `scratch`: 2 * WPR floats of the row's own in LDS, used in turn.
template <int WPR>
__device__ __forceinline__ float row_total(float v, float* scratch, int wave, int turn) {
    v = wave_sum(v);
    if (WPR == 1) return v;
    float* s = scratch + (turn & 1) * WPR;
    if (lane_id() == 0) s[wave] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) t += s[i];
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

template <class TX, class TY, int WPR, int V>
__global__ __launch_bounds__(WPR * kWave > kNormThreads ? WPR * kWave : kNormThreads)
void norm_fwd_kernel(NormArgs p) {
    constexpr int THREADS = WPR * kWave > kNormThreads ? WPR * kWave : kNormThreads;
    constexpr int ROWS = THREADS / (WPR * kWave);        // rows of a workgroup at once
    static_assert(WPR == 1 || ROWS == 1, "a workgroup's barriers are one row's");
    __shared__ float s_sum[2 * WPR];
    const int t = threadIdx.x % (WPR * kWave), wave = t / kWave;
    const float inv = 1.0f / static_cast<float>(p.D);
    float w[V][kPiece], b[V][kPiece];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (i * WPR * kWave + t) * kPiece;
        load8(p.weight, c, p.D, w[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) b[i][j] = 0.0f;
        if (p.bias) load8(p.bias, c, p.D, b[i]);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    int turn = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / (WPR * kWave); r < p.rows; r += step) {
        const TX* x = static_cast<const TX*>(p.x) + r * p.D;
        float h[V][kPiece];
#pragma unroll
        for (int i = 0; i < V; ++i) load8(x, (i * WPR * kWave + t) * kPiece, p.D, h[i]);
        if (p.residual) {
            const TX* res = static_cast<const TX*>(p.residual) + r * p.D;
            TX* total = static_cast<TX*>(p.total) + r * p.D;
            float a[V][kPiece];
#pragma unroll
            for (int i = 0; i < V; ++i) load8(res, (i * WPR * kWave + t) * kPiece, p.D, a[i]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {       // what is stored is what is normalised
                    TX o;
                    narrow(h[i][j] + a[i][j], &o);
                    h[i][j] = widen(o);
                }
                store8(total, (i * WPR * kWave + t) * kPiece, p.D, h[i]);
            }
        }
        float mean = 0.0f;
        if (p.centre) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) s += h[i][j];
            mean = row_total<WPR>(s, s_sum, wave, turn++) * inv;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j)
                    h[i][j] = (i * WPR * kWave + t) * kPiece + j < p.D ? h[i][j] - mean : 0.0f;
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) s += h[i][j] * h[i][j];
        const float rstd = 1.0f / __builtin_sqrtf(row_total<WPR>(s, s_sum, wave, turn++) * inv + p.eps);
        TY* y = static_cast<TY*>(p.y) + r * p.D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) h[i][j] = h[i][j] * rstd * w[i][j] + b[i][j];
            store8(y, (i * WPR * kWave + t) * kPiece, p.D, h[i]);
        }
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

// The backward: dx of each row, and each workgroup's sums of the weights'
// gradients over its rows, in `part` [2][G][D] (db's half only with a mean or
// a bias: `both`).
template <class TX, class TY, int WPR, int V>
__global__ __launch_bounds__(WPR * kWave > kNormThreads ? WPR * kWave : kNormThreads)
void norm_bwd_kernel(NormArgs p) {
    constexpr int THREADS = WPR * kWave > kNormThreads ? WPR * kWave : kNormThreads;
    constexpr int ROWS = THREADS / (WPR * kWave);
    static_assert(WPR == 1 || ROWS == 1, "a workgroup's barriers are one row's");
    __shared__ float s_sum[2 * WPR];
    __shared__ float s_part[ROWS > 1 ? ROWS - 1 : 1][ROWS > 1 ? V * kWave * kPiece : 1];
    const int t = threadIdx.x % (WPR * kWave), wave = t / kWave, team = threadIdx.x / (WPR * kWave);
    const float inv = 1.0f / static_cast<float>(p.D);
    float w[V][kPiece], dw[V][kPiece], db[V][kPiece];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load8(p.weight, (i * WPR * kWave + t) * kPiece, p.D, w[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) dw[i][j] = db[i][j] = 0.0f;
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    int turn = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + team; r < p.rows; r += step) {
        const TX* h = static_cast<const TX*>(p.x) + r * p.D;
        const TY* dy = static_cast<const TY*>(p.dy) + r * p.D;
        float xh[V][kPiece], g[V][kPiece];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            load8(h, (i * WPR * kWave + t) * kPiece, p.D, xh[i]);
            load8(dy, (i * WPR * kWave + t) * kPiece, p.D, g[i]);
        }
        const float mean = p.centre ? p.mean[r] : 0.0f, rstd = p.rstd[r];
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {           // columns past the end: dy = 0
                xh[i][j] = (xh[i][j] - mean) * rstd;
                dw[i][j] += g[i][j] * xh[i][j];
                db[i][j] += g[i][j];
                g[i][j] *= w[i][j];
                c1 += g[i][j] * xh[i][j];
                c2 += g[i][j];
            }
        c1 = row_total<WPR>(c1, s_sum, wave, turn++) * inv;
        c2 = p.centre ? row_total<WPR>(c2, s_sum, wave, turn++) * inv : 0.0f;
        TX* dx = static_cast<TX*>(p.dx) + r * p.D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * WPR * kWave + t) * kPiece;
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) o[j] = (g[i][j] - c2 - xh[i][j] * c1) * rstd;
            if (p.dtotal) {
                float a[kPiece];
                load8(static_cast<const TX*>(p.dtotal) + r * p.D, c, p.D, a);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) o[j] += a[j];
            }
            store8(dx, c, p.D, o);
        }
    }
    // the teams of the workgroup add theirs in order
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        if (half == 1 && !p.bias) break;
        if (ROWS > 1) {
            __syncthreads();
            if (team > 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < kPiece; ++j)
                        s_part[ROWS > 1 ? team - 1 : 0][ROWS > 1 ? (i * kPiece + j) * kWave + t : 0] = half ? db[i][j] : dw[i][j];
            }
            __syncthreads();
        }
        if (team == 0) {
            float* part = p.part + (static_cast<int64_t>(half) * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float o[kPiece];
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {
                    o[j] = half ? db[i][j] : dw[i][j];
                    if (ROWS > 1)
                        for (int k = 0; k < ROWS - 1; ++k) o[j] += s_part[k][ROWS > 1 ? (i * kPiece + j) * kWave + t : 0];
                }
                store8(part, (i * WPR * kWave + t) * kPiece, p.D, o);
            }
        }
    }
}

// dweight and dbias: the workgroups' sums, in order.  Workgroup (x, y): 64
// columns of gradient y; its waves take the sums in turn and add theirs in order.
constexpr int kFinishWaves = 8;
__global__ __launch_bounds__(kFinishWaves * kWave) void norm_finish_kernel(const float* __restrict__ part, int G, int D,
                                                                           int accumulate, float* __restrict__ dweight,
                                                                           float* __restrict__ dbias) {
    __shared__ float s_part[kFinishWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int c = blockIdx.x * kWave + lane;
    const float* mine = part + static_cast<int64_t>(blockIdx.y) * G * D;
    float s = 0.0f;
    if (c < D)
        for (int g = wave; g < G; g += kFinishWaves) s += mine[static_cast<int64_t>(g) * D + c];
    s_part[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < D) {
        for (int i = 1; i < kFinishWaves; ++i) s += s_part[i][lane];
        float* out = blockIdx.y ? dbias : dweight;
        out[c] = accumulate ? out[c] + s : s;
    }
}

constexpr int kMaxNormDim = 16384;

// Workgroups of the backward: their sums are 8 * D bytes each, written and read
// once, so no more than two for a compute unit.
int bwd_groups(int64_t rows) {
    return static_cast<int>(std::min<int64_t>(std::max<int64_t>((rows + 3) / 4, 1), 512));
}

// Pieces a lane and waves a row for D columns.
template <template <class, class, int, int> class L, class TX, class TY>
void by_width(const NormArgs& a, int groups, hipStream_t s) {
    const int pieces = (a.D + kPiece - 1) / kPiece;
    if (pieces <= kWave) L<TX, TY, 1, 1>::go(a, groups, s);
    else if (pieces <= 2 * kWave) L<TX, TY, 1, 2>::go(a, groups, s);
    else if (pieces <= 4 * kWave) L<TX, TY, 1, 4>::go(a, groups, s);
    else if (pieces <= 8 * kWave) L<TX, TY, 4, 2>::go(a, groups, s);
    else if (pieces <= 16 * kWave) L<TX, TY, 4, 4>::go(a, groups, s);
    else L<TX, TY, 8, 4>::go(a, groups, s);
}
template <class TX, class TY, int WPR, int V>
struct Fwd {
    static void go(const NormArgs& a, int, hipStream_t s) {
        constexpr int THREADS = std::max(WPR * kWave, kNormThreads), ROWS = THREADS / (WPR * kWave);
        const int64_t blocks = std::min<int64_t>((a.rows + ROWS - 1) / ROWS, 2048);
        norm_fwd_kernel<TX, TY, WPR, V><<<static_cast<unsigned>(blocks), THREADS, 0, s>>>(a);
    }
};
template <class TX, class TY, int WPR, int V>
struct Bwd {
    static void go(const NormArgs& a, int groups, hipStream_t s) {
        norm_bwd_kernel<TX, TY, WPR, V><<<groups, std::max(WPR * kWave, kNormThreads), 0, s>>>(a);
    }
};
template <template <class, class, int, int> class L>
void by_type(const NormArgs& a, int x_type, int y_type, int groups, hipStream_t s) {
    if (x_type == MOE_BF16) by_width<L, Bf16, Bf16>(a, groups, s);
    else if (y_type == MOE_BF16) by_width<L, float, Bf16>(a, groups, s);
    else by_width<L, float, float>(a, groups, s);
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
    by_type<Fwd>(a, x_type, y_type, 0, stream);
    return launch_status();
}

extern "C" size_t moe_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t D) {
    if (moe::check_norm(rows, D, MOE_F32, MOE_F32) != MOE_OK) return 0;
    return static_cast<size_t>(moe::bwd_groups(rows)) * D * 2 * sizeof(float);
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
    const int G = bwd_groups(rows);
    if (workspace_bytes < moe_layer_norm_bwd_workspace_bytes(rows, D)) return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = h; a.dy = dy; a.dtotal = dtotal; a.weight = weight; a.bias = dbias; a.dx = dx;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.part = static_cast<float*>(workspace); a.rows = rows; a.D = D; a.centre = mean != nullptr;
    if (rows) by_type<Bwd>(a, x_type, y_type, G, stream);
    norm_finish_kernel<<<dim3((D + kWave - 1) / kWave, dbias ? 2 : 1), kFinishWaves * kWave, 0, stream>>>(
        a.part, rows ? G : 0, D, accumulate, dweight, dbias);
    return launch_status();
}

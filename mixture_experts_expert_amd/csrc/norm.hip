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
// columns stay in registers from row to row.  Loads and stores are of 16 aligned
// bytes whatever D is, but for a row's first and last columns; not aligned are those
// of D 16377 to 16383, and, at widths above 1016 that are no multiple of 8, of a few
// rows' backward by one workgroup after its first rows.
//
// TL and V are the fewest lanes, then pieces, that a row fits: idle ones take issue
// slots (three pieces a lane instead of four where they do: bf16 rows of 8200
// columns 54 us instead of 66, of 1111 67 for 80), and past 64 lanes a row's sums
// meet over barriers.
// Measured with 2^25 elements, read and written (a copy here reaches 4.9 to 5.4
// TB/s): forward with the addition 4.6 to 5.2 TB/s in bf16, 4.4 to 5.0 in float32,
// backward with dtotal 4.0 to 5.0 and 4.1 to 5.3; rows of an odd number of bf16
// 3.1 to 4.2 and 2.4 to 3.7, where the wave of a row's first and last columns takes
// the time (1111 columns 110 us against 61 for 1112).  8 rows of 2048 take 3.8 us.
#include <algorithm>
#include <initializer_list>

#include "gemm_common.h"
#include "span.h"
#include "../../include/moe_block.h"

namespace moe {
namespace {

constexpr int kPiece = 8;            // columns a lane holds together
constexpr int kNormThreads = 256;

typedef float floatx4 __attribute__((ext_vector_type(4)));

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
    // The columns before lo and from hi on become 0.
    __device__ __forceinline__ void keep(int lo, int hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] &= (2 * i >= lo && 2 * i < hi ? 0xFFFFu : 0u) | (2 * i + 1 >= lo && 2 * i + 1 < hi ? 0xFFFF0000u : 0u);
    }
    // What was made of it is not known to be the same when it is made again.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("" : "+v"(w[i]));
    }
    // Column j + n comes to place j (n < 8), anything to the last n.
    __device__ __forceinline__ void move_down(int n) {
        if (n & 4) w[0] = w[2], w[1] = w[3];
        if (n & 2) w[0] = w[1], w[1] = w[2], w[2] = w[3];
        if (n & 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = w[i] >> 16 | (i < 3 ? w[i + 1] << 16 : 0u);
        }
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
    __device__ __forceinline__ void keep(int lo, int hi) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) w[j] = j >= lo && j < hi ? w[j] : 0.0f;
    }
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) asm("" : "+v"(w[j]));
    }
    __device__ __forceinline__ void move_down(int n) {
#pragma unroll
        for (int s = 4; s >= 1; s /= 2)
            if (n & s) {
#pragma unroll
                for (int j = 0; j + s < kPiece; ++j) w[j] = w[j + s];
            }
    }
};

// A lane's piece of a row: columns c .. c+7, of which j = lo .. hi-1 are the
// row's.  Where D is no multiple of 8 rows begin anywhere in 16 bytes of memory,
// so a row's pieces begin `before` columns ahead of it, on 16 bytes: a first and
// a last one are shared with its neighbours, whose columns are loaded, count as 0
// and are not stored.  (Loaded where they fall, 2 bytes off: 2^25 elements in rows
// of 5003 87 us forward and 101 backward; so 64 and 73.)
enum Width { kFew, kAny, kEights };      // under 8 columns; any more; a multiple of 8, all pieces whole

template <int WIDTH>
struct Place {
    int c, lo, hi;
    __device__ __forceinline__ Place(int piece, int before, int D) {
        c = piece * kPiece - (WIDTH == kEights ? 0 : before);
        lo = WIDTH == kEights ? 0 : max(-c, 0);
        hi = WIDTH == kEights ? (c < D ? kPiece : 0) : min(max(D - c, 0), kPiece);
    }
    __device__ __forceinline__ bool whole() const { return lo == 0 && hi == kPiece; }
    __device__ __forceinline__ bool none() const { return hi == 0; }
    __device__ __forceinline__ bool part() const { return WIDTH != kEights && !whole() && !none(); }
    __device__ __forceinline__ bool has(int j) const { return j >= lo && j < hi; }
};

// The columns ahead of row r, a team's first.  They are the same for every row it
// works on where those are a multiple of 8 apart: everywhere but in a backward of
// one workgroup of 1, 2 or 4 teams, whose later rows are loaded where this puts
// them, off 16 bytes.
__device__ __forceinline__ int columns_before(int64_t r, int D, int align) {
    return static_cast<int>(r & 7) * (D & 7) & align;
}

// `last`: nothing may be read behind this row, whose last columns are then
// loaded with those before them, and moved down by `settle` before they are used
// (not here: what follows a load would wait for it).
template <int WIDTH, class T>
__device__ __forceinline__ Piece<T> load8(const T* row, Place<WIDTH> at, bool last) {
    Piece<T> p{};
    if (WIDTH == kFew) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (at.has(j)) p.set(j, row[at.c + j]);
    } else if (!at.none()) {
        __builtin_memcpy(&p.w, row + at.c - (WIDTH == kAny && last ? kPiece - at.hi : 0), kPiece * sizeof(T));
    }
    return p;
}
// Other rows' columns become 0 (a lane without a piece has zeros).
template <int WIDTH, class T>
__device__ __forceinline__ void settle(Piece<T>& p, Place<WIDTH> at, bool last) {
    if (WIDTH == kAny && at.part()) {
        if (last && at.hi < kPiece) p.move_down(kPiece - at.hi);
        p.keep(at.lo, at.hi);
    }
}
// A vector of D, the same for all rows.
template <int WIDTH>
__device__ __forceinline__ void load_columns(const float* v, Place<WIDTH> at, float (&o)[kPiece]) {
    Piece<float> p{};
    if (at.whole()) {
        __builtin_memcpy(&p.w, v + at.c, sizeof(p.w));
    } else if (at.part()) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (at.has(j)) p.set(j, v[at.c + j]);
    }
#pragma unroll
    for (int j = 0; j < kPiece; ++j) o[j] = p[j];
}
template <int WIDTH, class T>
__device__ __forceinline__ void store8(T* row, Place<WIDTH> at, const float (&v)[kPiece]) {
    if (at.whole()) {
        Piece<T> p;
        p.from(v);
        __builtin_memcpy(row + at.c, &p.w, kPiece * sizeof(T));
    } else if (WIDTH == kFew) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (at.has(j)) narrow(v[j], &row[at.c + j]);
    } else if (at.part()) {                              // 4, 2 and 1 of them, from the first on
        Piece<T> p;
        p.from(v);
        T* to = row + at.c + at.lo;
        p.move_down(at.lo);
        const int n = at.hi - at.lo;
#pragma unroll
        for (int s = 4; s >= 1; s /= 2)
            if (n & s) {
                __builtin_memcpy(to, &p.w, s * sizeof(T));
                p.move_down(s);
                to += s;
            }
    }
}
// The same of values that have become others.
template <int WIDTH>
__device__ __forceinline__ void clear_others(float (&v)[kPiece], Place<WIDTH> at) {
    if (at.part() || at.none()) {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
            if (!at.has(j)) v[j] = 0.0f;
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
    float *mean, *rstd, *part, *dweight, *dbias;
    int64_t rows;
    int D, centre;
    int align;                   // 7: pieces begin on 16 bytes, 0: on the row's first column
    float eps;
    int accumulate;
};

template <class TX, class TY, int TL, int V, int WIDTH>
__global__ __launch_bounds__(TL > kNormThreads ? TL : kNormThreads) void norm_fwd_kernel(NormArgs p) {
    constexpr int THREADS = TL > kNormThreads ? TL : kNormThreads;
    constexpr int ROWS = THREADS / TL;                   // rows of a workgroup at once
    static_assert(TL <= kWave || ROWS == 1, "a workgroup's barriers are one row's");
    __shared__ float s_sum[2 * (TL / kWave > 0 ? TL / kWave : 1)];
    const int t = threadIdx.x % TL, D = p.D;
    const float inv = 1.0f / static_cast<float>(D);
    const int64_t group = blockIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS, r0 = group * ROWS + threadIdx.x / TL;
    const int before = columns_before(r0, D, p.align);
    auto place = [&](int i) { return Place<WIDTH>(i * TL + t, before, D); };
    float w[V][kPiece], b[V][kPiece];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_columns(p.weight, place(i), w[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) b[i][j] = 0.0f;
        if (p.bias) load_columns(p.bias, place(i), b[i]);
    }
    int turn = 0;
    for (int64_t r = r0; r < p.rows; r += step) {
        const bool last = r + 1 == p.rows;
        const TX* x = static_cast<const TX*>(p.x) + r * D;
        float h[V][kPiece];
        Piece<TX> in[V], add[V];
#pragma unroll
        for (int i = 0; i < V; ++i) in[i] = load8(x, place(i), last);
        if (p.residual) {
            const TX* res = static_cast<const TX*>(p.residual) + r * D;
#pragma unroll
            for (int i = 0; i < V; ++i) add[i] = load8(res, place(i), last);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                settle(in[i], place(i), last);
                settle(add[i], place(i), last);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {       // what is stored is what is normalised
                    TX o;
                    narrow(in[i][j] + add[i][j], &o);
                    h[i][j] = widen(o);
                }
                store8(static_cast<TX*>(p.total) + r * D, place(i), h[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                settle(in[i], place(i), last);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) h[i][j] = in[i][j];
            }
        }
        float mean = 0.0f;
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
                clear_others(h[i], place(i));
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
            store8(y, place(i), h[i]);
        }
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

// The backward: dx of each row, and each workgroup's sums of the weights'
// gradients over its rows, in `part` [2][G][D] (the gradients themselves where
// there is one workgroup).  The next row is on its way
// while one is worked on: without its dtotal, loaded behind the row's sums, 2^25
// bf16 elements of 2048 columns take 64 us instead of 54.  With four pieces a lane
// (over 8192 columns) a row is held as it is in memory and widened twice, the
// weights' sums are in LDS, a lane's own, and float32 rows are not loaded ahead, so
// that registers hold the rest (12288 columns in bf16 63 us; sums in registers 174).
constexpr int kBwdThreads = 512;

template <class TX, class TY, int TL, int V, int WIDTH>
__global__ __launch_bounds__(kBwdThreads) void norm_bwd_kernel(NormArgs p) {
    constexpr int ROWS = kBwdThreads / TL;
    constexpr bool AHEAD = V <= 2 || sizeof(TX) == 2;
    constexpr bool KEEP = V <= 2;
    constexpr int PIECES = V * TL;
    __shared__ float s_sum[ROWS][2 * (TL / kWave > 0 ? TL / kWave : 1)];
    __shared__ float s_part[ROWS][ROWS > 1 ? (PIECES + 1) * kPiece * (kWave + 1) / kWave + 1 : 1];
    const int t = threadIdx.x % TL, team = threadIdx.x / TL, D = p.D;
    const float inv = 1.0f / static_cast<float>(D);
    const int64_t group = blockIdx.x;
    // (a team without a row loads the last one, from its own first piece on)
    int before = columns_before(min(group * ROWS + team, p.rows - 1), D, p.align);
    auto place = [&](int i) { return Place<WIDTH>(i * TL + t, before, D); };
    float w[V][kPiece], dw[KEEP ? V : 1][kPiece], db[KEEP ? V : 1][kPiece];
    __shared__ floatx4 s_acc[KEEP ? 1 : 2 * V * 2][KEEP ? 1 : kBwdThreads];       // a lane's own, 16 bytes each: [half, piece, half a piece]
    auto in_lds = [&](int half, int i, int j) -> float& { return reinterpret_cast<float*>(&s_acc[(half * V + i) * 2 + j / 4][t])[j % 4]; };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_columns(p.weight, place(i), w[i]);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) {
            if (KEEP) dw[i][j] = db[i][j] = 0.0f;
            else in_lds(0, i, j) = in_lds(1, i, j) = 0.0f;
        }
    }
    struct Row {
        Piece<TX> h[V];
        Piece<TY> dy[V];
        Piece<TX> dtotal[V];
        float mean, rstd;
    };
    auto load = [&](int64_t r) {
        Row o;
        // A team without a row keeps the others' barriers company, with the last row: a
        // branch around its loads costs 60 registers.
        if (ROWS > 1) r = min(r, p.rows - 1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            o.h[i] = load8(static_cast<const TX*>(p.x) + r * D, place(i), r + 1 == p.rows);
            o.dy[i] = load8(static_cast<const TY*>(p.dy) + r * D, place(i), r + 1 == p.rows);
        }
        if (p.dtotal) {
#pragma unroll
            for (int i = 0; i < V; ++i) o.dtotal[i] = load8(static_cast<const TX*>(p.dtotal) + r * D, place(i), r + 1 == p.rows);
        }
        o.mean = p.centre ? p.mean[r] : 0.0f;
        o.rstd = p.rstd[r];
        return o;
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    int turn = 0;
    Row next{};
    if (AHEAD) next = load(group * ROWS + team);
    for (int64_t r0 = group * ROWS; r0 < p.rows; r0 += step) {
        const int64_t r = r0 + team;
        asm volatile("" : "+v"(before));                 // places are made anew: kept, what depends on them takes 10 registers a piece
        Row now = AHEAD ? next : load(r);
        if (AHEAD && r0 + step < p.rows) next = load(r + step);
        if (ROWS > 1 && r >= p.rows) {                   // no row: an infinity in the last one is not this team's to count
#pragma unroll
            for (int i = 0; i < V; ++i) {
                now.h[i] = Piece<TX>{};
                now.dy[i] = Piece<TY>{};
            }
            now.mean = now.rstd = 0.0f;
        }
        float c1 = 0.0f, c2 = 0.0f;
        float xh[KEEP ? V : 1][kPiece], g[KEEP ? V : 1][kPiece];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const auto at = place(i);
            const int k = KEEP ? i : 0;
            settle(now.h[i], at, r + 1 == p.rows);
            settle(now.dy[i], at, r + 1 == p.rows);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                xh[k][j] = (now.h[i][j] - now.mean) * now.rstd;
                g[k][j] = now.dy[i][j];
                (KEEP ? dw[k][j] : in_lds(0, i, j)) += g[k][j] * xh[k][j];
                (KEEP ? db[k][j] : in_lds(1, i, j)) += g[k][j];
                g[k][j] *= w[i][j];
                c1 += g[k][j] * xh[k][j];
                c2 += g[k][j];
            }
            if (!KEEP) {
                now.h[i].forget();
                now.dy[i].forget();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        c1 = row_total<TL>(c1, s_sum[team], turn++) * inv;
        c2 = p.centre ? row_total<TL>(c2, s_sum[team], turn++) * inv : 0.0f;
        if (ROWS > 1 && r >= p.rows) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const auto at = place(i);
            const int k = KEEP ? i : 0;
            float o[kPiece];
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
                if (!KEEP) xh[k][j] = (now.h[i][j] - now.mean) * now.rstd, g[k][j] = now.dy[i][j] * w[i][j];
                o[j] = (g[k][j] - c2 - xh[k][j] * c1) * now.rstd;
            }
            if (p.dtotal) {
                if (WIDTH == kAny && r + 1 == p.rows && at.part()) now.dtotal[i].move_down(kPiece - at.hi);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) o[j] += now.dtotal[i][j];
            }
            store8(static_cast<TX*>(p.dx) + r * D, at, o);
            if (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
    }
    // The teams' sums of a column are added in order.  In LDS a column of 64 is
    // left out after every 64, so that lanes eight columns apart meet no other's bank.
    auto spot = [](int column) { return column + column / kWave; };
#pragma unroll 1
    for (int half = 0; half < (p.dbias ? 2 : 1); ++half) {
        const bool only = gridDim.x == 1;                // nothing else to add
        float* part = only ? (half ? p.dbias : p.dweight) : p.part + (static_cast<int64_t>(half) * gridDim.x + group) * D;
        if (ROWS > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < kPiece; ++j) s_part[team][spot(place(i).c + kPiece + j)] = half ? db[KEEP ? i : 0][j] : dw[KEEP ? i : 0][j];
            __syncthreads();
            for (int c = threadIdx.x; c < D; c += kBwdThreads) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < ROWS; ++k) s += s_part[k][spot(c + kPiece)];
                part[c] = only && p.accumulate ? part[c] + s : s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float o[kPiece];
#pragma unroll
                for (int j = 0; j < kPiece; ++j) o[j] = KEEP ? (half ? db[KEEP ? i : 0][j] : dw[KEEP ? i : 0][j]) : in_lds(half, i, j);
                if (only && p.accumulate) {
                    float old[kPiece];
                    load_columns(part, place(i), old);
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) o[j] += old[j];
                }
                store8(part, place(i), o);
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

template <class TX, class TY, int TL, int V, int WIDTH>
void launch_fwd(const NormArgs& a, hipStream_t s) {
    constexpr int THREADS = std::max(TL, kNormThreads), ROWS = THREADS / TL;
    const int64_t blocks = std::min<int64_t>((a.rows + ROWS - 1) / ROWS, 2048);
    norm_fwd_kernel<TX, TY, TL, V, WIDTH><<<static_cast<unsigned>(blocks), THREADS, 0, s>>>(a);
}

// Pieces of a row of D columns, on 16 bytes: it begins up to 8 less its and 8's
// common divisor behind one.  Rows too wide for one more begin at theirs.
int pieces_on_16_bytes(int D) { return (D + (D % 8 ? 8 - (D & -D) : 0) + kPiece - 1) / kPiece; }
int row_align(int D) { return D >= kPiece && pieces_on_16_bytes(D) <= kMaxNormDim / kPiece ? 7 : 0; }
int row_pieces(int D) { return row_align(D) ? pieces_on_16_bytes(D) : (D + kPiece - 1) / kPiece; }

// Lanes a row and pieces a lane.  The backward's sums take twice the registers:
// two pieces a lane, four above 8192 columns, where they are in LDS.
constexpr int bwd_lanes(int pieces) {
    return pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 128 ? 64 : pieces <= 256 ? 128
           : pieces <= 512 ? 256 : 512;
}
template <class TX, class TY, int WIDTH>
void by_pieces_fwd(const NormArgs& a, hipStream_t s) {
    const int pieces = row_pieces(a.D);
    if (pieces <= 8) launch_fwd<TX, TY, 8, 1, WIDTH>(a, s);
    else if (pieces <= 16) launch_fwd<TX, TY, 16, 1, WIDTH>(a, s);
    else if (pieces <= 32) launch_fwd<TX, TY, 32, 1, WIDTH>(a, s);
    else if (pieces <= 64) launch_fwd<TX, TY, 64, 1, WIDTH>(a, s);
    else if (pieces <= 128) launch_fwd<TX, TY, 64, 2, WIDTH>(a, s);
    else if (pieces <= 192) launch_fwd<TX, TY, 64, 3, WIDTH>(a, s);
    else if (pieces <= 256) launch_fwd<TX, TY, 64, 4, WIDTH>(a, s);
    else if (pieces <= 512) launch_fwd<TX, TY, 256, 2, WIDTH>(a, s);
    else if (pieces <= 768) launch_fwd<TX, TY, 256, 3, WIDTH>(a, s);
    else if (pieces <= 1024) launch_fwd<TX, TY, 256, 4, WIDTH>(a, s);
    else if (pieces <= 1536) launch_fwd<TX, TY, 512, 3, WIDTH>(a, s);
    else launch_fwd<TX, TY, 512, 4, WIDTH>(a, s);
}
template <class TX, class TY>
void by_width_fwd(const NormArgs& a, hipStream_t s) {
    if (a.D < kPiece) launch_fwd<TX, TY, 8, 1, kFew>(a, s);
    else if (a.D % kPiece) by_pieces_fwd<TX, TY, kAny>(a, s);
    else by_pieces_fwd<TX, TY, kEights>(a, s);
}
template <class TX, class TY, int WIDTH>
void by_pieces_bwd(const NormArgs& a, int G, hipStream_t s) {
    const int pieces = row_pieces(a.D);
    switch (bwd_lanes(pieces)) {
        case 8: norm_bwd_kernel<TX, TY, 8, 1, WIDTH><<<G, kBwdThreads, 0, s>>>(a); return;
        case 16: norm_bwd_kernel<TX, TY, 16, 1, WIDTH><<<G, kBwdThreads, 0, s>>>(a); return;
        case 32: norm_bwd_kernel<TX, TY, 32, 1, WIDTH><<<G, kBwdThreads, 0, s>>>(a); return;
        case 64:
            if (pieces <= 64) norm_bwd_kernel<TX, TY, 64, 1, WIDTH><<<G, kBwdThreads, 0, s>>>(a);
            else norm_bwd_kernel<TX, TY, 64, 2, WIDTH><<<G, kBwdThreads, 0, s>>>(a);
            return;
        case 128: norm_bwd_kernel<TX, TY, 128, 2, WIDTH><<<G, kBwdThreads, 0, s>>>(a); return;
        case 256: norm_bwd_kernel<TX, TY, 256, 2, WIDTH><<<G, kBwdThreads, 0, s>>>(a); return;
        default:
            if (pieces <= 1024) norm_bwd_kernel<TX, TY, 512, 2, WIDTH><<<G, kBwdThreads, 0, s>>>(a);
            else norm_bwd_kernel<TX, TY, 512, 4, WIDTH><<<G, kBwdThreads, 0, s>>>(a);
    }
}
template <class TX, class TY>
void by_width_bwd(const NormArgs& a, int G, hipStream_t s) {
    if (a.D < kPiece) norm_bwd_kernel<TX, TY, 8, 1, kFew><<<G, kBwdThreads, 0, s>>>(a);
    else if (a.D % kPiece) by_pieces_bwd<TX, TY, kAny>(a, G, s);
    else by_pieces_bwd<TX, TY, kEights>(a, G, s);
}

// Workgroups of the backward: one a compute unit, since their sums, 8 * D bytes
// each, are written and read once more, and no more than have a row.  A few rows
// are one workgroup's, which writes the weights' gradients itself: up to four a
// team (two where rows share 16 bytes, whose ends take longer), 7.8 to 9.3 us a call
// against 10.2 with the second launch (eight: 14; four of 777 columns: 13).
int bwd_groups(int64_t rows, int D) {
    const int teams = kBwdThreads / bwd_lanes(row_pieces(D));
    if (rows <= (D % kPiece ? 2 : 4) * teams) return 1;
    return static_cast<int>(std::min<int64_t>((rows + teams - 1) / teams, 256));
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

size_t type_bytes(int32_t type) { return type == MOE_F32 ? 4 : 2; }

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
    const size_t n = static_cast<size_t>(rows) * D, row = static_cast<size_t>(rows) * sizeof(float), col = static_cast<size_t>(D) * sizeof(float);
    const Span sx{x, n * type_bytes(x_type)}, sr{residual, sx.bytes}, sw{weight, col}, sb{bias, col}, sh{total, sx.bytes},
        sy{y, n * type_bytes(y_type)}, sm{mean, row}, ss{rstd, row};
    // (a row's total is stored before its y: one of them would be lost)
    if (!sh.apart_or_one_of({sx, sr}) || !sh.apart({sw, sb, sy, sm, ss}) || !sy.apart_or_one_of({sx, sr}) ||
        !sy.apart({sw, sb, sm, ss}) || !sm.apart({sx, sr, sw, sb, ss}) || !ss.apart({sx, sr, sw, sb}))
        return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.total = total; a.y = y;
    a.mean = mean; a.rstd = rstd; a.rows = rows; a.D = D; a.centre = mean != nullptr; a.align = row_align(D);
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
    const size_t need = moe_layer_norm_bwd_workspace_bytes(rows, D);
    if (workspace_bytes < need) return MOE_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(rows) * D, row = static_cast<size_t>(rows) * sizeof(float), col = static_cast<size_t>(D) * sizeof(float);
    const Span sy{dy, n * type_bytes(y_type)}, sh{h, n * type_bytes(x_type)}, sw{weight, col}, sm{mean, row}, ss{rstd, row},
        sd{dtotal, sh.bytes}, sx{dx, sh.bytes}, sdw{dweight, col}, sdb{dbias, col}, sp{workspace, need};
    if (!sx.apart_or_one_of({sy, sh, sd}) || !sx.apart({sw, sm, ss, sdw, sdb, sp}) || !sdw.apart({sy, sh, sd, sw, sm, ss, sdb, sp}) ||
        !sdb.apart({sy, sh, sd, sw, sm, ss, sp}) || !sp.apart({sy, sh, sd, sw, sm, ss}))
        return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = h; a.dy = dy; a.dtotal = dtotal; a.weight = weight; a.dx = dx;
    a.dweight = dweight; a.dbias = dbias; a.accumulate = accumulate;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.part = static_cast<float*>(workspace); a.rows = rows; a.D = D; a.centre = mean != nullptr;
    a.align = row_align(D);
    if (rows) {
        if (x_type == MOE_BF16) by_width_bwd<Bf16, Bf16>(a, G, stream);
        else if (y_type == MOE_BF16) by_width_bwd<float, Bf16>(a, G, stream);
        else by_width_bwd<float, float>(a, G, stream);
    }
    if (!rows || G > 1) norm_finish_kernel<<<dim3((D + kWave - 1) / kWave, dbias ? 2 : 1), kFinishThreads, 0, stream>>>(
        a.part, rows ? G : 0, D, accumulate, dweight, dbias);
    return launch_status();
}

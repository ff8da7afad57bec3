// Steps 4-5 of the dropless MoE FFN forward on 4-bit expert weights, for the
// few tokens of a decode step.
//
//   act[s]       = silu(x_r W1g^T) * (x_r W1u^T) * p_s     r = sorted_slot_ids[s]
//   route_out[s] = act[s] W2^T                             (float32)
//   y[t]         = bf16( sum_k route_out[token_routes[t, k]] )
//
// With a handful of rows per expert the weights' bytes are the time: every
// byte of an expert in use is read once for up to 32 of its rows, and
// everything else is kept out of the way of that stream.
//   * gfx950's v_cvt_scalef32_pk_bf16_fp4 turns two codes into two scaled bf16
//     (exact: a 2-bit significand times a power of two) in one instruction,
//     half a vector instruction per weight.
//   * The products are 16x16x32 bf16 MFMAs with 16 weight rows as the first
//     operand and up to 16 routes as the second.
//   * A row's scale bytes are loaded for 2048 columns at once and kept in LDS.
//     Loaded step by step, 8 bytes of each of 64 rows, they took a quarter of
//     the time (a wide layer's FC1 266 us against 186 without them, 173 now).
//   * A contraction is summed in four parts, added in order.  With few tiles
//     (w4_split_kernel) the four waves of a workgroup take a part each; with
//     many (w4_stream_kernel) every wave runs all four for its own rows and
//     the routes' rows are shared through LDS.  The additions are the same, so
//     a route's result is the same, bit for bit, whatever else is in the batch.
//   * FC1 pairs gate and up rows in one wave, so the SwiGLU and the route's
//     probability are applied to the sums in registers.
//   * The weights' first loads leave as soon as the expert is known, before
//     the block's row count and tokens are.
//
// A layer of 128 experts (8 a token, H 2048, I 768), device time with so many
// sets of weights in turn that none stays in the caches: one token 14.2 us (FC1
// 7.4, FC2 and the sum 6.7; 10.4 us when the caches hold the weights), 16 tokens 54
// us (FC1 31, FC2 18), 128 tokens 79 us (FC1 47, FC2 27: 4.3 TB/s of weights; a
// plain read of as many bytes takes 34 + 18).
#include <algorithm>
#include <initializer_list>

#include "gemm_common.h"
#include "lowbit.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kW4Step = 256;     // columns of a step: 128 bytes of codes a row, 8 scale bytes
constexpr int kW4Parts = 4;      // parts of a contraction, summed apart and added in order
constexpr int kW4Waves = 4;      // waves of a workgroup of the grouped kernel
constexpr int kW4Panel = 8;      // steps whose scale bytes are staged together
constexpr int kW4Pitch = 72;     // LDS bytes of a weight row's panel: 64, and 8 that spread the banks

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

// 8 codes (one word) as 8 bf16 times 2^(b - 127), the scale byte b in the
// float's exponent field: the instruction reads that field alone, so b = 0
// is 2^-127 and b = 255 makes every value NaN.
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

// Half a 256-wide step of one 16-row weight tile against CT column tiles.  The
// codes of columns 64q + 32h .. +31 of its row are one 16-byte piece and one
// scale group of lane (r16, q), 8 columns a word; any order of the contraction
// will do that both operands share, so the i-th MFMA takes every lane's i-th
// word, and the other operand's lanes the same columns of their rows.
template <int CT>
__device__ __forceinline__ void w4_piece(u32x4 codes, uint32_t scale_byte, const u32x4 (&xw)[CT][4], floatx4 (&acc)[CT]) {
    const float scale = __uint_as_float(scale_byte << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x8 a = w4_values(codes[i], scale);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, xw[c][i]), acc[c], 0, 0, 0);
    }
}

// A wave's LDS operations are in order; this keeps the compiler from moving
// reads and writes past each other.
__device__ __forceinline__ void w4_wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// First step of part i of a contraction of `steps` steps.
__device__ __forceinline__ int w4_part(int steps, int i) { return steps * i / kW4Parts; }

// What a wave knows of its weights: WT tiles of 16 rows (FC1: a gate and an up
// tile for each of its WT/2 output column tiles) from output column col0 on.
// SALIGN: rows of scale bytes are whole words (Kdim a multiple of 128).
template <bool FC1, int WT, bool SALIGN>
struct W4Rows {
    static constexpr int ROWS = 16 * WT;
    static constexpr int RT = FC1 ? WT / 2 : WT;        // output column tiles
    static constexpr int SREGS = SALIGN ? kW4Panel * 2 : kW4Panel * 2 + 1;
    static_assert(ROWS <= kWave, "a row of scales a lane");
    const W4Args& p;
    const int lane, wave, r16, q, steps, sbytes;
    int lo, hi;                  // the wave's steps
    int col0, slot0, n;          // first output column and slot, live routes
    __amdgpu_buffer_rsrc_t codes, scales, rows;
    uint32_t soff, shift;
    uint32_t sv[SREGS];
    uint8_t* s_scale;            // the wave's LDS panel of scale bytes

    __device__ __forceinline__ W4Rows(const W4Args& a, bool split)
        : p(a), lane(threadIdx.x & (kWave - 1)),
          wave(__builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave)),
          r16(lane & 15), q(lane >> 4), steps((a.Kdim + kW4Step - 1) / kW4Step), sbytes(a.Kdim / kGroup) {
        lo = split ? w4_part(steps, wave) : 0;
        hi = split ? w4_part(steps, wave + 1) : steps;
    }

    __device__ __forceinline__ int row_of(int t, int r) const {   // weight row r of tile t, or -1
        const int col = col0 + (FC1 ? t / 2 : t) * 16 + r;
        return col < p.ncols ? (FC1 && (t & 1) ? p.ncols + col : col) : -1;
    }
    __device__ __forceinline__ uint32_t code_offset(int t, int r, int byte) const {
        const int row = row_of(t, r);
        return row >= 0 ? static_cast<uint32_t>(row) * (p.Kdim / 2) + byte : kOob;
    }

    // Descriptors of expert e's weights; rows past the last read zeros.
    __device__ __forceinline__ void weights(int e) {
        const int64_t base = static_cast<int64_t>(e) * p.wrows;
        codes = buffer(p.codes + base * (p.Kdim / 2), static_cast<uint32_t>(p.wrows) * (p.Kdim / 2));
        scales = buffer(p.scales + base * sbytes, static_cast<uint32_t>(p.wrows) * sbytes);
        const int row = lane < ROWS ? row_of(lane >> 4, lane & 15) : -1;
        soff = row >= 0 ? static_cast<uint32_t>(row) * sbytes : kOob;
        shift = (soff & 2) * 8;
        soff &= ~3u;
    }
    // The block's live routes, and the descriptor of their rows.  False: none.
    __device__ __forceinline__ bool routes(int b, int e) {
        const int rel = b - p.block_start[e];
        n = rel < 0 ? 0 : min(min(p.route_counts[e] - rel * kBlockM, kBlockM), p.R - slot0);
        if (n <= 0) return false;
        rows = FC1 ? buffer(p.a, static_cast<uint32_t>(p.N) * p.Kdim * 2u)
                   : buffer(p.a + static_cast<int64_t>(slot0) * p.Kdim, static_cast<uint32_t>(n) * p.Kdim * 2u);
        return true;
    }
    // Byte offset of column byte `byte` of route i's row, which FC1 finds at
    // token `tok`; a route that is none reads zeros.
    __device__ __forceinline__ uint32_t row_offset(int i, int tok, int byte) const {
        const int row = FC1 ? tok : i;
        return i < n && static_cast<unsigned>(row) < static_cast<unsigned>(FC1 ? p.N : n)
            ? static_cast<uint32_t>(row) * p.Kdim * 2u + byte : kOob;
    }

    // The scale bytes of the panel that starts at step kp, one weight row a
    // lane, in words.  Where rows are not whole words, every other row starts in
    // the middle of one: then one word more is loaded, and the pieces are put
    // together on the way to LDS.  Bytes past the row's end (the next row's,
    // which may stand for NaN) become 0.
    __device__ __forceinline__ int panel_bytes(int kp) const {
        return min(min(kW4Panel, hi - kp) * 8, sbytes - kp * 8);
    }
    __device__ __forceinline__ void load_scales(int kp) {
        const int cnt = panel_bytes(kp);
        const uint32_t at = soff + kp * 8;
#pragma unroll
        for (int i = 0; i < SREGS; ++i) sv[i] = 0;
        if (SALIGN) {
#pragma unroll
            for (int i = 0; i < kW4Panel * 2; i += 4) {
                if (i * 4 + 16 <= cnt) {
                    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(scales, at + i * 4, 0, 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) sv[i + j] = v[j];
                } else {
#pragma unroll
                    for (int j = i; j < i + 4; ++j)
                        if (j * 4 < cnt) sv[j] = __builtin_amdgcn_raw_buffer_load_b32(scales, at + j * 4, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < SREGS; ++i)
                if (i * 4 < cnt + 2) sv[i] = __builtin_amdgcn_raw_buffer_load_b32(scales, at + i * 4, 0, 0);
        }
    }
    // The panel is the wave's own.
    __device__ __forceinline__ void store_scales(int kp) {
        const int cnt = panel_bytes(kp);
        w4_wave_fence();
#pragma unroll
        for (int i = 0; i < kW4Panel; ++i) {
            u32x2 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int w = 2 * i + h;
                v[h] = SALIGN ? sv[w] : __builtin_amdgcn_alignbit(sv[SALIGN ? w : w + 1], sv[w], shift);
                if (!SALIGN) v[h] = w * 4 >= cnt ? 0u : w * 4 + 2 == cnt ? v[h] & 0xFFFFu : v[h];
            }
            if (lane < ROWS) *reinterpret_cast<u32x2*>(s_scale + lane * kW4Pitch + i * 8) = v;
        }
        w4_wave_fence();
    }
    // The scale byte of half h of the lane's columns of tile t, at step k of a
    // panel that starts at kp.
    __device__ __forceinline__ uint32_t scale_byte(int t, int k, int kp, int h) const {
        return s_scale[(t * 16 + r16) * kW4Pitch + (k - kp) * 8 + q * 2 + h];
    }

    // Output tile t of one route: the lane's 4 columns col0 + 16t + 4q .. +3,
    // from the sums sum(weight tile).
    template <class SUM>
    __device__ __forceinline__ void put(int t, int route, SUM sum) const {
        const int col = col0 + 16 * t + 4 * q;
        if (route >= n || col >= p.ncols) return;
        const int64_t at = static_cast<int64_t>(slot0 + route) * p.ncols + col;
        if (FC1) {
            const floatx4 g = sum(2 * t), u = sum(2 * t + 1);
            const float pr = p.slot_probs[slot0 + route];
            uint2 o;
            o.x = pack_bf16x2(silu(g[0]) * u[0] * pr, silu(g[1]) * u[1] * pr);
            o.y = pack_bf16x2(silu(g[2]) * u[2] * pr, silu(g[3]) * u[3] * pr);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = o;
        } else {
            *reinterpret_cast<floatx4*>(static_cast<float*>(p.out) + at) = sum(t);
        }
    }
};

// ---------------------------------------------------------------- few tiles
// Workgroup (x, y): WT weight tiles and layout block y; wave w sums part w of
// the contraction.  Loads go straight to operand registers, the shortest way
// when a wave has one step.  Lane (r16, q) takes the 32 bytes of codes of
// columns 64q .. 64q+63 of its row, and the other operand's lanes those columns
// of their rows.  STAGED: the codes come in whole lines and through LDS of the
// wave's own (which needs no barrier), for contractions of 6 steps and more,
// where 64 cache accesses a load add up (FC1 of one token in 64 or 128 experts:
// 6 steps 5.3 us against 5.7, 8 5.9 against 6.5, 27 10.7 against 13.0; FC2 of 8
// rows an expert, 5 steps 8.8 against 8.6, 6 9.0 against 9.3).  Only where rows are
// whole words of scales: the codes of the others begin in the middle of a 64-byte
// piece (9 steps 7.0 us staged, 6.5 straight, 17 9.4 against 9.1).
template <bool FC1, int WT, bool SALIGN, bool STAGED>
struct W4Split : W4Rows<FC1, WT, SALIGN> {
    typedef W4Rows<FC1, WT, SALIGN> B;
    using B::p; using B::lane; using B::wave; using B::r16; using B::q; using B::lo; using B::hi; using B::n;
    static constexpr int CODES = STAGED ? B::ROWS * 128 : 0;   // LDS bytes of a step's codes
    uint32_t coff[STAGED ? 2 * WT : WT];
    u32x4 cw[2 * WT];            // direct: [tile][half]; STAGED: 8 rows each, on their way
    uint8_t* s_codes;

    __device__ __forceinline__ explicit W4Split(const W4Args& a) : B(a, true) {}

    __device__ __forceinline__ void load_codes(int k) {
        // past the row's end: zeros
        const bool live = k * kW4Step + (STAGED ? lane % 8 * 32 : q * 64) < p.Kdim;
#pragma unroll
        for (int i = 0; i < 2 * WT; ++i)
            cw[i] = __builtin_amdgcn_raw_buffer_load_b128(
                this->codes, !live ? kOob : k * (kW4Step / 2) + (STAGED ? coff[i] : coff[i / 2] + i % 2 * 16), 0, 0);
    }
    __device__ __forceinline__ void store_codes() const {
        w4_wave_fence();
#pragma unroll
        for (int i = 0; i < 2 * WT; ++i) {
            const int row = 8 * i + lane / 8;
            *reinterpret_cast<u32x4*>(s_codes + row * 128 + ((lane % 8) ^ (row / 2 % 8)) * 16) = cw[i];
        }
        w4_wave_fence();
    }
    __device__ __forceinline__ u32x4 operand(int t, int h) const {
        return STAGED ? *reinterpret_cast<const u32x4*>(
                            s_codes + (t * 16 + r16) * 128 + ((q * 2 + h) ^ (r16 / 2 % 8)) * 16)
                      : cw[2 * t + h];
    }

    // Routes c0 .. c0 + 16*CT - 1.  fetched: the first step's codes and scales
    // are already on their way.
    template <int CT>
    __device__ __forceinline__ void run(int c0, const int* tok, bool fetched, floatx4* s_acc) {
        uint32_t aoff[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) aoff[c] = this->row_offset(c0 + c * 16 + r16, tok[c], q * 128);
        floatx4 acc[WT][CT];
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[t][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = lo, kp = lo; k < hi; ++k) {
            if (k - kp == kW4Panel) kp = k;
            if (!(fetched && k == lo)) {
                if (k == kp) this->load_scales(k);
                load_codes(k);
            }
            u32x4 xw[2][CT][4];
            const bool live = k * kW4Step + q * 64 < p.Kdim;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    xw[i / 4][c][i % 4] = __builtin_amdgcn_raw_buffer_load_b128(
                        this->rows, live ? aoff[c] + k * (kW4Step * 2) + i * 16 : kOob, 0, 0);
            // every load of the step is issued before the first result is waited for
            __builtin_amdgcn_sched_barrier(0);
            if (k == kp) this->store_scales(k);
            if (STAGED) store_codes();
#pragma unroll
            for (int t = 0; t < WT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w4_piece<CT>(operand(t, h), this->scale_byte(t, k, kp, h), xw[h], acc[t]);
        }
        // the parts meet in LDS, in the place of codes and scales
        __syncthreads();
        floatx4* mine = s_acc + wave * WT * CT * kWave + lane;
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) mine[(t * CT + c) * kWave] = acc[t][c];
        __syncthreads();
        for (int i = wave; i < B::RT * CT; i += kW4Waves) {
            const int c = i % CT;
            this->put(i / CT, c0 + 16 * c + r16, [&](int t) {
                const floatx4* at = s_acc + (t * CT + c) * kWave + lane;
                floatx4 v = at[0];
#pragma unroll
                for (int j = 1; j < kW4Parts; ++j) v += at[j * WT * CT * kWave];
                return v;
            });
        }
    }
};

// CTMAX: the most 16-route tiles held at once; with 1, a block of more than 16
// routes reads its weights twice, the second time from the caches.
template <bool FC1, int WT, int CTMAX, bool SALIGN, bool STAGED>
__global__ __launch_bounds__(kW4Waves * kWave) void w4_split_kernel(W4Args p) {
    typedef W4Split<FC1, WT, SALIGN, STAGED> Wave;
    constexpr int WAVE_BYTES = Wave::CODES + Wave::ROWS * kW4Pitch;
    constexpr int ACC_BYTES = kW4Waves * WT * CTMAX * kWave * 16;
    __shared__ __attribute__((aligned(16))) uint8_t smem[kW4Waves * WAVE_BYTES > ACC_BYTES ? kW4Waves * WAVE_BYTES : ACC_BYTES];
    static_assert(kW4Waves == kW4Parts, "a part a wave");
    Wave w(p);
    const int b = blockIdx.y;                           // < R / BM
    w.slot0 = b * kBlockM;
    int tok[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) tok[c] = FC1 ? p.sorted_slot_ids[w.slot0 + c * 16 + w.r16] : 0;
    const int e = p.expert_ids[b];                      // device data: range-checked
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.E)) return;      // past the extent
    w.s_codes = smem + w.wave * WAVE_BYTES;
    w.s_scale = w.s_codes + Wave::CODES;
    w.col0 = blockIdx.x * (16 * Wave::RT);
    w.weights(e);
#pragma unroll
    for (int i = 0; i < (STAGED ? 2 * WT : WT); ++i)
        w.coff[i] = STAGED ? w.code_offset(i / 2, i % 2 * 8 + w.lane / 8, w.lane % 8 * 16)
                           : w.code_offset(i, w.r16, w.q * 32);
    if (w.lo < w.hi) {
        w.load_scales(w.lo);
        w.load_codes(w.lo);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!w.routes(b, e)) return;
    floatx4* const s_acc = reinterpret_cast<floatx4*>(smem);
    if (CTMAX == 1) {
        w.template run<1>(0, tok, true, s_acc);
        if (w.n > 16) {
            __syncthreads();                            // the sums are read
            w.template run<1>(16, tok + 1, false, s_acc);
        }
    } else if (w.n <= 16) {
        w.template run<1>(0, tok, true, s_acc);
    } else {
        w.template run<CTMAX>(0, tok, true, s_acc);
    }
}

// --------------------------------------------------------------- many tiles
// Workgroup (x, y): the weight tiles of its four waves, WT each, and layout
// block y.  Loads straight to operand registers take 64 cache accesses each,
// since neighbouring lanes are different rows; that, not memory, bounded them
// (the address units 60% busy).  Here codes come in whole lines, 8 rows of 128
// bytes a load, and the routes' rows once for the four waves; both pass
// through LDS into operand layout, and the next step's loads run beside this
// step's products.  An operand is read from LDS where it is used and one wave
// needs few registers, which is what lets four workgroups share a compute unit
// (three with two route tiles).  128 tokens of the 128-expert layer, three sets of
// weights in turn: FC1 45 us (48.6 with the split kernel), FC2 26 us (29.3); 256
// tokens 48.6 (69) and 30 (45).  Two steps'
// loads on their way, 64-row waves, waves two by two, eight waves a workgroup
// and several column tiles a workgroup in turn were no faster.
template <bool FC1, int WT, bool SALIGN>
struct W4Stream : W4Rows<FC1, WT, SALIGN> {
    typedef W4Rows<FC1, WT, SALIGN> B;
    using B::p; using B::lane; using B::wave; using B::r16; using B::q; using B::steps; using B::n;
    static_assert(64 % (16 * B::RT) == 0, "a wave's columns are all there or none");
    // LDS pitches: 16 bytes past the 128 of a row's codes and the 512 of a route's
    // step, so that 16 lanes with a row each meet no bank twice, and every
    // operand is one address and a constant away
    static constexpr int CPITCH = 144, RPITCH = 528;
    uint32_t coff;               // of the lane's piece of the first 8 rows
    u32x4 cr[2 * WT];            // codes on their way
    uint8_t* s_codes;            // the wave's own
    uint8_t* s_rows;             // the workgroup's

    __device__ __forceinline__ explicit W4Stream(const W4Args& a) : B(a, false) {}

    // Load i brings rows 8(i % 2) .. +7 of tile i / 2: this far below the first.
    __device__ __forceinline__ int below(int i) const {
        return (FC1 ? i / 4 : i / 2) * 16 + i % 2 * 8 + (FC1 && (i & 2) ? p.ncols : 0);
    }
    __device__ __forceinline__ void load_codes(int k) {
        const bool live = k * kW4Step + lane % 8 * 32 < p.Kdim;   // past the row's end: zeros
#pragma unroll
        for (int i = 0; i < 2 * WT; ++i)
            cr[i] = __builtin_amdgcn_raw_buffer_load_b128(
                this->codes, live ? coff : kOob, below(i) * (p.Kdim / 2) + k * (kW4Step / 2), 0);
    }

    template <int CT>
    __device__ __forceinline__ void run(int c0, const int (*tok)[2], bool fetched) {
        // the wave brings 4 rows of each 16-row tile, two a load, 512 bytes each
        uint32_t aoff[CT][2];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = c0 + c * 16 + 4 * wave + 2 * j + lane / 32;
                aoff[c][j] = this->row_offset(i, tok[c][j], lane % 32 * 16);
            }
        u32x4 xr[CT][2];
        auto load_rows = [&](int k) {
            const bool live = k * kW4Step + lane % 32 * 8 < p.Kdim;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    xr[c][j] = __builtin_amdgcn_raw_buffer_load_b128(
                        this->rows, live ? aoff[c][j] : kOob, k * (kW4Step * 2), 0);
        };
        floatx4 acc[WT][CT], tot[WT][CT];
#pragma unroll
        for (int t = 0; t < WT; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[t][c] = tot[t][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        if (!fetched) {
            this->load_scales(0);
            load_codes(0);
        }
        load_rows(0);
        int k = 0, kp = 0;
        auto step = [&]() {
            if (k - kp == kW4Panel) kp = k;
            __builtin_amdgcn_sched_barrier(0);
            if (k > 0) __syncthreads();                 // the last step's rows are read
            if (k == kp) this->store_scales(k);
#pragma unroll
            for (int i = 0; i < 2 * WT; ++i) {
                const int row = 8 * i + lane / 8;
                *reinterpret_cast<u32x4*>(s_codes + row * CPITCH + lane % 8 * 16) = cr[i];
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = 4 * wave + 2 * j + lane / 32;
                    *reinterpret_cast<u32x4*>(s_rows + (c * 16 + row) * RPITCH + lane % 32 * 16) = xr[c][j];
                }
            __builtin_amdgcn_sched_barrier(0);
            if (k + 1 < steps) {
                if (k + 1 - kp == kW4Panel) this->load_scales(k + 1);
                load_codes(k + 1);
                load_rows(k + 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            __syncthreads();                            // the rows are there
#pragma unroll
            for (int h = 0; h < 2; ++h) {               // half a step at a time: its operands in registers
                u32x4 cw[WT];
                float sc[WT];
#pragma unroll
                for (int t = 0; t < WT; ++t) {
                    cw[t] = *reinterpret_cast<const u32x4*>(s_codes + (t * 16 + r16) * CPITCH + (q * 2 + h) * 16);
                    sc[t] = __uint_as_float(this->scale_byte(t, k, kp, h) << 23);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u32x4 xw[CT];
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        xw[c] = *reinterpret_cast<const u32x4*>(
                            s_rows + (c * 16 + r16) * RPITCH + (q * 8 + h * 4 + i) * 16);
#pragma unroll
                    for (int t = 0; t < WT; ++t) {
                        const bf16x8 a = w4_values(cw[t][i], sc[t]);
#pragma unroll
                        for (int c = 0; c < CT; ++c)
                            acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                a, __builtin_bit_cast(bf16x8, xw[c]), acc[t][c], 0, 0, 0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
#pragma unroll 1
        for (int part = 0; part < kW4Parts; ++part) {
#pragma unroll 1
            for (const int end = w4_part(steps, part + 1); k < end; ++k) step();
#pragma unroll
            for (int t = 0; t < WT; ++t)
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    tot[t][c] += acc[t][c];
                    acc[t][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
                }
        }
#pragma unroll
        for (int t = 0; t < B::RT; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c)
                this->put(t, c0 + 16 * c + r16, [&](int i) { return tot[i][c]; });
    }
};

// One route tile takes 107 to 111 registers, four waves a SIMD; two are held to
// three (167 registers instead of 179: 256 tokens of 8 experts of 4096 x 1792 FC1
// 36.4 us against 43.6, of 128 experts of 2048 x 768 48.6 against 51.6).
template <bool FC1, int WT, int CTMAX, bool SALIGN>
__global__ __launch_bounds__(kW4Waves * kWave, CTMAX == 1 ? 4 : 3) void w4_stream_kernel(W4Args p) {
    typedef W4Stream<FC1, WT, SALIGN> Wave;
    constexpr int SCALE = Wave::ROWS * kW4Pitch, CODES = Wave::ROWS * Wave::CPITCH, ROWS = CTMAX * 16 * Wave::RPITCH;
    __shared__ __attribute__((aligned(256))) uint8_t smem[ROWS + kW4Waves * (CODES + SCALE)];
    Wave w(p);
    const int b = blockIdx.y;                           // < R / BM
    w.slot0 = b * kBlockM;
    int tok[2][2];                                      // of the rows that the wave brings
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            tok[c][j] = FC1 ? p.sorted_slot_ids[w.slot0 + c * 16 + 4 * w.wave + 2 * j + w.lane / 32] : 0;
    const int e = p.expert_ids[b];                      // device data: range-checked
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(p.E)) return;      // past the extent
    w.s_rows = smem;
    w.s_codes = smem + ROWS + w.wave * CODES;
    w.s_scale = smem + ROWS + kW4Waves * CODES + w.wave * SCALE;
    w.col0 = (blockIdx.x * kW4Waves + w.wave) * (16 * Wave::RT);
    w.weights(e);
    w.coff = w.code_offset(0, w.lane / 8, w.lane % 8 * 16);
    w.load_scales(0);
    w.load_codes(0);
    __builtin_amdgcn_sched_barrier(0);
    if (!w.routes(b, e)) return;                        // uniform over the workgroup
    if (CTMAX == 1) {
        w.template run<1>(0, tok, true);
        if (w.n > 16) {
            __syncthreads();                            // the last step's rows are read
            w.template run<1>(16, tok + 1, false);
        }
    } else if (w.n <= 16) {
        w.template run<1>(0, tok, true);
    } else {
        w.template run<CTMAX>(0, tok, true);
    }
}

// ------------------------------------------------------------ a few tokens
// FC2 and the token's sum in one launch: workgroup (x, y) forms 16 columns of
// y[token y].  Its waves share out the token's K routes times the parts of the
// contraction; a part's sums of 16 columns go to LDS, and 16 threads add them,
// parts in order to a route's row, routes in k order to the token's: the
// additions of the kernels above and of combine_f32_kernel, without the pass
// through route_out.  Every token reads its own experts, and most columns of
// the second operand are empty.
constexpr int kW4TokenWaves = 16;

__global__ __launch_bounds__(kW4TokenWaves * kWave) void w4_fc2_token_kernel(W4Args p,
                                                                             const int* __restrict__ token_routes,
                                                                             int K, uint16_t* __restrict__ y) {
    __shared__ __attribute__((aligned(16))) float s_sum[kMaxK * kW4Parts][16];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int r16 = lane & 15, q = lane >> 4;
    const int col0 = blockIdx.x * 16;                   // ncols is a multiple of 16
    const int64_t t = blockIdx.y;
    const int steps = (p.Kdim + kW4Step - 1) / kW4Step, sbytes = p.Kdim / kGroup;
    for (int i = wave; i < K * kW4Parts; i += kW4TokenWaves) {
        const int slot = token_routes[t * K + i / kW4Parts], part = i % kW4Parts;
        int e = -1;                                     // device data: range-checked
        if (static_cast<unsigned>(slot) < static_cast<unsigned>(p.R)) e = p.expert_ids[slot / kBlockM];
        floatx4 acc[1] = {floatx4{0.0f, 0.0f, 0.0f, 0.0f}};
        if (static_cast<unsigned>(e) < static_cast<unsigned>(p.E)) {
            const int64_t base = static_cast<int64_t>(e) * p.wrows + col0;
            const __amdgpu_buffer_rsrc_t codes = buffer(p.codes + base * (p.Kdim / 2), 16u * (p.Kdim / 2));
            const __amdgpu_buffer_rsrc_t scales = buffer(p.scales + base * sbytes, 16u * sbytes);
            const __amdgpu_buffer_rsrc_t row = buffer(p.a + static_cast<int64_t>(slot) * p.Kdim, p.Kdim * 2u);
            for (int s = w4_part(steps, part); s < w4_part(steps, part + 1); ++s) {
                const bool live = s * kW4Step + q * 64 < p.Kdim;   // past the row's end: zeros
                u32x4 cw[2], xw[2][1][4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    cw[h] = __builtin_amdgcn_raw_buffer_load_b128(
                        codes, live ? r16 * (p.Kdim / 2) + s * (kW4Step / 2) + q * 32 + h * 16 : kOob, 0, 0);
                const uint32_t sc = __builtin_amdgcn_raw_buffer_load_b16(
                    scales, live ? r16 * sbytes + s * (kW4Step / kGroup) + q * 2 : kOob, 0, 0);
#pragma unroll
                for (int j = 0; j < 8; ++j)             // the route is the first of 16 columns, the others zeros
                    xw[j / 4][0][j % 4] = __builtin_amdgcn_raw_buffer_load_b128(
                        row, live && r16 == 0 ? s * (kW4Step * 2) + q * 128 + j * 16 : kOob, 0, 0);
                w4_piece<1>(cw[0], sc & 255u, xw[0], acc);
                w4_piece<1>(cw[1], sc >> 8, xw[1], acc);
            }
        }
        if (r16 == 0) *reinterpret_cast<floatx4*>(&s_sum[i][4 * q]) = acc[0];
    }
    __syncthreads();
    if (threadIdx.x < 16) {
        float v = 0.0f;
        for (int k = 0; k < K; ++k) {
            float r = s_sum[k * kW4Parts][threadIdx.x];
#pragma unroll
            for (int i = 1; i < kW4Parts; ++i) r += s_sum[k * kW4Parts + i][threadIdx.x];
            v += r;
        }
        y[t * p.ncols + col0 + threadIdx.x] = f32_to_bf16(v);
    }
}

// y[t] = bf16( sum over k, from +0.0 in k order, of the token's routes ).
// Workgroup (x, y): 1024 columns of token y, 4 a thread; the token's routes are
// uniform, so all K rows are on their way after one scalar load.
template <int KMAX>
__global__ __launch_bounds__(256) void combine_f32_kernel(const float* __restrict__ route_out,
                                                          const int* __restrict__ token_routes, int K, int H,
                                                          int R, uint16_t* __restrict__ y) {
    const int64_t t = blockIdx.y;
    const int col = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (col >= H) return;
    floatx4 v[KMAX];
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
        const int r = k < K ? token_routes[t * K + k] : -1;
        v[k] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        if (static_cast<unsigned>(r) < static_cast<unsigned>(R))   // device data is range-checked, never trusted
            v[k] = *reinterpret_cast<const floatx4*>(route_out + static_cast<int64_t>(r) * H + col);
    }
    floatx4 s = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < KMAX; ++k) s += v[k];
    uint2 o;
    o.x = pack_bf16x2(s[0], s[1]);
    o.y = pack_bf16x2(s[2], s[3]);
    *reinterpret_cast<uint2*>(y + t * H + col) = o;
}

template <int KMAX>
void launch_combine_f32(const float* ro, const int* tr, int N, int K, int H, int R, uint16_t* y, hipStream_t s) {
    combine_f32_kernel<KMAX><<<dim3((H + 1023) / 1024, N), 256, 0, s>>>(ro, tr, K, H, R, y);
}

// Layout blocks that can hold routes: at most one partly filled block per
// expert in use beside the full ones.
int w4_blocks(int64_t N, int32_t E, int32_t K, int64_t R) {
    const int64_t routes = N * K;
    return static_cast<int>(std::min<int64_t>(R, routes + (kBlockM - 1) * std::min<int64_t>(E, routes)) / kBlockM);
}

// Whether FC2 and the combine run in one launch, token by token.  An expert is
// read by every token that picks it, and a compute unit runs two workgroups of
// 16 waves at once: it pays while that is at most 24 MB of codes (12 us instead of
// 15.2 for one token of the 128-expert layer, 6 MB; 4 tokens, 24 MB 21.7 instead
// of 24.9; one of 64 experts of 7168 x 2048, 56 MB 51.9 against 49.3) and three
// workgroups a compute unit (768: 24 tokens of a 512-wide layer 8.9 instead of
// 9.0, 12 of 32 experts of 1024 x 768 16.3 instead of 16.4; 1024: 16 of them 18.0
// against 16.7, 8 of 8 experts of 2048 x 768 15.8 against 13.7), four where the
// codes are few (256 tokens of a 64-wide layer 7.6 instead of 8.9).
bool w4_by_token(int64_t N, int32_t H, int32_t I, int32_t K) {
    const int64_t codes = N * K * (static_cast<int64_t>(H) * I / 2), mb = 1 << 20;
    return N * H / 16 <= (codes <= 4 * mb ? 4 : 3) * device_cus() && codes <= 24 * mb;
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

template <bool FC1, int WT, int CTMAX, bool SALIGN>
void launch_split(const W4Args& a, dim3 grid, int steps, hipStream_t s) {
    constexpr int threads = kW4Waves * kWave;
    if constexpr (CTMAX == 1 && SALIGN) {
        if (steps >= 6) {
            w4_split_kernel<FC1, WT, CTMAX, SALIGN, true><<<grid, threads, 0, s>>>(a);
            return;
        }
    }
    w4_split_kernel<FC1, WT, CTMAX, SALIGN, false><<<grid, threads, 0, s>>>(a);
}

template <bool FC1, int CTMAX, bool SALIGN>
void launch_w4(const W4Args& a, int blocks, int64_t tiles, double mean, hipStream_t s) {
    const int steps = (a.Kdim + kW4Step - 1) / kW4Step;
    const bool inside = a.Kdim % kW4Step != 0, brief = inside && steps >= (SALIGN ? 3 : 2) && steps <= 4;
    int64_t rows64, stream;      // tiles from which on: 64-row workgroups, the streaming kernel
    if (CTMAX == 1) {
        rows64 = mean > 2 ? 500 : 640;
        stream = brief ? (FC1 ? 2000 : SALIGN ? 6000 : INT64_MAX) : mean > 4 ? 800 : mean > 2 ? 900 : 1100;
    } else {
        rows64 = steps > 2 ? 200 : 340;
        if (brief && !SALIGN) stream = mean > 24 ? 650 : 900;
        else stream = mean > 48 ? 300 : mean > 24 ? 350 : inside && steps <= 7 ? 650 : 480;
    }
    auto grid = [&](int cols) { return dim3((a.ncols + cols - 1) / cols, blocks); };
    if (tiles >= stream)
        w4_stream_kernel<FC1, 2, CTMAX, SALIGN><<<grid((FC1 ? 16 : 32) * kW4Waves), kW4Waves * kWave, 0, s>>>(a);
    else if (tiles >= rows64)
        launch_split<FC1, 4, CTMAX, SALIGN>(a, grid(FC1 ? 32 : 64), steps, s);
    else
        launch_split<FC1, 2, CTMAX, SALIGN>(a, grid(FC1 ? 16 : 32), steps, s);
}

// Which kernel: by the most tiles of 64 weight rows that the route list can
// ask for, counted as for 256 compute units (all of this device's; a partition
// of it has fewer), and the routes an expert has on average.  Over 508 sizes
// about the bounds the choice is 0.9% off the fastest of the three kernels on
// average, 14% at most.
//   * Few tiles: the split kernel with 32-row workgroups, for more of them (264
//     tiles 4.7 us against 5.0 with 64 rows).  With one or two routes an expert up
//     to 640 (one, 512 tiles of 8 steps 7.5 us against 8.5, 640 8.9 against 9.0,
//     1024 of 3 7.2 against 6.5), with more, whose operands they read more often,
//     up to 500 (4, 490 tiles of 4 steps 7.4 with either, 560 of 8 10.4 against
//     9.8).
//   * Many: the streaming kernel, which with more routes pays sooner: from 1100
//     (4 steps, one route: 960 tiles 8.5 us with either, 1216 8.7 against 10.0
//     split), 900 (4: 770 8.7 against 9.0, 910 8.9 against 11.1; of 28 steps 910
//     45 against 46, 1190, where its last round is short, 63 against 56) or 800
//     (8: 624 of 8 steps 10.4 with either, 858 of 4 8.8 against 9.5).
//   * It pays for a step that the contraction ends inside of, which counts with 2
//     to 4 steps and few rounds of workgroups.  FC1: 1260 tiles of 576 columns
//     10.0 us against 9.5 split, 2240 12.6 against 13.0, 8960 39 against 47, of 640
//     40 against 52.  FC2, whose float32 rows split writes sooner: 2240 tiles of
//     640 columns 12.8 against 12.1, 4480 20.9 against 21.2, 6160 29.7 against
//     30.8, 8960 40 against 43; where rows of scales are not whole words split
//     stays ahead with one route an expert (8192 of 832 35 against 31) and with 4
//     (8960 52.8 against 49.8), and with 8 is 3% behind (9984 58.0 against 56.5).
//   * Two 16-route tiles are held at once where experts have more than 8 routes on
//     average (10: FC1 46 us against 52, FC2 28 against 29; 8: 44.5 against 45.8
//     and 27.3 against 26.6; 3, of 28 steps: 178 against 170: the second tile's
//     registers cost a workgroup a compute unit).  The split kernel then reads
//     twice the operands, and its address units are the time: 64-row workgroups
//     from 200 tiles (4 steps: 154 6.0 us against 5.0 with 32 rows, 210 6.5 against
//     7.5), with one or two steps from 340 (286 4.5 against 4.2, 374 4.7 against
//     5.3).  Streaming from 480 (16 routes, 4 steps: 414 8.8 against 8.3 split, 506
//     9.0 with either, 782 9.7 against 11.5), 350 (32: 270 8.5 against 7.0, 390 8.9
//     against 9.7) or 300 (64: 230 8.7 against 7.2, 322 8.9 against 10.1); with 5 to
//     7 steps that end inside and up to 24 routes 650 (598 10.3 against 9.9, 782
//     11.5 against 12.1); with 2 to 4 of them and scales that are not whole words
//     900, with more routes 650 (16: 782 tiles of 576 columns 8.3 against 7.9).
template <bool FC1>
void dispatch_w4(const W4Args& a, int blocks, double mean, hipStream_t s) {
    const int64_t tiles = static_cast<int64_t>(blocks) * (a.ncols / (FC1 ? 32 : 64)) * 256 / device_cus();
    const bool salign = a.Kdim % 128 == 0;              // rows of scales are whole words
    if (mean > 8) salign ? launch_w4<FC1, 2, true>(a, blocks, tiles, mean, s) : launch_w4<FC1, 2, false>(a, blocks, tiles, mean, s);
    else salign ? launch_w4<FC1, 1, true>(a, blocks, tiles, mean, s) : launch_w4<FC1, 1, false>(a, blocks, tiles, mean, s);
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
        dispatch_w4<true>(a, blocks, mean, stream);
    }
    if (which & 2) {
        a.a = act; a.codes = w2_codes; a.scales = w2_scales;
        a.out = route_out; a.Kdim = I; a.ncols = H; a.wrows = H;
        if (which == 7 && w4_by_token(N, H, I, K)) {
            w4_fc2_token_kernel<<<dim3(H / 16, static_cast<unsigned>(N)), kW4TokenWaves * kWave, 0, stream>>>(
                a, token_routes, K, y);
            return launch_status();
        }
        dispatch_w4<false>(a, blocks, mean, stream);
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

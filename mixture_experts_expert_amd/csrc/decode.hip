// The whole MoE FFN layer for the few tokens of a decode step, in two kernels.
//
//   routing     top-K by logit, p = softmax over the K
//   act[t, k]   = bf16( silu(x_t Wg^T) * (x_t Wu^T) * p )        e = ids[t, k]
//   y[t]        = bf16( sum_k act[t, k] W2[e]^T + residual[t] )
//
// With a few rows an expert the weights' bytes are the time: each chosen
// expert is read once a block of its routes (the block for the mean of the batch),
// and everything else is kept out of the way of that stream.
//   * No route list in memory and no launches for it: every workgroup of the
//     first kernel routes all tokens itself (the first one writes ids and
//     probabilities out) and sorts the routes by expert in LDS; the last one hands
//     its lists on to the second kernel (sorted again there from the ids, 61 tokens
//     of 12 experts take 28.1 us instead of 26.5).  The probabilities are computed when the
//     first weights are on their way.
//   * A wave streams rows of weights, a line of 128 bytes of each at a time,
//     through a ring of its own in LDS: LDS DMA loads, whole lines, no barrier
//     and no registers held by loads on their way.  The routes' rows of the
//     other operand come the same way in the same step.
//   * The products are 16x16x32 bf16 MFMAs with 16 weight rows as the first
//     operand and up to 16 routes as the second.
//   * First kernel: a tile holds 8 gate rows and their 8 up rows, so that a
//     layer has many of them, and the SwiGLU is a lane exchange.
//   * Second kernel: a team of waves owns 8 (or 4) columns of y for all tokens
//     and walks all experts in use; a wave adds an expert's products to its sums
//     of those columns in LDS, and the waves' sums meet in order at the end.  No
//     atomics.
//
// A layer of 128 experts (8 a token, H 2048, I 768), three sets of weights in
// turn: one token 19.5 us a call (FC1 10, FC2 6.5: 3 of each before the first
// weights leave), 16 tokens 125 us (FC1 82, FC2 42: 6.2 TB/s over both), 64 tokens
// 202 us; 8 tokens of 64 experts of 7168 x 2048 533-560 us (6.6-6.9 TB/s; a plain
// read reaches 7.0).  Where a batch keeps to few experts they have several blocks:
// 16 tokens on the same 32, 16 and 8 of the 128 60, 49 and 38 us, where their weights
// once take 43, 22 and 11 (dropless form 80, 69, 66); 64 tokens 92, 80 and 70 (80, 69, 63).
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "gemm_common.h"
#include "span.h"
#include "topk.h"
#include "../../include/moe_block.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kDecodeMaxN = 64;
constexpr int kDecodeWaves = 8;          // of a workgroup
constexpr int kLine = 64;                // columns of a 128-byte line
constexpr int kCuLds = 160 * 1024;       // LDS of a compute unit, all of it used

struct DecodeArgs {
    const float* logits;         // [N, E]
    const uint16_t* a;           // first: x [N, H]; second: act [N*K, I]
    const uint16_t* w;           // [E, wrows, Kdim]
    const uint16_t* residual;    // second; may be null
    const int* n_live;           // may be null
    int* topk_ids;               // [N, K]
    float* topk_probs;           // first
    uint16_t* out;               // first: act [N*K, I]; second: y [N, H]
    int N, E, K, Kdim, ncols, wrows;
    int* lists;                  // the second kernel's: [0] blocks, then from [4] on the blocks and the routes
    int next_log2;               // first: log2 of the second kernel's routes a block
    int share;                   // waves that share an item or a tile: 1, 2, 4 or 8
    uint32_t per_token;          // ceil(2^16 / K): route r is token r * per_token >> 16, exact for r < 2048
    __device__ __forceinline__ int token(int route) const { return static_cast<int>(static_cast<uint32_t>(route) * per_token >> 16); }
};

// The batch's routes sorted by expert, in LDS.  A block is up to XR routes of
// one expert: expert | first route << 10 | routes << 22.
struct DecodeLists {
    int* at;                     // [E] counts, then each expert's next free route | its count << 16
    uint32_t* block;             // [blocks]
    uint16_t* route;             // [N*K] routes t*K + k, an expert's together
    int* total;                  // blocks, and whether some expert's routes are to be in order
};
__device__ __forceinline__ int block_expert(uint32_t b) { return static_cast<int>(b & 1023u); }
__device__ __forceinline__ int block_first(uint32_t b) { return static_cast<int>(b >> 10 & 4095u); }
__device__ __forceinline__ int block_routes(uint32_t b) { return static_cast<int>(b >> 22); }

// From the counts in `at` to blocks and each expert's first route (one wave).
// `whole`: the routes of an expert that no block divides, here or further on.
template <int XR>
__device__ __forceinline__ void list_blocks(const DecodeLists& l, int E, int whole, int lane) {
    int routes = 0, blocks = 0, split = 0;
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = e0 + lane, n = e < E ? l.at[e] : 0, nb = (n + XR - 1) / XR;
        const int inc = wave_inclusive_scan(n | nb << 16);     // both sums stay below 2^16
        const int first = routes + (inc & 0xFFFF) - n;
        int b = blocks + (inc >> 16) - nb;
        if (e < E) l.at[e] = first | n << 16;
        for (int i = 0; i < n; i += XR)
            l.block[b++] = static_cast<uint32_t>(e) | static_cast<uint32_t>(first + i) << 10 |
                           static_cast<uint32_t>(min(XR, n - i)) << 22;
        const int last = __builtin_amdgcn_readlane(inc, kWave - 1);
        routes += last & 0xFFFF;
        blocks += last >> 16;
        split |= __ballot(n > whole) != 0;
    }
    if (lane == 0) {
        l.total[0] = blocks;
        l.total[1] = split;
    }
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A barrier that leaves the wave's loads on their way.
__device__ __forceinline__ void meet() {
    wait_lds();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A wave's ring: steps of one tile of 16 weight rows and XL * 8 rows of the other
// operand, each row a line of 128 bytes, DEPTH deep.  A line is 8 pieces of 16
// bytes, piece c at place c ^ (row/2 % 8), so that an operand read (16 rows, one
// piece each) meets every bank once.
template <int XL, int DEPTH>
struct DecodeRing {
    static constexpr int LOADS = 2 + XL, BYTES = LOADS * 1024;
    uint32_t base;               // LDS address
    const uint8_t* mem;
    uint32_t woff[2], xoff[XL];  // of the first step
    i32x4 wsrc, xsrc;
    int put, take;

    __device__ __forceinline__ void init(uint8_t* m) {
        mem = m;
        base = lds_addr(m);
        put = take = 0;
        wsrc = xsrc = i32x4{0, 0, 0, kRsrcWord3};
        close();
    }
    // Nothing follows: further steps load nothing (but count like any other).
    __device__ __forceinline__ void close() {
        woff[0] = woff[1] = kOob;
#pragma unroll
        for (int i = 0; i < XL; ++i) xoff[i] = kOob;
    }
    // The lane's 16 bytes of a line, for the row it has in the step.
    static __device__ __forceinline__ uint32_t piece(int row) {
        return static_cast<uint32_t>(((lane_id() % 8) ^ (row / 2 % 8)) * 16);
    }
    // Issue a step, `at` bytes behind the first one; the place it goes to has been
    // read.  Lines that wlive(i) and xlive(i) deny (past a row's end) become zeros.
    template <class WLIVE, class XLIVE>
    __device__ __forceinline__ void issue(uint32_t at, WLIVE wlive, XLIVE xlive) {
        const uint32_t to = base + put * BYTES;
        wait_lds();
#pragma unroll
        for (int i = 0; i < 2; ++i) dma16<true>(wsrc, wlive(i) ? woff[i] + at : kOob, to + i * 1024);
#pragma unroll
        for (int i = 0; i < XL; ++i) dma16(xsrc, xlive(i) ? xoff[i] + at : kOob, to + (2 + i) * 1024);
        put = put + 1 == DEPTH ? 0 : put + 1;
    }
    // Multiply the oldest step, which has arrived once DEPTH - 1 are on their way.
    // Column r16 of tile c of the other operand is its row xrow(c).
    template <int CT, class XROW>
    __device__ __forceinline__ void multiply(floatx4 (&acc)[CT], XROW xrow) {
        wait_vmcnt<(DEPTH - 1) * LOADS>();
        const int lane = lane_id(), r16 = lane & 15, q = lane >> 4;
        const uint8_t* s = mem + take * BYTES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bf16x8 w = *reinterpret_cast<const bf16x8*>(s + r16 * 128 + (((h * 4 + q) ^ (r16 / 2 % 8)) << 4));
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int row = xrow(c);
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(s + 2048 + row * 128 + (((h * 4 + q) ^ (row / 2 % 8)) << 4));
                acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, acc[c], 0, 0, 0);
            }
        }
        take = take + 1 == DEPTH ? 0 : take + 1;
    }
};

// The largest and the smallest of a 16-lane row's values, in all its lanes, and
// the largest of a wave's.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, static_cast<uint32_t>(dpp<kDppXor1>(static_cast<int>(v))));
    v = max(v, static_cast<uint32_t>(dpp<kDppXor2>(static_cast<int>(v))));
    v = max(v, static_cast<uint32_t>(dpp<kDppHalfMirror>(static_cast<int>(v))));
    return max(v, static_cast<uint32_t>(dpp<kDppMirror>(static_cast<int>(v))));
}
__device__ __forceinline__ uint32_t wave_max_of(uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x111, 0xF, 0xF, false)));   // row_shr:1
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x112, 0xF, 0xF, false)));
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x114, 0xF, 0xF, false)));
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x118, 0xF, 0xF, false)));
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x142, 0xA, 0xF, false)));   // row_bcast:15
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x143, 0xC, 0xF, false)));   // row_bcast:31
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), kWave - 1));
}
__device__ __forceinline__ int row_min(int v) {
    v = min(v, dpp<kDppXor1>(v));
    v = min(v, dpp<kDppXor2>(v));
    v = min(v, dpp<kDppHalfMirror>(v));
    return min(v, dpp<kDppMirror>(v));
}

// Routing of all tokens by the whole workgroup: the routes' experts (-1 past the
// live tokens) and logits in LDS, the experts' counts in `at` (null: not wanted).
// A token has LANES lanes, PER logits each (expert j*LANES + lane).  Keys are
// topk_key's upper words (0: no expert, or picked), so the picks are
// topk_rounds', which takes more than 256 experts itself.  The kernel's
// probabilities repeat topk_prob's operations in its order, a lane a pick of
// several tokens.
//   * 16 lanes: a round finds the row's largest key and its lowest expert in eight
//     lane moves, for four tokens a wave (16 tokens of 128 experts 3.9 us from the
//     kernel's start, a wave a token 5.1; 61 of 12 experts 2.3 against 7.1).
//   * A wave, for no more tokens than waves: the largest key in six lane moves,
//     its lowest expert in the lanes' votes, two or four logits a lane instead of
//     eight or sixteen (one token of 128 experts 1.7 us against 3.9).
template <int LANES, int PER, int W>
__device__ __forceinline__ void decode_route(const DecodeArgs& p, int live, int* at, int* ids, float* logits) {
    constexpr bool KEYS32 = LANES * PER <= 256;
    const int g = threadIdx.x % LANES;
    for (int t = threadIdx.x / LANES; t < p.N; t += W * kWave / LANES) {
        int id[2] = {-1, -1};                           // picks g and, with 16 lanes, g + 16
        float logit[2] = {0.0f, 0.0f};
        if (t < live) {
            const float* row = p.logits + static_cast<int64_t>(t) * p.E;
            if constexpr (KEYS32) {
                uint32_t key[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    key[j] = j * LANES + g < p.E ? static_cast<uint32_t>(topk_key(row[j * LANES + g], 0) >> 32) : 0u;
                for (int k = 0; k < p.K; ++k) {
                    uint32_t m = key[0];
#pragma unroll
                    for (int j = 1; j < PER; ++j) m = max(m, key[j]);
                    int e = INT32_MAX;
                    if constexpr (LANES == 16) {
                        m = row_max(m);
#pragma unroll
                        for (int j = PER - 1; j >= 0; --j)
                            if (key[j] == m && j * LANES + g < p.E) e = j * LANES + g;
                        e = row_min(e);
                    } else {
                        m = wave_max_of(m);
#pragma unroll
                        for (int j = PER - 1; j >= 0; --j) {
                            const uint64_t has = __ballot(key[j] == m && j * LANES + g < p.E);
                            if (has) e = j * LANES + __builtin_ctzll(has);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (j * LANES + g == e) key[j] = 0u;
                    const float l = key_logit(static_cast<uint64_t>(m) << 32);
                    if (g == k % LANES) {
                        if (k < LANES) id[0] = e, logit[0] = l;
                        else id[1] = e, logit[1] = l;
                    }
                }
            } else {
                uint64_t key[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) key[j] = j * LANES + g < p.E ? topk_key(row[j * LANES + g], j * LANES + g) : 0ull;
                topk_rounds<LANES, PER>(key, p.K, g, id[0], logit[0]);
            }
        }
#pragma unroll
        for (int i = 0; i < (LANES == 16 ? 2 : 1); ++i) {
            const int k = g + i * 16;
            if (k < p.K) {
                const bool pick = t < live && static_cast<unsigned>(id[i]) < static_cast<unsigned>(p.E);
                const int r = t * p.K + k;
                ids[r] = pick ? id[i] : -1;
                logits[r] = logit[i];
                if (blockIdx.x == 0) p.topk_ids[r] = pick ? id[i] : -1;
                if (at && pick) atomicAdd(&at[id[i]], 1);
            }
        }
    }
}

// One token: its picks are the blocks, in their order.
__device__ __forceinline__ void list_one(const DecodeLists& l, int e, int lane) {
    const uint64_t there = __ballot(e >= 0);
    if (e >= 0) {
        const int i = __popcll(there & ((1ull << lane) - 1ull));
        l.block[i] = static_cast<uint32_t>(e) | static_cast<uint32_t>(i) << 10 | 1u << 22;
        l.route[i] = static_cast<uint16_t>(lane);
    }
    if (lane == 0) *l.total = __popcll(there);
}

// The routes of each expert together, by the whole workgroup, as they come.  The
// order among an expert's routes moves no result as long as they are one block
// (each is a column of its own).  Where some expert has several, the block decides
// which waves sum a route, so that the same inputs give the same bits only in one
// order, ascending: in every workgroup for the first kernel's blocks, and in the
// one that hands its lists on for the second one's, which are smaller.  `spare`: [N*K].
__device__ __forceinline__ void list_routes(const DecodeLists& l, const int* ids, uint16_t* spare, int routes) {
    const bool split = l.total[1] != 0;
    uint16_t* const to = split ? spare : l.route;
    for (int r = threadIdx.x; r < routes; r += blockDim.x) {
        const int e = ids[r];
        if (e >= 0) to[atomicAdd(&l.at[e], 1) & 0xFFFF] = static_cast<uint16_t>(r);
    }
    __syncthreads();
    if (!split) return;
    for (int r = threadIdx.x; r < routes; r += blockDim.x) {
        const int e = ids[r];
        if (e < 0) continue;
        const int n = l.at[e] >> 16, first = (l.at[e] & 0xFFFF) - n;
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += spare[first + i] < r;
        l.route[first + rank] = static_cast<uint16_t>(r);
    }
    __syncthreads();
}

// What the second kernel needs of the lists, by one workgroup: the same routes in
// blocks of 2^log2 (by the last wave, which has the least to do where there are
// few items), and their order.
__device__ __forceinline__ int most_blocks(int E, int routes, int log2) { return min(routes, E + (routes >> log2)); }
__device__ __forceinline__ void hand_on(const DecodeLists& l, const DecodeArgs& p, int routes, int wave, int lane) {
    uint32_t* const block = reinterpret_cast<uint32_t*>(p.lists + 4);
    uint16_t* const route = reinterpret_cast<uint16_t*>(block + most_blocks(p.E, routes, p.next_log2));
    for (int r = threadIdx.x; r < routes; r += blockDim.x) route[r] = l.route[r];
    if (wave != kDecodeWaves - 1) return;
    const int XR = 1 << p.next_log2;
    int blocks = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWave) {
        const int e = e0 + lane, at = e < p.E ? l.at[e] : 0, n = at >> 16, first = (at & 0xFFFF) - n;
        const int nb = (n + XR - 1) >> p.next_log2, inc = wave_inclusive_scan(nb);
        int b = blocks + inc - nb;
        for (int i = 0; i < n; i += XR)
            block[b++] = static_cast<uint32_t>(e) | static_cast<uint32_t>(first + i) << 10 | static_cast<uint32_t>(min(XR, n - i)) << 22;
        blocks += __builtin_amdgcn_readlane(inc, kWave - 1);
    }
    if (lane == 0) p.lists[0] = blocks;
}

// The lists as they were handed on.  They are device data: what lies outside the
// batch (nothing, unless the workspace was written to in between) becomes empty.
template <int XR>
__device__ __forceinline__ void take_lists(const DecodeLists& l, const DecodeArgs& p, int routes) {
    const int most = min(routes, p.E + routes / XR);
    const uint32_t* const block = reinterpret_cast<const uint32_t*>(p.lists + 4);
    const uint16_t* const route = reinterpret_cast<const uint16_t*>(block + most);
    for (int i = threadIdx.x; i < most; i += blockDim.x) {
        const uint32_t b = block[i];
        const bool good = block_expert(b) < p.E && block_routes(b) <= XR && block_first(b) + block_routes(b) <= routes;
        l.block[i] = good ? b : 0u;
    }
    for (int r = threadIdx.x; r < routes; r += blockDim.x) l.route[r] = static_cast<uint16_t>(min(static_cast<int>(route[r]), routes - 1));
    if (threadIdx.x == 0) *l.total = min(max(p.lists[0], 0), most);
    __syncthreads();
}

// Bytes of the lists in LDS, for a batch of `routes`.
__host__ __device__ constexpr int list_bytes(int E, int routes, int XR, bool first) {
    return 16 + (first ? E * 4 + routes * 4 : 0) + (routes < E + routes / XR ? routes : E + routes / XR) * 4 + routes * 2;
}

// A workgroup's waves in teams of p.share.  Unit u of a kernel's work (an item, a
// tile) is team u / G of workgroup u % G's, so that neighbouring workgroups are at
// neighbouring weights and every compute unit has work when there is little.
struct Teams {
    int size, member, first, stride;
    __device__ __forceinline__ Teams(int share, int wave) {
        size = share;
        member = wave & (share - 1);
        const int teams = kDecodeWaves / share, team = wave / share;
        first = team * static_cast<int>(gridDim.x);     // past this workgroup's own number
        stride = teams * static_cast<int>(gridDim.x);
    }
};

// ---------------------------------------------------------------- first kernel
// An item is a tile (8 gate rows and their 8 up rows) for a block of up to 8*XL
// routes.  A team's waves share its contraction; the first one adds the others'
// parts in order, while they go on with the next item.  A step is a line of the
// 16 rows and of the routes' tokens; items begin at different lines of theirs,
// since rows whose pitch is a large power of two put the same line of all rows on
// few memory channels.

template <int LANES, int PER, int XL, int DEPTH>
__global__ __launch_bounds__(kDecodeWaves * kWave) void decode_fc1_kernel(DecodeArgs p) {
    typedef DecodeRing<XL, DEPTH> Ring;
    constexpr int W = kDecodeWaves;
    constexpr int XR = 8 * XL, CT = XL > 1 ? XL / 2 : 1, RING = W * DEPTH * Ring::BYTES, PARTS = 2 * W * CT * 1024;
    static_assert(RING + PARTS < kCuLds, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kCuLds];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int routes = p.N * p.K;                       // <= 2048
    floatx4* const parts = reinterpret_cast<floatx4*>(smem + RING);    // [2][W][CT][64]
    DecodeLists l;
    l.total = reinterpret_cast<int*>(smem + RING + PARTS);
    l.at = l.total + 4;
    float* const probs = reinterpret_cast<float*>(l.at + p.E);
    l.block = reinterpret_cast<uint32_t*>(probs + routes);
    l.route = reinterpret_cast<uint16_t*>(l.block + min(routes, p.E + routes / XR));
    const bool one = p.N == 1, hands_on = !one && blockIdx.x == gridDim.x - 1;
    int* const ids = one ? l.at : reinterpret_cast<int*>(smem);        // (in the ring's place, which is not in use yet)
    const int live = p.n_live ? min(max(p.n_live[0], 0), p.N) : p.N;

    if (one) {
        if (wave == 0) {
            decode_route<LANES, PER, W>(p, live, nullptr, ids, probs);
            list_one(l, lane < p.K ? ids[lane] : -1, lane);
        }
        __syncthreads();
    } else {
        for (int e = threadIdx.x; e < p.E; e += W * kWave) l.at[e] = 0;
        __syncthreads();
        decode_route<LANES, PER, W>(p, live, l.at, ids, probs);
        __syncthreads();
        if (wave == 0) list_blocks<XR>(l, p.E, hands_on ? min(XR, 1 << p.next_log2) : XR, lane);
        __syncthreads();
        list_routes(l, ids, reinterpret_cast<uint16_t*>(ids + routes), routes);
    }

    const int tiles = p.ncols / 8, items = *l.total * tiles;           // < 2^22
    const Teams team(p.share, wave);
    const int lines = p.Kdim / kLine, lo = lines * team.member / team.size, n = lines * (team.member + 1) / team.size - lo;   // n >= 1
    Ring ring;
    ring.init(smem + wave * DEPTH * Ring::BYTES);
    ring.xsrc = make_rsrc(p.a, static_cast<uint32_t>(p.N) * p.Kdim * 2u);
    int item = team.first + static_cast<int>(blockIdx.x), k = 0, left = 0;   // what is issued next
    auto aim = [&]() {                                  // at the rows of `item`
        if (item >= items) {
            ring.close();
            return;
        }
        k = item * 5 % n;
        left = n;
        const uint32_t b = l.block[item / tiles];
        const int e = __builtin_amdgcn_readfirstlane(block_expert(b)), c0 = item % tiles * 8;
        const int64_t each = static_cast<int64_t>(p.wrows) * p.Kdim;
        ring.wsrc = make_rsrc(p.w + e * each, static_cast<uint32_t>(each * 2));
#pragma unroll
        for (int i = 0; i < 2; ++i)                     // rows 0-7 of the step are gate rows, 8-15 the up rows beside them
            ring.woff[i] = static_cast<uint32_t>((i ? p.ncols : 0) + c0 + lane / 8) * p.Kdim * 2u + Ring::piece(i * 8 + lane / 8);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int j = i * 8 + lane / 8;
            ring.xoff[i] = j < block_routes(b)
                ? static_cast<uint32_t>(p.token(l.route[block_first(b) + j])) * p.Kdim * 2u + Ring::piece(j) : kOob;
        }
    };
    auto issue = [&]() {
        ring.issue(item < items ? (lo + k) * 128 : 0, [](int) { return true; }, [](int) { return true; });
        if (item >= items) return;
        if (++k == n) k = 0;
        if (--left == 0) {
            item += team.stride;
            aim();
        }
    };
    aim();
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) issue();
    if (hands_on) hand_on(l, p, routes, wave, lane);    // (it has no more items than the others)
    // with the first loads on their way, probabilities from the logits: a wave takes
    // as many tokens as have their picks in its lanes, added in pick order
    const int fit = kWave / p.K;
    for (int t0 = wave * fit; t0 < p.N; t0 += W * fit) {
        const int r = t0 * p.K + lane;
        const bool there = lane < fit * p.K && r < routes;
        const int pick0 = p.token(lane) * p.K;          // the lane of the token's first pick
        const float logit = there ? probs[r] : 0.0f;
        const double e = exp(static_cast<double>(logit) - static_cast<double>(__shfl(logit, pick0)));
        double sum = 0.0;
        for (int k = 0; k < p.K; ++k) sum += __shfl(e, pick0 + k);
        if (there) {
            const float prob = t0 + p.token(lane) < live ? static_cast<float>(e / sum) : 0.0f;
            probs[r] = prob;
            if (blockIdx.x == 0) p.topk_probs[r] = prob;
        }
    }
    meet();                                             // the probabilities are there
    int turn = 0;
#pragma unroll 1
    for (int it0 = blockIdx.x; it0 < items; it0 += team.stride, turn ^= 1) {
        const int it = it0 + team.first;
        floatx4 acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        if (it < items) {
#pragma unroll 1
            for (int s = 0; s < n; ++s) {
                issue();
                ring.template multiply<CT>(acc, [&](int c) { return XL == 1 ? lane & 7 : c * 16 + (lane & 15); });
            }
        }
        if (team.size > 1) {
            floatx4* const mine = parts + (turn * W + wave) * CT * kWave + lane;
            if (team.member > 0) {
#pragma unroll
                for (int c = 0; c < CT; ++c) mine[c * kWave] = acc[c];
            }
            // A buffer is written again two items on, past the next item's meeting,
            // to which the first wave comes when it has read this one.
            meet();
            if (team.member > 0) continue;
            for (int m = 1; m < team.size; ++m) {
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[c] += mine[(m * CT + c) * kWave];
            }
        }
        if (it >= items) continue;
        // lane (j, q): gate rows 4q .. 4q+3 of route j for q < 2, the up rows beside them 32 lanes on
        const uint32_t b = l.block[it / tiles];
        const int c0 = it % tiles * 8;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            float u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __shfl_xor(acc[c][i], 32);
            const int j = c * 16 + (lane & 15);
            if (lane < 32 && (lane & 15) < min(XR, 16) && j < block_routes(b)) {
                const int route = l.route[block_first(b) + j];
                const float pr = probs[route];
                uint2 o;
                o.x = pack_bf16x2(silu(acc[c][0]) * u[0] * pr, silu(acc[c][1]) * u[1] * pr);
                o.y = pack_bf16x2(silu(acc[c][2]) * u[2] * pr, silu(acc[c][3]) * u[3] * pr);
                *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(route) * p.ncols + c0 + (lane >> 4) * 4) = o;
            }
        }
    }
    wait_vmcnt<0>();                                    // no load may land after the workgroup's LDS is given away
}

// ---------------------------------------------------------------- second kernel
// A tile is R columns of y.  A step is 16/R lines of each of its R weight rows, line
// after line as the 16 rows of the product, and the same lines of up to XR routes'
// activations as its columns, R a line: of the 16x16 products the RxR blocks on the
// diagonal are the lines', the others mean nothing.  (Tiles of 16 columns would be
// too few for the device: 128 of them in a layer of 2048 columns read 4.0 TB/s.)
// A team's waves share a tile's (block, step) pairs.

// 8-row loads of the routes' lines in a step, and its column tiles; with 8 rows and
// 4 routes half the columns repeat the other half's.
constexpr int fc2_loads(int R, int XR) { return XR * (16 / R) / 8; }
constexpr int fc2_tiles(int R, int XR) { return XR > R ? XR / R : 1; }

template <int R, int XR, int DEPTH>
__global__ __launch_bounds__(kDecodeWaves * kWave) void decode_fc2_kernel(DecodeArgs p) {
    constexpr int W = kDecodeWaves, XL = fc2_loads(R, XR), CT = fc2_tiles(R, XR), LINES = 16 / R;
    constexpr int COLS = XR < R ? XR : R;               // columns of a line
    typedef DecodeRing<XL, DEPTH> Ring;
    constexpr int RING = W * DEPTH * Ring::BYTES;
    static_assert(RING < kCuLds, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kCuLds];
    const int lane = lane_id(), r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int routes = p.N * p.K;
    float* const sums = reinterpret_cast<float*>(smem + RING);         // [waves][N][R]
    DecodeLists l;
    l.total = reinterpret_cast<int*>(sums + W * p.N * R);
    l.block = reinterpret_cast<uint32_t*>(l.total + 4);
    l.route = reinterpret_cast<uint16_t*>(l.block + min(routes, p.E + routes / XR));
    const int live = p.n_live ? min(max(p.n_live[0], 0), p.N) : p.N;
    const Teams team(p.share, wave);
    // what a tile's last lines add is loaded first
    constexpr int OUTS = kDecodeMaxN * R / kWave;
    const int out0 = team.member * kWave + lane, outs = team.size * kWave;
    const int tiles = p.ncols / R;
    float added[OUTS];
    auto load_added = [&](int tile) {
#pragma unroll
        for (int j = 0; j < OUTS; ++j) {
            const int i = out0 + j * outs;
            added[j] = p.residual && tile < tiles && i < live * R
                ? bf16_to_f32(p.residual[static_cast<int64_t>(i / R) * p.ncols + tile * R + i % R]) : 0.0f;
        }
    };
    load_added(team.first + static_cast<int>(blockIdx.x));
    if (p.N == 1) {
        if (wave == 0) {
            const int e = lane < p.K ? p.topk_ids[lane] : -1;          // device data: range-checked
            list_one(l, static_cast<unsigned>(e) < static_cast<unsigned>(p.E) ? e : -1, lane);
        }
        __syncthreads();
    } else {
        take_lists<XR>(l, p, routes);
    }

    const int lines = p.Kdim / kLine, steps = (lines + LINES - 1) / LINES, pairs = *l.total * steps;   // < 2^19
    const int lo = pairs * team.member / team.size, hi = pairs * (team.member + 1) / team.size;
    Ring ring;
    ring.init(smem + wave * DEPTH * Ring::BYTES);
    ring.xsrc = make_rsrc(p.a, static_cast<uint32_t>(routes) * p.Kdim * 2u);
    // the line, and the row or route, of the lane's row of load i
    auto w_line = [&](int i) { return (i * 8 + lane / 8) / R; };
    auto w_row = [&](int i) { return (i * 8 + lane / 8) % R; };
    auto x_line = [&](int i) { return (i * 8 + lane / 8) % (COLS * LINES) / COLS; };
    auto x_route = [&](int i) { return (i * 8 + lane / 8) / (COLS * LINES) * COLS + (i * 8 + lane / 8) % COLS; };
    const int block0 = lo / steps, k0 = lo - block0 * steps;
    int tile = lo < hi ? team.first + static_cast<int>(blockIdx.x) : tiles;
    int next = lo, block = block0, k = k0;                             // what is issued next
    auto aim = [&]() {
        if (tile >= tiles) {
            ring.close();
            return;
        }
        const uint32_t b = l.block[block];
        const int e = __builtin_amdgcn_readfirstlane(block_expert(b));
        const int64_t each = static_cast<int64_t>(p.wrows) * p.Kdim;
        ring.wsrc = make_rsrc(p.w + e * each, static_cast<uint32_t>(each * 2));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ring.woff[i] = static_cast<uint32_t>(tile * R + w_row(i)) * p.Kdim * 2u + w_line(i) * 128 + Ring::piece(i * 8 + lane / 8);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int j = x_route(i);
            ring.xoff[i] = j < block_routes(b)
                ? static_cast<uint32_t>(l.route[block_first(b) + j]) * p.Kdim * 2u + x_line(i) * 128 + Ring::piece(i * 8 + lane / 8)
                : kOob;
        }
    };
    auto issue = [&]() {
        const int rest = lines - k * LINES;             // lines from here on
        ring.issue(tile < tiles ? k * (128 * LINES) : 0, [&](int i) { return w_line(i) < rest; },
                   [&](int i) { return x_line(i) < rest; });
        if (tile >= tiles) return;
        ++k;
        if (++next == hi) {
            tile += team.stride;
            next = lo;
            block = block0;
            k = k0;
            aim();
        } else if (k == steps) {
            k = 0;
            ++block;
            aim();
        }
    };
    aim();
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) issue();
    float* const mine = sums + wave * p.N * R;
#pragma unroll 1
    for (int t0 = blockIdx.x; t0 < tiles; t0 += team.stride) {
        const int c0 = (t0 + team.first) * R;
        const bool there = t0 + team.first < tiles;
        for (int i = lane; i < p.N * R; i += kWave) mine[i] = 0.0f;
        int at = there ? lo : hi, b = block0, end = min(hi, (block0 + 1) * steps);
#pragma unroll 1
        while (at < hi) {
            floatx4 acc[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
            for (; at < end; ++at) {
                issue();
                ring.template multiply<CT>(acc, [&](int c) { return c * 16 + (COLS < R ? r16 / R * COLS + r16 % COLS : r16); });
            }
            const uint32_t entry = l.block[b];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                // The blocks of the diagonal: lane (q, r16) with r16 / R the line of its
                // rows 4q .. 4q+3.  A line on is R rows and R columns on: xor 40 with
                // two lines, 20 and 40 with four.
                floatx4 v = acc[c];
                if (R == 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], 20);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], 40);
                const int j = c * COLS + r16;
                if (q < R / 4 && r16 < COLS && j < block_routes(entry)) {     // a token has an expert once: lanes meet no one's sums
                    const int t = p.token(l.route[block_first(entry) + j]);
                    *reinterpret_cast<floatx4*>(mine + t * R + q * 4) += v;
                }
            }
            ++b;
            end = min(hi, end + steps);
        }
        if (team.size > 1) meet();
        else wait_lds();
        if (there) {
#pragma unroll
            for (int j = 0; j < OUTS; ++j) {
                const int i = out0 + j * outs;
                if (i >= live * R) break;
                float v = 0.0f;
                for (int m = 0; m < team.size; ++m) v += (mine - team.member * p.N * R)[m * p.N * R + i];
                p.out[static_cast<int64_t>(i / R) * p.ncols + c0 + i % R] = f32_to_bf16(v + added[j]);
            }
        }
        if (t0 + team.stride < tiles) {
            load_added(t0 + team.stride + team.first);
            if (team.size > 1) meet();                  // the sums are read
        }
    }
    wait_vmcnt<0>();
}

// Waves that share a unit of work of `length` steps, of which there are `units`
// (on average): as many as make the longest wave's time least.  A unit's end counts
// as half a step, with several waves, who meet, as two.  (Always eight against this
// rule: 2 tokens of 28 experts of 768 x 320 15.0 us against 13.9, 23 of 113 of 384 x
// 896 33 against 30, 28 of 5 of 2496 x 192 18.3 against 16.8; large layers gain 1%
// with eight: 16 tokens of 128 of 2048 x 768 124.9 against 125.9.)
int decode_share(double units, int length) {
    const int waves = device_cus() * kDecodeWaves;
    int best = 1;
    double least = 0.0;
    for (int share = 1; share <= kDecodeWaves && share <= length; share *= 2) {
        const double rounds = std::max(1.0, std::ceil(units * share / waves - 0.05));
        const double time = rounds * ((length + share - 1) / share + (share > 1 ? 2.0 : 0.5));
        if (share == 1 || time < least) {
            least = time;
            best = share;
        }
    }
    return best;
}

// Deep rings where the lists leave the room (LESS always does).
template <int LANES, int PER, int XL, int DEEP, int LESS>
void launch_fc1(const DecodeArgs& a, hipStream_t s) {
    constexpr int W = kDecodeWaves, XR = 8 * XL, PARTS = 2 * W * (XL > 1 ? XL / 2 : 1) * 1024;
    const int64_t most = std::min<int64_t>(a.N * a.K, a.E + a.N * a.K / XR) * (a.ncols / 8);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(most, device_cus()));
    if (W * DEEP * DecodeRing<XL, DEEP>::BYTES + PARTS + list_bytes(a.E, a.N * a.K, XR, true) <= kCuLds)
        decode_fc1_kernel<LANES, PER, XL, DEEP><<<grid, W * kWave, 0, s>>>(a);
    else
        decode_fc1_kernel<LANES, PER, XL, LESS><<<grid, W * kWave, 0, s>>>(a);
}

template <int LANES, int PER>
void launch_fc1(const DecodeArgs& a, double mean, hipStream_t s) {
    if (mean <= 2) launch_fc1<LANES, PER, 1, 4, 4>(a, s);
    else if (mean <= 8) launch_fc1<LANES, PER, 2, 4, 3>(a, s);
    else launch_fc1<LANES, PER, 4, 2, 2>(a, s);
}

template <int R, int XR, int DEEP, int LESS>
void launch_fc2(DecodeArgs a, double blocks, hipStream_t s) {
    constexpr int W = kDecodeWaves, LINES = 16 / R;
    const int lists = list_bytes(a.E, a.N * a.K, XR, false) + W * a.N * R * 4, tiles = a.ncols / R;
    const unsigned grid = static_cast<unsigned>(std::min(tiles, device_cus()));
    a.share = decode_share(tiles, std::max(1, static_cast<int>(blocks * ((a.Kdim / kLine + LINES - 1) / LINES))));
    if (W * DEEP * DecodeRing<fc2_loads(R, XR), DEEP>::BYTES + lists <= kCuLds)
        decode_fc2_kernel<R, XR, DEEP><<<grid, W * kWave, 0, s>>>(a);
    else
        decode_fc2_kernel<R, XR, LESS><<<grid, W * kWave, 0, s>>>(a);
}

int check_decode(int64_t N, int32_t H, int32_t I, int32_t E, int32_t K) {
    if (N < 0 || E < 1 || K < 1 || K > E) return MOE_ERR_INVALID_ARG;
    if (N > kDecodeMaxN || E > kMaxE || K > kMaxK) return MOE_ERR_UNSUPPORTED;
    return check_dims(H, I);
}

}  // namespace
}  // namespace moe

extern "C" int32_t moe_ffn_decode_max_tokens(void) { return moe::kDecodeMaxN; }

extern "C" size_t moe_ffn_decode_workspace_bytes(int64_t N, int32_t H, int32_t I, int32_t E, int32_t K) {
    if (moe::check_decode(N, H, I, E, K) != MOE_OK) return 0;
    const size_t routes = static_cast<size_t>(std::max<int64_t>(N, 1)) * K;
    return routes * I * 2 + (16 + routes * 6 + 15) / 16 * 16;          // (at most a block a route)
}

extern "C" int moe_ffn_decode(const float* logits, const uint16_t* x, const uint16_t* w1, const uint16_t* w2,
                              const uint16_t* residual, const int32_t* n_live, int64_t N, int32_t H, int32_t I,
                              int32_t E, int32_t K, int32_t* topk_ids, float* topk_probs, void* workspace,
                              size_t workspace_bytes, uint16_t* y, hipStream_t stream) {
    using namespace moe;
    const int st = check_decode(N, H, I, E, K);
    if (st != MOE_OK) return st;
    if (N == 0) return MOE_OK;
    const void* const needed[] = {logits, x, w1, w2, topk_ids, topk_probs, workspace, y};
    for (const void* q : needed)
        if (!q) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_ffn_decode_workspace_bytes(N, H, I, E, K)) return MOE_ERR_INVALID_ARG;
    for (const void* q : needed)
        if (!aligned16(q)) return MOE_ERR_MISALIGNED;
    if (!aligned16(residual) || (reinterpret_cast<uintptr_t>(n_live) & 3u)) return MOE_ERR_MISALIGNED;
    const size_t routes = static_cast<size_t>(N) * K, matrix = static_cast<size_t>(E) * H * I * 2;
    const Span sl{logits, static_cast<size_t>(N) * E * 4}, sx{x, static_cast<size_t>(N) * H * 2}, s1{w1, 2 * matrix}, s2{w2, matrix},
        sr{residual, sx.bytes}, sn{n_live, 4}, si{topk_ids, routes * 4}, sp{topk_probs, routes * 4},
        sw{workspace, moe_ffn_decode_workspace_bytes(N, H, I, E, K)}, sy{y, sx.bytes};
    if (!sy.apart_or_one_of({sx, sr}) || !sy.apart({sl, s1, s2, sn, si, sp, sw}) || !si.apart({sl, sx, s1, s2, sr, sn, sp, sw}) ||
        !sp.apart({sl, sx, s1, s2, sr, sn, sw}) || !sw.apart({sl, sx, s1, s2, sr, sn}))
        return MOE_ERR_INVALID_ARG;
    const double mean = static_cast<double>(N) * K / E;
    DecodeArgs a{};
    a.logits = logits; a.a = x; a.w = w1; a.n_live = n_live; a.topk_ids = topk_ids; a.topk_probs = topk_probs;
    a.out = static_cast<uint16_t*>(workspace);
    a.N = static_cast<int>(N); a.E = E; a.K = K; a.Kdim = H; a.ncols = I; a.wrows = 2 * I;
    a.per_token = (65536u + K - 1) / K;
    // experts that some token picks, on average, and blocks of up to XR of their routes
    const double used = E * (1.0 - std::pow(1.0 - static_cast<double>(K) / E, static_cast<double>(N)));
    const bool narrow = H / 8 * 8 < 5 * device_cus(), slim = mean <= 8 && H / 4 <= device_cus();
    const int xr1 = mean <= 2 ? 8 : mean <= 8 ? 16 : 32, xr2 = mean <= 1 ? 4 : mean <= 3 || slim ? 8 : 16;
    const double blocks1 = used + N * K / (xr1 * 2.0) * (mean > 8), blocks2 = used + N * K / (xr2 * 2.0) * (mean > xr2 / 2);
    a.share = decode_share(blocks1 * (I / 8), H / kLine);
    a.lists = reinterpret_cast<int*>(static_cast<uint16_t*>(workspace) + N * K * I);
    a.next_log2 = xr2 == 4 ? 2 : xr2 == 8 ? 3 : 4;
    const bool few = N <= kDecodeWaves;
    if (E <= 16) launch_fc1<16, 1>(a, mean, stream);
    else if (E <= 64) few ? launch_fc1<64, 1>(a, mean, stream) : launch_fc1<16, 4>(a, mean, stream);
    else if (E <= 128) few ? launch_fc1<64, 2>(a, mean, stream) : launch_fc1<16, 8>(a, mean, stream);
    else if (E <= 256) few ? launch_fc1<64, 4>(a, mean, stream) : launch_fc1<16, 16>(a, mean, stream);
    else launch_fc1<64, 16>(a, mean, stream);
    a.a = static_cast<const uint16_t*>(workspace); a.w = w2; a.residual = residual; a.out = y;
    a.Kdim = I; a.ncols = H; a.wrows = H;
    // Tiles of 4 columns where those of 8 are few, up to 5 for 8 compute units (128 of
    // them: 16 tokens of 64 experts of 1024 x 1024 65.7 us against 71, 48: 23 of 113 of
    // 384 x 896 29.7 against 32.8; 192: 2 of 32 of 1536 x 1536 26.5 against 25.9, 232: 41
    // of 26 of 1856 x 384 30.6 against 26.4).
    // With more than 3 routes an expert, blocks of 8 for 4 columns instead of 16 for 8,
    // where a compute unit has a tile at most and experts up to 8 routes (61 tokens of 61
    // experts of 256 x 704, 6 each, 41.6 us against 48.7, 9 of 22 of 512 x 1088 28.3 against
    // 32.9, 20 of 8 of 1024 x 1024 18.7 against 19.7; 27 routes of 1024 x 448 28.4 against 26.2,
    // 11 of 960 x 576 20.1 against 18.3).
    if (mean <= 1) narrow ? launch_fc2<4, 4, 4, 4>(a, blocks2, stream) : launch_fc2<8, 4, 4, 4>(a, blocks2, stream);
    else if (mean <= 3) narrow ? launch_fc2<4, 8, 3, 2>(a, blocks2, stream) : launch_fc2<8, 8, 4, 3>(a, blocks2, stream);
    else slim ? launch_fc2<4, 8, 3, 2>(a, blocks2, stream) : launch_fc2<8, 16, 2, 2>(a, blocks2, stream);
    return launch_status();
}

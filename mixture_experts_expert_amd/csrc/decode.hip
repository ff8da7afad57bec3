// The whole MoE FFN layer for the few tokens of a decode step, in two kernels.
//
//   routing     top-K by logit, p = softmax over the K
//   act[t, k]   = bf16( silu(x_t Wg^T) * (x_t Wu^T) * p )        e = ids[t, k]
//   y[t]        = bf16( sum_k act[t, k] W2[e]^T + residual[t] )
//
// With a few rows an expert the weights' bytes are the time: each chosen
// expert is read once, and everything else is kept out of the way of that
// stream.
//   * No route list in memory and no launches for it: every workgroup of the
//     first kernel routes all tokens itself (the first one writes ids and
//     probabilities out) and sorts the routes by expert in LDS, the second one
//     sorts them again from the ids.
//   * A wave streams rows of weights in 64-column steps through a ring of its
//     own in LDS: LDS DMA loads, whole 128-byte lines, no barrier and no
//     registers held by loads on their way.  The routes' rows of the other
//     operand come the same way in the same step.
//   * The products are 16x16x32 bf16 MFMAs with 16 weight rows as the first
//     operand and up to 16 routes as the second.
//   * First kernel: a tile holds 8 gate rows and their 8 up rows, so that a
//     layer has many of them; the waves of a workgroup share its contraction
//     and add their parts in order.
//   * Second kernel: a workgroup owns 16 columns of y for all tokens and walks
//     all experts in use, its waves sharing (expert, step) pairs evenly; a wave
//     adds an expert's products to its sums of those columns in LDS, and the
//     waves' sums meet in order at the end.  No atomics.
#include <algorithm>
#include <initializer_list>

#include "gemm_common.h"
#include "topk.h"
#include "../../include/moe_block.h"

namespace moe {
namespace {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kDecodeMaxN = 64;
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
    uint32_t per_token;          // ceil(2^16 / K): route r is token r * per_token >> 16, exact for r < 2048
    __device__ __forceinline__ int token(int route) const { return static_cast<int>(static_cast<uint32_t>(route) * per_token >> 16); }
};

// The batch's routes sorted by expert, in LDS.  A block is up to XR routes of
// one expert: expert | first route << 10 | routes << 22.
struct DecodeLists {
    int* at;                     // [E] counts, then each expert's next free route | its count << 16
    uint32_t* block;             // [blocks]
    uint16_t* route;             // [N*K] routes t*K + k, an expert's together
    int* total;                  // blocks, and whether an expert has several
};
__device__ __forceinline__ int block_expert(uint32_t b) { return static_cast<int>(b & 1023u); }
__device__ __forceinline__ int block_first(uint32_t b) { return static_cast<int>(b >> 10 & 4095u); }
__device__ __forceinline__ int block_routes(uint32_t b) { return static_cast<int>(b >> 22); }

// From the counts in `at` to blocks and each expert's first route (one wave).
template <int XR>
__device__ __forceinline__ void list_blocks(const DecodeLists& l, int E, int lane) {
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
        split |= __ballot(nb > 1) != 0;
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
    // read.  What `w1` and `x1` name (a row's second line) is left out past its end.
    template <class XLIVE>
    __device__ __forceinline__ void issue(uint32_t at, bool w1, XLIVE x1) {
        const uint32_t to = base + put * BYTES;
        wait_lds();
        dma16<true>(wsrc, woff[0] + at, to);
        dma16<true>(wsrc, w1 ? woff[1] + at : kOob, to + 1024);
#pragma unroll
        for (int i = 0; i < XL; ++i) dma16(xsrc, x1(i) ? xoff[i] + at : kOob, to + (2 + i) * 1024);
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
// topk_rounds', which takes more than 256 experts itself.
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

// The routes of each expert together, by the whole workgroup.  The order among
// an expert's routes moves no result as long as they are one block (each is a
// column of its own); of several blocks every workgroup has to have the same,
// and then the routes are put in order.  `spare`: [N*K].
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

// Bytes of the lists in LDS, for a batch of `routes`.
__host__ __device__ constexpr int list_bytes(int E, int routes, int XR, bool probs) {
    return 16 + E * 4 + (probs ? routes * 4 : 0) + (routes < E + routes / XR ? routes : E + routes / XR) * 4 + routes * 2;
}

// ---------------------------------------------------------------- first kernel
// A step is a line of the 8 gate rows and the 8 up rows of a tile, and of up to
// 8*XL routes' tokens.  Workgroups take (block, tile) items in turn, tiles of one
// block behind each other.  (A run of items for each, so that it reads front to
// back, leaves the slowest one 9% behind: a wide layer's 2.5 GB 372 us, 347 in
// turn.)

constexpr int kFc1Waves = 8;
template <int LANES, int PER, int XL, int DEPTH>
__global__ __launch_bounds__(kFc1Waves * kWave) void decode_fc1_kernel(DecodeArgs p) {
    typedef DecodeRing<XL, DEPTH> Ring;
    constexpr int W = kFc1Waves;
    constexpr int XR = 8 * XL, CT = XL > 1 ? XL / 2 : 1, RING = W * DEPTH * Ring::BYTES, PARTS = W * CT * 1024;
    static_assert(RING + PARTS < kCuLds, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kCuLds];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int routes = p.N * p.K;                       // <= 2048
    floatx4* const parts = reinterpret_cast<floatx4*>(smem + RING);
    DecodeLists l;
    l.total = reinterpret_cast<int*>(smem + RING + PARTS);
    l.at = l.total + 4;
    float* const probs = reinterpret_cast<float*>(l.at + p.E);
    l.block = reinterpret_cast<uint32_t*>(probs + routes);
    l.route = reinterpret_cast<uint16_t*>(l.block + min(routes, p.E + routes / XR));
    const bool one = p.N == 1;
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
        if (wave == 0) list_blocks<XR>(l, p.E, lane);
        __syncthreads();
        list_routes(l, ids, reinterpret_cast<uint16_t*>(ids + routes), routes);
    }

    const int tiles = p.ncols / 8, items = *l.total * tiles;           // < 2^22
    const int steps = p.Kdim / kLine, lo = steps * wave / W, hi = steps * (wave + 1) / W;
    Ring ring;
    ring.init(smem + wave * DEPTH * Ring::BYTES);
    ring.xsrc = make_rsrc(p.a, static_cast<uint32_t>(p.N) * p.Kdim * 2u);
    int item = lo < hi ? static_cast<int>(blockIdx.x) : items, k = lo;     // what is issued next
    auto aim = [&]() {                                  // at the rows of `item`
        if (item >= items) {
            ring.close();
            return;
        }
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
        ring.issue(item < items ? k * 128 : 0, true, [](int) { return true; });
        if (item < items && ++k == hi) {
            k = lo;
            item += gridDim.x;
            aim();
        }
    };
    aim();
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) issue();
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
#pragma unroll 1
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        floatx4 acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int s = lo; s < hi; ++s) {
            issue();
            ring.template multiply<CT>(acc, [&](int c) { return XL == 1 ? lane & 7 : c * 16 + (lane & 15); });
        }
        meet();                                         // the last item's parts are read
#pragma unroll
        for (int c = 0; c < CT; ++c) parts[(wave * CT + c) * kWave + lane] = acc[c];
        meet();
        const uint32_t b = l.block[it / tiles];
        const int n = block_routes(b), c0 = it % tiles * 8;
        for (int i = threadIdx.x; i < n * 8; i += W * kWave) {
            const int j = i / 8, r = i % 8;
            // gate row r of the tile is element r % 4 of lane (j % 16, r / 4), its up row 8 rows below
            const float* at = reinterpret_cast<const float*>(parts + j / 16 * kWave + r / 4 * 16 + j % 16) + r % 4;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                g += at[w * CT * kWave * 4];
                u += at[w * CT * kWave * 4 + 2 * 16 * 4];
            }
            const int route = l.route[block_first(b) + j];
            p.out[static_cast<int64_t>(route) * p.ncols + c0 + r] = f32_to_bf16(silu(g) * u * probs[route]);
        }
    }
    wait_vmcnt<0>();                                    // no load may land after the workgroup's LDS is given away
}

// ---------------------------------------------------------------- second kernel
// A workgroup owns 8 columns of y.  A step is two lines of each of its 8 weight
// rows, the second as rows 8-15 of the tile, and two lines of up to XR routes'
// activations, the second as columns 8-15: of the 16x16 products the two 8x8
// blocks on the diagonal are the two lines', the others mean nothing.  (Tiles of
// 16 rows would be too few for the device: 128 of them in a layer of 2048
// columns read 4.0 TB/s.)

template <int W, int XR, int DEPTH>
__global__ __launch_bounds__(W * kWave) void decode_fc2_kernel(DecodeArgs p) {
    constexpr int XL = XR / 4, CT = XR > 8 ? XR / 8 : 1;
    typedef DecodeRing<XL, DEPTH> Ring;
    constexpr int RING = W * DEPTH * Ring::BYTES;
    static_assert(RING < kCuLds, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kCuLds];
    const int lane = lane_id(), r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int routes = p.N * p.K;
    float* const sums = reinterpret_cast<float*>(smem + RING);         // [waves][N][8]
    DecodeLists l;
    l.total = reinterpret_cast<int*>(sums + W * p.N * 8);
    l.at = l.total + 4;
    l.block = reinterpret_cast<uint32_t*>(l.at + p.E);
    l.route = reinterpret_cast<uint16_t*>(l.block + min(routes, p.E + routes / XR));
    int* const ids = reinterpret_cast<int*>(smem);                     // in the ring's place

    const int live = p.n_live ? min(max(p.n_live[0], 0), p.N) : p.N;
    // what the last lines add, loaded first: a thread has at most kDecodeMaxN * 8 / threads of them
    constexpr int OUTS = (kDecodeMaxN * 8 + W * kWave - 1) / (W * kWave);
    float out[OUTS];
#pragma unroll
    for (int j = 0; j < OUTS; ++j) {
        const int i = static_cast<int>(threadIdx.x) + j * W * kWave;
        out[j] = p.residual && i < live * 8
            ? bf16_to_f32(p.residual[static_cast<int64_t>(i / 8) * p.ncols + blockIdx.x * 8 + i % 8]) : 0.0f;
    }
    for (int i = threadIdx.x; i < W * p.N * 8; i += W * kWave) sums[i] = 0.0f;
    if (p.N == 1) {
        if (wave == 0) {
            const int e = lane < p.K ? p.topk_ids[lane] : -1;          // device data: range-checked
            list_one(l, static_cast<unsigned>(e) < static_cast<unsigned>(p.E) ? e : -1, lane);
        }
        __syncthreads();
    } else {
        for (int e = threadIdx.x; e < p.E; e += W * kWave) l.at[e] = 0;
        __syncthreads();
        for (int r = threadIdx.x; r < routes; r += W * kWave) {
            const int e = p.topk_ids[r];
            const bool pick = static_cast<unsigned>(e) < static_cast<unsigned>(p.E);
            ids[r] = pick ? e : -1;
            if (pick) atomicAdd(&l.at[e], 1);
        }
        __syncthreads();
        if (wave == 0) list_blocks<XR>(l, p.E, lane);
        __syncthreads();
        list_routes(l, ids, reinterpret_cast<uint16_t*>(ids + routes), routes);
    }

    const int c0 = blockIdx.x * 8, lines = p.Kdim / kLine, steps = (lines + 1) / 2, pairs = *l.total * steps;
    const int lo = static_cast<int>(static_cast<int64_t>(pairs) * wave / W);
    const int hi = static_cast<int>(static_cast<int64_t>(pairs) * (wave + 1) / W);
    Ring ring;
    ring.init(smem + wave * DEPTH * Ring::BYTES);
    ring.xsrc = make_rsrc(p.a, static_cast<uint32_t>(routes) * p.Kdim * 2u);
    // the line and the route of the lane's row of load i: rows 0-7 of 16 are the first line's, of 8 rows 0-3
    auto x_line = [&](int i) { return XR == 4 ? lane / 32 : i & 1; };
    auto x_route = [&](int i) { return XR == 4 ? lane / 8 % 4 : i / 2 * 8 + lane / 8; };
    int next = lo, block = lo / steps, k = lo % steps;                 // what is issued next
    auto aim = [&]() {
        if (next >= hi) {
            ring.close();
            return;
        }
        const uint32_t b = l.block[block];
        const int e = __builtin_amdgcn_readfirstlane(block_expert(b));
        const int64_t each = static_cast<int64_t>(p.wrows) * p.Kdim;
        ring.wsrc = make_rsrc(p.w + e * each, static_cast<uint32_t>(each * 2));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ring.woff[i] = static_cast<uint32_t>(c0 + lane / 8) * p.Kdim * 2u + i * 128 + Ring::piece(i * 8 + lane / 8);
#pragma unroll
        for (int i = 0; i < XL; ++i) {
            const int j = x_route(i);
            ring.xoff[i] = j < block_routes(b)
                ? static_cast<uint32_t>(l.route[block_first(b) + j]) * p.Kdim * 2u + x_line(i) * 128 + Ring::piece(i * 8 + lane / 8)
                : kOob;
        }
    };
    auto issue = [&]() {
        const bool both = 2 * k + 1 < lines;
        ring.issue(next < hi ? k * 256 : 0, both, [&](int i) { return both || x_line(i) == 0; });
        if (next >= hi) return;
        ++next;
        if (++k == steps) {
            k = 0;
            ++block;
        }
        if (k == 0 || next == hi) aim();
    };
    aim();
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) issue();
    float* const mine = sums + wave * p.N * 8;
    int at = lo;
#pragma unroll 1
    while (at < hi) {
        const int b = at / steps, end = min(hi, (b + 1) * steps);
        floatx4 acc[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (; at < end; ++at) {
            issue();
            ring.template multiply<CT>(acc, [&](int c) { return XR == 4 ? (r16 >> 3) * 4 + (r16 & 3) : c * 16 + r16; });
        }
        const uint32_t entry = l.block[b];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            floatx4 v;                                  // the second line's block is 8 rows and 8 columns on
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = acc[c][j] + __shfl_xor(acc[c][j], 40);
            const int j = c * 8 + r16;
            if (q < 2 && r16 < min(XR, 8) && j < block_routes(entry)) {   // a token has an expert once: lanes meet no one's sums
                const int t = p.token(l.route[block_first(entry) + j]);
                *reinterpret_cast<floatx4*>(mine + t * 8 + q * 4) += v;
            }
        }
    }
    wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OUTS; ++j) {
        const int i = static_cast<int>(threadIdx.x) + j * W * kWave;
        if (i >= live * 8) break;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += sums[w * p.N * 8 + i];
        p.out[static_cast<int64_t>(i / 8) * p.ncols + c0 + i % 8] = f32_to_bf16(v + out[j]);
    }
}

// Deep rings where the lists leave the room (LESS always does).
template <int LANES, int PER, int XL, int DEEP, int LESS>
void launch_fc1(const DecodeArgs& a, hipStream_t s) {
    constexpr int W = kFc1Waves, XR = 8 * XL, PARTS = W * (XL > 1 ? XL / 2 : 1) * 1024;
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

template <int W, int XR, int DEEP, int LESS>
void launch_fc2(const DecodeArgs& a, hipStream_t s) {
    const int lists = list_bytes(a.E, a.N * a.K, XR, false) + W * a.N * 32;
    const unsigned grid = static_cast<unsigned>(a.ncols / 8);
    if (W * DEEP * DecodeRing<XR / 4, DEEP>::BYTES + lists <= kCuLds)
        decode_fc2_kernel<W, XR, DEEP><<<grid, W * kWave, 0, s>>>(a);
    else
        decode_fc2_kernel<W, XR, LESS><<<grid, W * kWave, 0, s>>>(a);
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
    return static_cast<size_t>(std::max<int64_t>(N, 1)) * K * I * 2;
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
    const double mean = static_cast<double>(N) * K / E;
    DecodeArgs a{};
    a.logits = logits; a.a = x; a.w = w1; a.n_live = n_live; a.topk_ids = topk_ids; a.topk_probs = topk_probs;
    a.out = static_cast<uint16_t*>(workspace);
    a.N = static_cast<int>(N); a.E = E; a.K = K; a.Kdim = H; a.ncols = I; a.wrows = 2 * I;
    a.per_token = (65536u + K - 1) / K;
    const bool few = N <= kFc1Waves;
    if (E <= 16) launch_fc1<16, 1>(a, mean, stream);
    else if (E <= 64) few ? launch_fc1<64, 1>(a, mean, stream) : launch_fc1<16, 4>(a, mean, stream);
    else if (E <= 128) few ? launch_fc1<64, 2>(a, mean, stream) : launch_fc1<16, 8>(a, mean, stream);
    else if (E <= 256) few ? launch_fc1<64, 4>(a, mean, stream) : launch_fc1<16, 16>(a, mean, stream);
    else launch_fc1<64, 16>(a, mean, stream);
    a.a = static_cast<const uint16_t*>(workspace); a.w = w2; a.residual = residual; a.out = y;
    a.Kdim = I; a.ncols = H; a.wrows = H;
    if (mean <= 1) launch_fc2<8, 4, 4, 4>(a, stream);
    else if (mean <= 3) launch_fc2<8, 8, 4, 3>(a, stream);
    else launch_fc2<8, 16, 2, 2>(a, stream);
    return launch_status();
}

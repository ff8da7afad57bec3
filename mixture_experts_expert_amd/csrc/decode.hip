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
constexpr int kDecodeWaves = 8;
constexpr int kDecodeThreads = kDecodeWaves * kWave;
constexpr int kDecodeStep = 64;          // columns of a step: one 128-byte line a row
constexpr int kDecodeLds = 160 * 1024;   // one workgroup a compute unit

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

// A wave's ring: steps of T tiles of 16 weight rows and 8*XT rows of the other
// operand, DEPTH deep.  A row's 128 bytes are 8 pieces of 16, piece c at place
// c ^ (row/2 % 8), so that an operand read (16 rows, one piece each) meets
// every bank once.
template <int T, int XT, int DEPTH>
struct DecodeRing {
    static constexpr int LOADS = 2 * T + XT, BYTES = LOADS * 1024, XR = 8 * XT, CT = XT > 1 ? XT / 2 : 1;
    uint32_t base;               // LDS address
    const uint8_t* mem;
    uint32_t woff[2 * T], xoff[XT];
    i32x4 wsrc, xsrc;
    int put, take;

    __device__ __forceinline__ void init(uint8_t* m) {
        mem = m;
        base = lds_addr(m);
        put = take = 0;
        wsrc = xsrc = i32x4{0, 0, 0, kRsrcWord3};
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) woff[i] = kOob;
#pragma unroll
        for (int i = 0; i < XT; ++i) xoff[i] = kOob;
    }
    // Nothing follows: further steps load nothing (but count like any other).
    __device__ __forceinline__ void close() {
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) woff[i] = kOob;
#pragma unroll
        for (int i = 0; i < XT; ++i) xoff[i] = kOob;
    }
    // The lane's 16 bytes of row `row` of a tile's 16 (bytes within the step's line).
    static __device__ __forceinline__ uint32_t piece(int row) {
        return static_cast<uint32_t>(((lane_id() % 8) ^ (row / 2 % 8)) * 16);
    }
    // Issue step k of the current rows.  The place it goes to has been read.
    __device__ __forceinline__ void issue(int k) {
        const uint32_t at = base + put * BYTES;
        wait_lds();
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) dma16<true>(wsrc, woff[i] + k * 128, at + i * 1024);
#pragma unroll
        for (int i = 0; i < XT; ++i) dma16(xsrc, xoff[i] + k * 128, at + (2 * T + i) * 1024);
        put = put + 1 == DEPTH ? 0 : put + 1;
    }
    // Multiply the oldest step, which has arrived once DEPTH - 1 are on their way.
    __device__ __forceinline__ void multiply(floatx4 (&acc)[T][CT]) {
        wait_vmcnt<(DEPTH - 1) * LOADS>();
        const int lane = lane_id(), r16 = lane & 15, q = lane >> 4;
        const uint8_t* s = mem + take * BYTES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 x[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int row = c * 16 + (XT == 1 ? r16 & 7 : r16);
                x[c] = *reinterpret_cast<const bf16x8*>(s + 2 * T * 1024 + row * 128 + (((h * 4 + q) ^ (row / 2 % 8)) << 4));
            }
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const bf16x8 w = *reinterpret_cast<const bf16x8*>(s + t * 2048 + r16 * 128 + (((h * 4 + q) ^ (r16 / 2 % 8)) << 4));
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[c], acc[t][c], 0, 0, 0);
            }
        }
        take = take + 1 == DEPTH ? 0 : take + 1;
    }
};

// Routing of all tokens by the whole workgroup: ids and probabilities of the
// routes in LDS (id -1 past the live ones), the experts' counts in `at`.
template <int LPT, int VPL>
__device__ __forceinline__ void decode_route(const DecodeArgs& p, int* at, int* ids, float* probs, bool write) {
    const int g = threadIdx.x % LPT, live = p.n_live ? min(max(p.n_live[0], 0), p.N) : p.N;
    for (int t = threadIdx.x / LPT; t < p.N; t += kDecodeThreads / LPT) {
        const float* row = p.logits + static_cast<int64_t>(t < live ? t : 0) * p.E;
        uint64_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = j * LPT + g;
            key[j] = t < live && e < p.E ? topk_key(row[e], e) : 0ull;
        }
        int id = 0;
        float logit = 0.0f;
        topk_rounds<LPT, VPL>(key, p.K, g, id, logit);
        const float prob = topk_prob<LPT>(logit, p.K, g);
        if (g < p.K) {
            const bool pick = t < live && static_cast<unsigned>(id) < static_cast<unsigned>(p.E);
            const int r = t * p.K + g;
            ids[r] = pick ? id : -1;
            probs[r] = pick ? prob : 0.0f;
            if (pick) atomicAdd(&at[id], 1);
            if (write) {
                p.topk_ids[r] = pick ? id : -1;
                p.topk_probs[r] = pick ? prob : 0.0f;
            }
        }
    }
}

// The routes of each expert together, by the whole workgroup.  The order among
// an expert's routes moves no result as long as they are one block (each is a
// column of its own); of several blocks every workgroup has to have the same,
// and then the routes are put in order.  `spare`: [N*K].
__device__ __forceinline__ void list_routes(const DecodeLists& l, const int* ids, uint16_t* spare, int routes) {
    const bool split = l.total[1] != 0;
    uint16_t* const to = split ? spare : l.route;
    for (int r = threadIdx.x; r < routes; r += kDecodeThreads) {
        const int e = ids[r];
        if (e >= 0) to[atomicAdd(&l.at[e], 1) & 0xFFFF] = static_cast<uint16_t>(r);
    }
    __syncthreads();
    if (!split) return;
    for (int r = threadIdx.x; r < routes; r += kDecodeThreads) {
        const int e = ids[r];
        if (e < 0) continue;
        const int n = l.at[e] >> 16, first = (l.at[e] & 0xFFFF) - n;
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += spare[first + i] < r;
        l.route[first + rank] = static_cast<uint16_t>(r);
    }
    __syncthreads();
}

// ---------------------------------------------------------------- first kernel

template <int LPT, int VPL, int T, int XT, int DEPTH>
__global__ __launch_bounds__(kDecodeThreads) void decode_fc1_kernel(DecodeArgs p) {
    typedef DecodeRing<T, XT, DEPTH> Ring;
    constexpr int CT = Ring::CT, RING = kDecodeWaves * DEPTH * Ring::BYTES, PARTS = kDecodeWaves * T * CT * 1024;
    static_assert(RING + PARTS + 28 * 1024 <= kDecodeLds, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kDecodeLds];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int routes = p.N * p.K;                       // <= 2048
    floatx4* const parts = reinterpret_cast<floatx4*>(smem + RING);
    DecodeLists l;
    l.total = reinterpret_cast<int*>(smem + RING + PARTS);
    l.at = l.total + 4;
    float* const probs = reinterpret_cast<float*>(l.at + p.E);
    l.block = reinterpret_cast<uint32_t*>(probs + routes);
    l.route = reinterpret_cast<uint16_t*>(l.block + min(routes, p.E + routes / Ring::XR));
    int* const ids = reinterpret_cast<int*>(smem);      // in the ring's place, which is not in use yet

    for (int e = threadIdx.x; e < p.E; e += kDecodeThreads) l.at[e] = 0;
    __syncthreads();
    decode_route<LPT, VPL>(p, l.at, ids, probs, blockIdx.x == 0);
    __syncthreads();
    if (wave == 0) list_blocks<Ring::XR>(l, p.E, lane);
    __syncthreads();
    list_routes(l, ids, reinterpret_cast<uint16_t*>(ids + routes), routes);

    const int tiles = p.ncols / (8 * T), items = *l.total * tiles;
    const int steps = p.Kdim / kDecodeStep, lo = steps * wave / kDecodeWaves, hi = steps * (wave + 1) / kDecodeWaves;
    Ring ring;
    ring.init(smem + wave * DEPTH * Ring::BYTES);
    int item = blockIdx.x, k = lo;                      // what is issued next
    auto aim = [&]() {                                  // at the rows of `item`
        if (item >= items || lo == hi) {
            ring.close();
            item = items;
            return;
        }
        const uint32_t b = l.block[item / tiles];
        const int e = __builtin_amdgcn_readfirstlane(block_expert(b)), c0 = item % tiles * (8 * T);
        const int64_t each = static_cast<int64_t>(p.wrows) * p.Kdim;
        ring.wsrc = make_rsrc(p.w + e * each, static_cast<uint32_t>(each * 2));
        ring.xsrc = make_rsrc(p.a, static_cast<uint32_t>(p.N) * p.Kdim * 2u);
#pragma unroll
        for (int i = 0; i < 2 * T; ++i)                 // rows 0-7 of a tile are gate rows, 8-15 the up rows beside them
            ring.woff[i] = static_cast<uint32_t>((i & 1 ? p.ncols : 0) + c0 + i / 2 * 8 + lane / 8) * p.Kdim * 2u +
                           Ring::piece(i % 2 * 8 + lane / 8);
#pragma unroll
        for (int i = 0; i < XT; ++i) {
            const int j = i * 8 + lane / 8;
            ring.xoff[i] = j < block_routes(b)
                ? static_cast<uint32_t>(l.route[block_first(b) + j] / p.K) * p.Kdim * 2u + Ring::piece(j) : kOob;
        }
    };
    auto issue = [&]() {
        ring.issue(item < items ? k : 0);
        if (item < items && ++k == hi) {
            k = lo;
            item += gridDim.x;
            aim();
        }
    };
    aim();
#pragma unroll 1
    for (int i = 0; i < DEPTH - 1; ++i) issue();
#pragma unroll 1
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        floatx4 acc[T][CT];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[t][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int s = lo; s < hi; ++s) {
            issue();
            ring.multiply(acc);
        }
        meet();                                         // the last item's parts are read
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) parts[(wave * T * CT + t * CT + c) * kWave + lane] = acc[t][c];
        meet();
        const uint32_t b = l.block[it / tiles];
        const int n = block_routes(b), c0 = it % tiles * (8 * T);
        for (int i = threadIdx.x; i < n * 8 * T; i += kDecodeThreads) {
            const int j = i / (8 * T), t = i % (8 * T) / 8, r = i % 8;
            // gate row r of the tile is element r % 4 of lane (j % 16, r / 4), its up row 8 rows below
            const float* at = reinterpret_cast<const float*>(parts + (t * CT + j / 16) * kWave + r / 4 * 16 + j % 16) + r % 4;
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kDecodeWaves; ++w) {
                g += at[w * T * CT * kWave * 4];
                u += at[w * T * CT * kWave * 4 + 2 * 16 * 4];
            }
            const int route = l.route[block_first(b) + j];
            p.out[static_cast<int64_t>(route) * p.ncols + c0 + t * 8 + r] = f32_to_bf16(silu(g) * u * probs[route]);
        }
    }
    wait_vmcnt<0>();                                    // no load may land after the workgroup's LDS is given away
}

// ---------------------------------------------------------------- second kernel

template <int XT, int DEPTH>
__global__ __launch_bounds__(kDecodeThreads) void decode_fc2_kernel(DecodeArgs p) {
    typedef DecodeRing<1, XT, DEPTH> Ring;
    constexpr int CT = Ring::CT, RING = kDecodeWaves * DEPTH * Ring::BYTES;
    static_assert(RING + kDecodeWaves * kDecodeMaxN * 64 + 28 * 1024 <= kDecodeLds, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kDecodeLds];
    const int lane = lane_id(), r16 = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int routes = p.N * p.K;
    float* const sums = reinterpret_cast<float*>(smem + RING);         // [waves][N][16]
    DecodeLists l;
    l.total = reinterpret_cast<int*>(sums + kDecodeWaves * p.N * 16);
    l.at = l.total + 4;
    l.block = reinterpret_cast<uint32_t*>(l.at + p.E);
    l.route = reinterpret_cast<uint16_t*>(l.block + min(routes, p.E + routes / Ring::XR));
    int* const ids = reinterpret_cast<int*>(smem);                     // in the ring's place

    for (int e = threadIdx.x; e < p.E; e += kDecodeThreads) l.at[e] = 0;
    for (int i = threadIdx.x; i < kDecodeWaves * p.N * 16; i += kDecodeThreads) sums[i] = 0.0f;
    __syncthreads();
    for (int r = threadIdx.x; r < routes; r += kDecodeThreads) {
        const int e = p.topk_ids[r];                                   // device data: range-checked
        const bool pick = static_cast<unsigned>(e) < static_cast<unsigned>(p.E);
        ids[r] = pick ? e : -1;
        if (pick) atomicAdd(&l.at[e], 1);
    }
    __syncthreads();
    if (wave == 0) list_blocks<Ring::XR>(l, p.E, lane);
    __syncthreads();
    list_routes(l, ids, reinterpret_cast<uint16_t*>(ids + routes), routes);

    const int c0 = blockIdx.x * 16, steps = p.Kdim / kDecodeStep, pairs = *l.total * steps;
    const int lo = static_cast<int>(static_cast<int64_t>(pairs) * wave / kDecodeWaves);
    const int hi = static_cast<int>(static_cast<int64_t>(pairs) * (wave + 1) / kDecodeWaves);
    Ring ring;
    ring.init(smem + wave * DEPTH * Ring::BYTES);
    ring.xsrc = make_rsrc(p.a, static_cast<uint32_t>(routes) * p.Kdim * 2u);
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
            ring.woff[i] = static_cast<uint32_t>(c0 + i * 8 + lane / 8) * p.Kdim * 2u + Ring::piece(i * 8 + lane / 8);
#pragma unroll
        for (int i = 0; i < XT; ++i) {
            const int j = i * 8 + lane / 8;
            ring.xoff[i] = j < block_routes(b)
                ? static_cast<uint32_t>(l.route[block_first(b) + j]) * p.Kdim * 2u + Ring::piece(j) : kOob;
        }
    };
    auto issue = [&]() {
        ring.issue(next < hi ? k : 0);
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
    float* const mine = sums + wave * p.N * 16;
    floatx4 acc[1][CT];
    int at = lo;
#pragma unroll 1
    while (at < hi) {
        const int b = at / steps, end = min(hi, (b + 1) * steps);
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[0][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (; at < end; ++at) {
            issue();
            ring.multiply(acc);
        }
        const uint32_t entry = l.block[b];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int j = c * 16 + r16;
            if (j < block_routes(entry)) {              // a token has an expert once: lanes meet no one's sums
                const int t = l.route[block_first(entry) + j] / p.K;
                floatx4* s = reinterpret_cast<floatx4*>(mine + t * 16 + q * 4);
                *s += acc[0][c];
            }
        }
    }
    wait_vmcnt<0>();
    __syncthreads();
    const int live = p.n_live ? min(max(p.n_live[0], 0), p.N) : p.N;
    for (int i = threadIdx.x; i < live * 16; i += kDecodeThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) v += sums[w * p.N * 16 + i];
        const int64_t o = static_cast<int64_t>(i / 16) * p.ncols + c0 + i % 16;
        if (p.residual) v += bf16_to_f32(p.residual[o]);
        p.out[o] = f32_to_bf16(v);
    }
}

template <int LPT, int VPL>
void launch_fc1(const DecodeArgs& a, double mean, hipStream_t s) {
    const int64_t most = std::min<int64_t>(a.N * a.K, a.E) * (a.ncols / 8);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(most, device_cus()));
    if (mean <= 2) decode_fc1_kernel<LPT, VPL, 1, 1, 4><<<grid, kDecodeThreads, 0, s>>>(a);
    else if (mean <= 8) decode_fc1_kernel<LPT, VPL, 1, 2, 3><<<grid, kDecodeThreads, 0, s>>>(a);
    else decode_fc1_kernel<LPT, VPL, 1, 4, 2><<<grid, kDecodeThreads, 0, s>>>(a);
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
    if (E <= 128 && K <= 16) launch_fc1<16, 8>(a, mean, stream);
    else if (E <= 256) launch_fc1<64, 4>(a, mean, stream);
    else launch_fc1<64, 16>(a, mean, stream);
    a.a = static_cast<const uint16_t*>(workspace); a.w = w2; a.residual = residual; a.out = y;
    a.Kdim = I; a.ncols = H; a.wrows = H;
    const unsigned grid = static_cast<unsigned>(H / 16);
    if (mean <= 2) decode_fc2_kernel<1, 4><<<grid, kDecodeThreads, 0, stream>>>(a);
    else if (mean <= 8) decode_fc2_kernel<2, 3><<<grid, kDecodeThreads, 0, stream>>>(a);
    else decode_fc2_kernel<4, 2><<<grid, kDecodeThreads, 0, stream>>>(a);
    return launch_status();
}

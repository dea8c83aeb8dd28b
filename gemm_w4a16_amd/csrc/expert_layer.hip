// expert_layer.hip -- a few tokens' whole pass through their experts in two launches: up products and SwiGLU, then
// down products and the weighted sum, on the int8 matrix cores, from rows already in 8 bits.
//
// Token t's choice j is pair p = t topk + j, of expert e = ids[p]; a pair whose id is outside [0, E) adds nothing.
//     g_i = a_t s_i sum_k xq[t][k] up[e][i][k],  u_i the same with row I + i   (integer sums exact)
//     v_i = g_i / (1 + exp(-g_i)) u_i            (fp32)
//     b = max |v| / 127 over each group of 64 columns (1 where 0, NaN where not finite), hq = clamp(rint(v / b))
//     o_n = s_n sum_groups b (sum_{i in group} hq_i down[e][n][i])            (integer sums exact, the rest fp32)
//     y[t][n] = sum_j weights[t][j] o_n          (in order of j, rounded once)
// The used experts' weights, read once, are what it costs: one token through two of eight experts of H = 4096, I = 14336
// takes 38 us up (6.2 TB/s) and 21 down (5.5); eight tokens, 6.3 experts, 111 (6.7) and 61 (6.1); 32 tokens x 8 of 64
// experts of 2048 x 1024 41 and 28 (5.6, 4.1).  Small layers: each launch's start, sort and finish, 4-5 us (five tokens x 3
// of 20 experts of 1008 x 496 8.0 and 5.6).
// A scale for 64 columns instead of one for the row: the first launch then finishes its codes by itself (a row's
// largest magnitude would need all of its blocks), and small values keep more bits.
#include <algorithm>
#include <type_traits>

#include "experts.h"
#include "launch.h"
#include "lds_dma.h"

namespace w4a16 {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kGroup = 64;  // columns of v that share a scale
constexpr int kPairs = (int)kLayerPairs;

// ---- the pairs, sorted by expert and cut into tiles of at most XR rows of one expert -------------------

constexpr int kExperts = (int)kMaxExperts;
constexpr int kExpertBits = 9;
constexpr int kPairWaves = kPairs / kWave;
static_assert(kExperts <= 1 << kExpertBits);

template <int XR>
struct alignas(16) PairTiles {
    union {
        uint8_t count[kPairWaves][kExperts];  // pairs of an expert among a wave's 64
        uint8_t row[kPairs][XR];              // a tile's pairs
    };
    uint16_t base[kExperts];                  // an expert's first tile
    uint16_t expert[kPairs], rows[kPairs];    // of a tile
    int wave_tiles[kPairWaves], tiles;
};

// Sums over the lanes up to and with this one.
__device__ __forceinline__ int lanes_up_to(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8: within 16 lanes
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, kDppRowBcast15, 0xA, 0xF, false);
    return v + __builtin_amdgcn_update_dpp(0, v, kDppRowBcast31, 0xC, 0xF, false);
}

// The lanes whose expert has the same bits as this one's (of those that have one).
__device__ __forceinline__ uint64_t lanes_alike(int e) {
    uint64_t alike = __ballot(e >= 0);
#pragma unroll
    for (int b = 0; b < kExpertBits; ++b) {
        const bool bit = (e >> b) & 1;
        const uint64_t set = __ballot(bit);
        alike &= bit ? set : ~set;
    }
    return alike;
}

// By every block for itself, the same in all of them: tiles in some order, an expert's pairs in their own order.  At least
// kPairs threads, a thread a pair.  Up to 64 pairs by one wave, with one barrier (one token x 2 of 8 experts of 1024 x
// 512 9.4 us against 10.6 in all); more: then a thread two experts.  Returns this thread's pair's expert (-1: none).  Ends
// with a barrier.
template <int XR, typename TI>
__device__ __forceinline__ int sort_pairs(const TI* __restrict__ ids, int P, int E, PairTiles<XR>& s) {
    static_assert(kExperts == 2 * kPairs, "a thread two experts");
    const int p = threadIdx.x, wave = wave_id(), lane = lane_id();
    int e = -1;
    if (p < P) {
        const TI id = ids[p];
        if (id >= 0 && id < E) e = (int)id;
    }
    if (P <= kWave) {
        if (wave == 0) {
            const uint64_t alike = lanes_alike(e), lower = (1ull << lane) - 1;
            const int same = __popcll(alike & lower);
            const bool head = e >= 0 && same % XR == 0;  // a tile's first pair
            const uint64_t heads = __ballot(head);
            uint64_t own = heads & alike;  // this expert's tiles: the pair's is the one of number same / XR
            for (int i = 0; i < same / XR; ++i) own &= own - 1;
            if (e >= 0) {
                const int t = __popcll(heads & ((own & (0 - own)) - 1));
                s.row[t][same % XR] = (uint8_t)p;
                if (head) s.expert[t] = (uint16_t)e, s.rows[t] = (uint16_t)min(__popcll(alike) - same, XR);
            }
            if (p == 0) s.tiles = __popcll(heads);
        }
        __syncthreads();
        return e;
    }
    for (int i = p; i < kPairWaves * kExperts / 16; i += blockDim.x) reinterpret_cast<uint4*>(s.count)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    // this pair's place among its expert's in the wave
    int same = 0;
    const uint64_t alike = lanes_alike(e);
    if (e >= 0) {
        same = __popcll(alike & ((1ull << lane) - 1));
        if ((alike >> lane) == 1) s.count[wave][e] = (uint8_t)(same + 1);
    }
    __syncthreads();
    int before[2], tiles[2], count[2];
    if (wave < kPairWaves) {
#pragma unroll
        for (int w = 0; w < kPairWaves; ++w)
            if (w < wave && e >= 0) same += s.count[w][e];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            count[i] = 0;
#pragma unroll
            for (int w = 0; w < kPairWaves; ++w) count[i] += s.count[w][2 * p + i];
            tiles[i] = (count[i] + XR - 1) / XR;
        }
        const int end = lanes_up_to(tiles[0] + tiles[1]);
        if (lane == kWave - 1) s.wave_tiles[wave] = end;
        before[0] = end - tiles[0] - tiles[1];
    }
    __syncthreads();  // (count is read: row may overwrite it)
    if (wave < kPairWaves) {
        int all = 0;
#pragma unroll
        for (int w = 0; w < kPairWaves; ++w) {
            if (w < wave) before[0] += s.wave_tiles[w];
            all += s.wave_tiles[w];
        }
        before[1] = before[0] + tiles[0];
        if (p == 0) s.tiles = all;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s.base[2 * p + i] = (uint16_t)before[i];
            for (int t = 0; t < tiles[i]; ++t) {
                s.expert[before[i] + t] = (uint16_t)(2 * p + i);
                s.rows[before[i] + t] = (uint16_t)min(count[i] - XR * t, XR);
            }
        }
    }
    __syncthreads();
    if (e >= 0) s.row[s.base[e] + same / XR][same % XR] = (uint8_t)p;
    __syncthreads();
    return e;
}

// ---- a wave's own stream of operands -------------------------------------------------------------------
//
// Each wave copies what it multiplies into a ring of R stages of its own in LDS, a stage being one k-tile (128 bytes)
// of its weight rows and of XR activation rows, and waits for its copies by their number; no barrier joins the
// waves until their sums do.  A stage past the wave's last is as many copies of one line, so that every wait is a
// constant.  LDS slot lane % 8 of a row takes its 16-byte chunk slot ^ ((row >> 1) & 7), so that fragment
// reads meet no bank twice.

// the chunk that this lane copies of row r, and where fragment chunk c of row r lies
__device__ __forceinline__ int copied_chunk(int r) { return (lane_id() % 8) ^ ((r >> 1) & 7); }
__device__ __forceinline__ i32x4_t fragment(const char* rows, int r, int c) {
    return *reinterpret_cast<const i32x4_t*>(rows + 128 * r + 16 * (c ^ ((r >> 1) & 7)));
}
// what a chunk's offset falls back by where only `left` (a multiple of 16) bytes of the k-tile are there
__device__ __forceinline__ uint32_t past_end(int chunk, int left) { return left < 128 ? (uint32_t)max(16 * chunk - (left - 16), 0) : 0u; }

template <bool kOnce>
__device__ __forceinline__ void copy_weights(uint32_t off, const void* base, uint32_t lds) {
    if constexpr (kOnce)
        dma16_once(off, base, lds);
    else
        dma16(off, base, lds);
}

// this wave's LDS reads are done: its copies may overwrite what they read
__device__ __forceinline__ void reads_done() { __builtin_amdgcn_s_waitcnt(0xC07F /* lgkmcnt(0), no other */); }

template <typename T>
__device__ __forceinline__ T* uniform(T* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v), hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return reinterpret_cast<T*>((uint64_t)hi << 32 | lo);
}

// ---- up products and SwiGLU ----------------------------------------------------------------------------

// A block: one tile of pairs, one group of 64 columns of v; a wave 16 of the columns (their gate rows and up rows, 32
// weight rows).  Two stages a wave, so that four blocks share a CU: while one sorts or finishes, the others stream
// (three stages, two blocks a CU: 49 us against 43 for 32 tokens x 8 of 64 experts, H = 2048, I = 1024).  Three where
// all blocks run at once, two on a CU (4 of 32 experts of 2048 x 768 for one token 8.2 us against 8.8, 20 tokens x 2 of 16 of
// 2048 x 1024 22.0 against 23.1 in all).
constexpr int64_t kUpDeepBlocks = 512;
template <int XR, int R_>
struct UpShape {
    static constexpr int R = R_, kStage = 4096 + 128 * XR, kCopies = 4 + XR / 8;
    static constexpr size_t kLds = 4 * R * kStage;
    static_assert(kLds >= sizeof(PairTiles<XR>), "the lists fit in the ring");
};

template <typename TI, int XR, int kStages, bool kOnce>
__global__ __launch_bounds__(256) void layer_up_kernel(const int8_t* __restrict__ xq, const float* __restrict__ ascale,
                                                            const TI* __restrict__ ids, int P, int topk, int E,
                                                            const int8_t* __restrict__ up, const float* __restrict__ up_scales, int H,
                                                            int I, int groups, int8_t* __restrict__ hq, float* __restrict__ hscale) {
    using S = UpShape<XR, kStages>;
    constexpr int R = S::R, C = S::kCopies;
    __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
    const int tile = blockIdx.x / groups, group = blockIdx.x - tile * groups;
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, kg = lane >> 4;
    PairTiles<XR>& s = *reinterpret_cast<PairTiles<XR>*>(smem);
    sort_pairs<XR>(ids, P, E, s);
    if (tile >= s.tiles) return;
    const int rows = s.rows[tile], expert = __builtin_amdgcn_readfirstlane(s.expert[tile]);
    const int pair = s.row[tile][min(l16, rows - 1)];  // of this lane's row
    uint32_t xoff[XR / 8], woff[2];
#pragma unroll
    for (int i = 0; i < XR / 8; ++i) {
        const int r = 8 * i + lane / 8;
        xoff[i] = (uint32_t)(s.row[tile][min(r, rows - 1)] / topk) * (uint32_t)H + 16u * copied_chunk(r);
    }
    const int i0 = group * kGroup + 16 * wave;
    // the scales, asked for before the operands
    float a = 0.0f;
    float4 sg = {}, su = {};
    if (i0 < I) {  // (I % 16 == 0: all of a wave's columns are there, or none)
        a = ascale[pair / topk];
        sg = *reinterpret_cast<const float4*>(up_scales + (size_t)expert * 2 * I + i0 + 4 * kg);
        su = *reinterpret_cast<const float4*>(up_scales + (size_t)expert * 2 * I + I + i0 + 4 * kg);
    }
    __syncthreads();  // the lists are read: the ring may overwrite them

    i32x4_t acc[2] = {};
    if (i0 < I) {
        const int T = (H + 127) / 128;
        const int8_t* gate = uniform(up + ((size_t)expert * 2 * I + i0) * H);
        const int8_t* other = uniform(gate + (size_t)I * H);
#pragma unroll
        for (int i = 0; i < 2; ++i) woff[i] = (uint32_t)(8 * i + lane / 8) * (uint32_t)H + 16u * copied_chunk(8 * i + lane / 8);
        char* ring = smem + wave * R * S::kStage;
        const uint32_t ring_lds = lds_addr(ring);
        // k-tiles from a place of the wave's own on: blocks in step with one another would all ask the same part of the
        // memory channels (rows of a power of two)
        const int turn = (int)((blockIdx.x * 5 + wave * 3) % (unsigned)T);
        auto k_tile = [&](int t) __attribute__((always_inline)) { return t + turn < T ? t + turn : t + turn - T; };
        auto issue = [&](int t, int slot) __attribute__((always_inline)) {
            const bool there = t < T;
            const int kt = there ? k_tile(t) : 0;
            const uint32_t lds = ring_lds + (uint32_t)(slot * S::kStage);
            const int left = H - kt * 128;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t off = there ? woff[i] - past_end(copied_chunk(8 * i + lane / 8), left) : 0;
                copy_weights<kOnce>(off, gate + kt * 128, lds + 1024 * i);
                copy_weights<kOnce>(off, other + kt * 128, lds + 2048 + 1024 * i);
            }
#pragma unroll
            for (int i = 0; i < XR / 8; ++i)
                dma16(there ? xoff[i] - past_end(copied_chunk(8 * i + lane / 8), left) : 0, xq + kt * 128, lds + 4096 + 1024 * i);
        };
#pragma unroll
        for (int t = 0; t < R - 1; ++t) issue(t, t);
        int slot = 0, ahead = R - 1;
        for (int t = 0; t < T; ++t) {
            issue(t + R - 1, ahead);
            wait_vm<(R - 1) * C>();
            const char* w = ring + slot * S::kStage;
            const int chunks = (H - k_tile(t) * 128) / 16;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                i32x4_t x = fragment(w + 4096, l16 % XR, 4 * ks + kg);
                if (4 * ks + kg >= chunks) x = i32x4_t{0, 0, 0, 0};
                acc[0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fragment(w, l16, 4 * ks + kg), x, acc[0], 0, 0, 0);
                acc[1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fragment(w + 2048, l16, 4 * ks + kg), x, acc[1], 0, 0, 0);
            }
            reads_done();
            slot = slot + 1 == R ? 0 : slot + 1;
            ahead = ahead + 1 == R ? 0 : ahead + 1;
        }
        wait_vm<0>();
    }
    __syncthreads();  // no copy is in flight: the ring's memory is free

    float* tops = reinterpret_cast<float*>(smem);  // [4][16]
    // lane (l16, kg): row l16, columns i0 + 4 kg ..
    float v[4] = {0, 0, 0, 0};
    uint32_t m = 0;
    if (i0 < I) {
        const float g4[4] = {sg.x, sg.y, sg.z, sg.w}, u4[4] = {su.x, su.y, su.z, su.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float g = (float)acc[0][i] * g4[i] * a, u = (float)acc[1][i] * u4[i] * a;
            v[i] = g / (1.0f + expf(-g)) * u;
            m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (kg == 0) tops[16 * wave + l16] = __uint_as_float(m);
    __syncthreads();
    if (l16 >= rows) return;
    m = __float_as_uint(tops[l16]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max(m, __float_as_uint(tops[16 * i + l16]));
    const float b = scale_i8(__uint_as_float(m));
    uint32_t q = 0;
    if (b == b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q |= code_i8(v[i], b) << (8 * i);
    }
    if (i0 < I) *reinterpret_cast<uint32_t*>(hq + (size_t)pair * I + i0 + 4 * kg) = q;
    if (wave == 0 && kg == 0) hscale[(size_t)pair * groups + group] = b;
}

// ---- down products and the weighted sum ----------------------------------------------------------------

// A block: kCols columns of y for every token.  Its waves share the tiles of pairs, each cut into parts of K; a
// tile's part is added by one wave, kept in LDS, and the parts and choices are added at the end, in order.
// kCols = 8 (XR = 8): a stage is two k-tiles, the first in the matrix instruction's rows and columns 0..7, the
// second in 8..15; the sums of rows with columns of the other k-tile are not used.  Twice the blocks, where 16
// columns a block would leave CUs idle.
constexpr int kDownWaves = 8, kDownRows = 256;  // rows of sums that LDS has room for
template <int XR, int kCols>
struct DownShape {
    static constexpr int kTiles = 16 / kCols;                      // k-tiles of a stage
    static constexpr int kX = 2048, kScales = kX + 128 * XR * kTiles, kStage = kScales + 256;
    static constexpr int kCopies = 2 + XR / 8 * kTiles + 1;
    static constexpr int R = 3;  // (four or five: no faster)
    static_assert(kTiles == 1 || XR == 8, "rows of one k-tile in each half");
};

template <typename TO, typename TI, int XR, int kCols, bool kOnce>
__global__ __launch_bounds__(64 * kDownWaves) void layer_down_kernel(const int8_t* __restrict__ hq, const float* __restrict__ hscale,
                                                                     const TI* __restrict__ ids, int T, int topk,
                                                                     const float* __restrict__ weights, int E,
                                                                     const int8_t* __restrict__ down,
                                                                     const float* __restrict__ down_scales, int H, int I, int groups,
                                                                     TO* __restrict__ y) {
    using S = DownShape<XR, kCols>;
    constexpr int R = S::R, C = S::kCopies, KW = S::kTiles;
    __shared__ __attribute__((aligned(1024))) char smem[kDownWaves * R * S::kStage];
    __shared__ float4 sums[kDownRows][4];
    __shared__ PairTiles<XR> s;
    __shared__ float pair_weight[kPairs];  // zero, and its sums not read, for a pair with no expert
    __shared__ uint8_t pair_there[kPairs];
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.x * kCols, P = T * topk, KT = (I + 128 * KW - 1) / (128 * KW);  // (of stages)
    float pw = 0.0f;
    if ((int)threadIdx.x < P) pw = weights[threadIdx.x];
    const int e0 = sort_pairs<XR>(ids, P, E, s);
    if ((int)threadIdx.x < P) pair_weight[threadIdx.x] = pw, pair_there[threadIdx.x] = e0 >= 0;
    const int tiles = __builtin_amdgcn_readfirstlane(s.tiles);

    // the parts of K (a power of two) that leave the busiest wave least to do
    int log = 0;
    for (int i = 1, least = (tiles + kDownWaves - 1) / kDownWaves * KT; i <= 3; ++i) {
        const int parts = 1 << i;
        if (parts > KT || parts * P > kDownRows) break;
        const int most = (tiles * parts + kDownWaves - 1) / kDownWaves * ((KT + parts - 1) >> i);
        if (most < least) least = most, log = i;
    }
    const int units = tiles << log;

    // What a lane copies of a stage: weight rows (stage half kt2, column r) in 16 of 128 bytes, activation rows alike, and
    // lanes 0.. of the last copy the groups' scales [k-tile][row][2], lanes 48.. the columns' own.
    struct Stream {
        int unit, kt, end;  // none left: unit >= units
        const int8_t* w;    // of the unit
        uint32_t xoff[XR / 8];
        const float* scale;
    };
    auto begin = [&](Stream& it, int unit) __attribute__((always_inline)) {
        it.unit = unit;
        it.kt = it.end = 0;
        if (unit >= units) return;
        const int tile = unit >> log, part = unit & ((1 << log) - 1);
        it.kt = (KT * part) >> log;
        it.end = (KT * (part + 1)) >> log;
        const int rows = s.rows[tile], expert = __builtin_amdgcn_readfirstlane(s.expert[tile]);
        it.w = uniform(down + ((size_t)expert * H + n0) * I);
#pragma unroll
        for (int i = 0; i < XR / 8; ++i) it.xoff[i] = (uint32_t)s.row[tile][min(8 * i + lane / 8, rows - 1)] * (uint32_t)I;
        it.scale = lane < 48 ? hscale + (uint32_t)s.row[tile][min(lane / 2 % XR, rows - 1)] * (uint32_t)groups
                             : down_scales + (size_t)expert * H + n0 + (lane - 48) % kCols;
    };
    char* ring = smem + wave * R * S::kStage;
    const uint32_t ring_lds = lds_addr(ring);
    auto issue = [&](Stream& it, int slot) __attribute__((always_inline)) {
        const bool there = it.unit < units;
        const uint32_t lds = ring_lds + (uint32_t)(slot * S::kStage);
        // LDS row 8 j + lane / 8 of 16, in k-tile j of the stage (KW = 2), its chunk c at 16 c of the k-tile; chunks past I
        // read the row's last one
        auto at = [&](int j) __attribute__((always_inline)) {
            const int k = (it.kt * KW + (KW == 2 ? j : 0)) * 128 + 16 * copied_chunk(8 * j + lane / 8);
            return (uint32_t)min(k, I - 16);
        };
        const int8_t* w = there ? it.w : hq;  // (no weights of experts that no token chose)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t row = KW == 2 ? lane / 8 : 8 * j + lane / 8;
            copy_weights<kOnce>(there ? row * (uint32_t)I + at(j) : 0, w, lds + 1024 * j);
        }
#pragma unroll
        for (int j = 0; j < XR / 8 * KW; ++j) dma16(there ? it.xoff[KW == 2 ? 0 : j] + at(j) : 0, hq, lds + S::kX + 1024 * j);
        const int group = min(2 * (it.kt * KW + (KW == 2 ? lane / 16 : 0)) + (lane & 1), groups - 1);
        const bool last = there && ++it.kt == it.end;
        // (the columns' scales with a unit's last stage only: asked for with each, they cost 40% more time)
        dma4_at(!there || (lane >= 48 && !last) ? hscale : it.scale + (lane < 48 ? group : 0), lds + S::kScales);
        if (last) begin(it, it.unit + kDownWaves);
    };

    Stream ahead;
    begin(ahead, wave);
    int unit = ahead.unit, kt = ahead.kt, end = ahead.end;
#pragma unroll
    for (int t = 0; t < R - 1; ++t) issue(ahead, t);
    int slot = 0, next = R - 1;
    float acc[4] = {0, 0, 0, 0};
    const int half = KW == 2 ? l16 / 8 : 0;  // the k-tile of this lane's row
    while (unit < units) {
        issue(ahead, next);
        wait_vm<(R - 1) * C>();
        const char* w = ring + slot * S::kStage;
        const int chunks = (I - (kt * KW + half) * 128) / 16;
        const float2 b = *reinterpret_cast<const float2*>(w + S::kScales + 64 * (KW == 2 ? half : 0) + 8 * (l16 % XR));
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            i32x4_t x = fragment(w + S::kX, KW == 2 ? l16 : l16 % XR, 4 * ks + kg);
            if (4 * ks + kg >= chunks) x = i32x4_t{0, 0, 0, 0};
            const i32x4_t sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(fragment(w, l16, 4 * ks + kg), x, i32x4_t{0, 0, 0, 0}, 0, 0, 0);
            // (a group past the last has no chunks: its scale, the last one's, meets a sum of zero)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf((float)sum[i], ks == 0 ? b.x : b.y, acc[i]);
        }
        if (++kt == end) {  // the unit's sums, times the columns' scales
            const int tile = unit >> log, part = unit & ((1 << log) - 1), rows = s.rows[tile];
            const float4 sn = *reinterpret_cast<const float4*>(w + S::kScales + 192 + 16 * (KW == 2 ? kg % 2 : kg));
            float4 o = make_float4(acc[0] * sn.x, acc[1] * sn.y, acc[2] * sn.z, acc[3] * sn.w);
            if constexpr (KW == 2) {  // columns 4 (kg % 2).. of row l16 % 8: in lanes (l16, kg) and (l16 + 8, kg + 2)
                const int other = (lane + 40) & 63;
                o.x += __shfl(o.x, other), o.y += __shfl(o.y, other), o.z += __shfl(o.z, other), o.w += __shfl(o.w, other);
                if (l16 < min(rows, 8) && kg < 2) sums[part * P + s.row[tile][l16]][kg] = o;
            } else {
                if (l16 < rows) sums[part * P + s.row[tile][l16]][kg] = o;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = 0.0f;
            unit += kDownWaves;
            const int p = unit & ((1 << log) - 1);
            kt = (KT * p) >> log;
            end = (KT * (p + 1)) >> log;
        }
        reads_done();
        slot = slot + 1 == R ? 0 : slot + 1;
        next = next + 1 == R ? 0 : next + 1;
    }
    wait_vm<0>();
    __syncthreads();
    const int t = threadIdx.x / kCols, c = threadIdx.x % kCols;
    if (t >= T) return;
    const float* part_sums = reinterpret_cast<const float*>(sums);
    float out = 0.0f;
    for (int p = t * topk; p < (t + 1) * topk; ++p) {
        if (!pair_there[p]) continue;
        float o = part_sums[p * 16 + c];
        for (int i = 1; i < 1 << log; ++i) o += part_sums[(i * P + p) * 16 + c];
        out = __builtin_fmaf(pair_weight[p], o, out);
    }
    y[(size_t)t * H + n0 + c] = from_f32<TO>(out);
}

}  // namespace

size_t expert_layer_scale_bytes(int64_t pairs, int64_t I) {
    return (size_t)pairs * (size_t)((I + kGroup - 1) / kGroup) * 4;
}

hipError_t launch_expert_layer_w8a8(int dtype, const int8_t* xq, const float* ascale, int64_t T, const void* ids, int id_bits,
                                    int64_t topk, const float* weights, int64_t E, const int8_t* up, const float* up_scales,
                                    const int8_t* down, const float* down_scales, int64_t H, int64_t I, void* y, int8_t* hq,
                                    float* hscale, hipStream_t stream) {
    const int64_t P = T * topk, groups = (I + kGroup - 1) / kGroup;
    auto run = [&](auto id, auto xr, auto cols, auto once) {
        using TI = decltype(id);
        constexpr int XR = decltype(xr)::value, kCols = decltype(cols)::value;
        constexpr bool kOnce = decltype(once)::value;
        const TI* idt = static_cast<const TI*>(ids);
        const int64_t blocks = expert_tiles(P, E, XR) * groups;
        auto launch_up = [&](auto stages) {
            hipLaunchKernelGGL((layer_up_kernel<TI, XR, decltype(stages)::value, kOnce>), dim3((unsigned)blocks), dim3(256), 0, stream, xq,
                               ascale, idt, (int)P, (int)topk, (int)E, up, up_scales, (int)H, (int)I, (int)groups, hq, hscale);
        };
        if (blocks <= kUpDeepBlocks)
            launch_up(std::integral_constant<int, 3>{});
        else
            launch_up(std::integral_constant<int, 2>{});
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        return with_act_type(dtype, [&](auto t) {
            using TO = decltype(t);
            hipLaunchKernelGGL((layer_down_kernel<TO, TI, XR, kCols, kOnce>), dim3((unsigned)(H / kCols)), dim3(64 * kDownWaves), 0,
                               stream, hq, hscale, idt, (int)T, (int)topk, weights, (int)E, down, down_scales, (int)H, (int)I,
                               (int)groups, static_cast<TO*>(y));
            return hipGetLastError();
        });
    };
    using I8 = std::integral_constant<int, 8>;
    using I16 = std::integral_constant<int, 16>;
    // (The ids are on the device: both rules are for pairs spread over the experts.  All 32 tokens x 8 on the same 8 of 64 experts of
    // 2048 x 1024 take 33.5 us, four tiles of 8 pairs reading each of those experts past the caches, against 23.9 for a layer of
    // 8 experts with its tiles of 16 pairs; spread over the 64 it is 70.)
    const double weight_bytes = 3.0 * (double)std::min(P, E) * (double)H * (double)I;
    auto with_once = [&](auto id, auto xr, auto cols) {
        return weight_bytes >= kOnceBytes ? run(id, xr, cols, std::true_type{}) : run(id, xr, cols, std::false_type{});
    };
    auto with_rows = [&](auto id) {
        if (T > 8 && P > 4 * E) return with_once(id, I16{}, I16{});
        return H < 16 * 256 ? with_once(id, I8{}, I8{}) : with_once(id, I8{}, I16{});
    };
    return id_bits == 32 ? with_rows(int32_t{}) : with_rows(int64_t{});
}

}  // namespace w4a16

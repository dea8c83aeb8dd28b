// expert_layer.hip -- a few tokens' whole pass through their experts in two launches: up products and SwiGLU, then
// down products and the weighted sum, on the int8 matrix cores, from rows already in 8 bits.
//
// Token t's choice j is pair p = t topk + j, of expert e = ids[p]; a pair whose id is outside [0, E) adds nothing.
//     g_i = a_t s_i sum_k xq[t][k] up[e][i][k],  u_i the same with row I + i   (integer sums exact)
//     v_i = g_i / (1 + exp(-g_i)) u_i            (fp32)
//     b = max |v| / 127 over each group of 64 columns (1 where 0, NaN where not finite), hq = clamp(rint(v / b))
//     o_n = s_n sum_groups b (sum_{i in group} hq_i down[e][n][i])            (integer sums exact, the rest fp32)
//     y[t][n] = sum_j weights[t][j] o_n          (in order of j, rounded once)
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

struct alignas(16) PairTiles {
    int ids[kPairs];             // a pair's expert, INT32_MAX for none
    uint16_t sorted[kPairs];     // pairs by expert, those of one expert in their own order
    uint16_t first[kPairs + 1];  // a tile's first place in sorted; first[tiles] the number of pairs with an expert
    int heads[kPairs / kWave], tiles;
};

// By every block for itself: a thread a pair, which counts the pairs that come before its own.  At least kPairs
// threads.  Ends with a barrier.
template <int XR, typename TI>
__device__ __forceinline__ void sort_pairs(const TI* __restrict__ ids, int P, int E, PairTiles& s) {
    const int p = threadIdx.x;
    int e = INT32_MAX;
    if (p < P) {
        const TI id = ids[p];
        if (id >= 0 && id < E) e = (int)id;
    }
    if (p < kPairs) s.ids[p] = e;
    __syncthreads();
    int less = 0, same = 0;
    if (p < P) {
        for (int q = 0; q < P; q += 4) {  // (places from P on hold INT32_MAX)
            const int4 v = *reinterpret_cast<const int4*>(s.ids + q);
            const int f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                less += f[i] < e;
                same += f[i] == e && q + i < p;
            }
        }
        // a pair that begins a tile is marked
        if (e != INT32_MAX) s.sorted[less + same] = (uint16_t)(p | (same % XR == 0 ? 0x8000 : 0));
    }
    const int n = __syncthreads_count(e != INT32_MAX);
    const bool head = p < n && (s.sorted[p] & 0x8000);
    const uint64_t heads = __ballot(head);
    if (p < kPairs && lane_id() == 0) s.heads[wave_id()] = __popcll(heads);
    __syncthreads();
    if (p < kPairs) {
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kPairs / kWave; ++w) {
            if (w < wave_id()) before += s.heads[w];
            all += s.heads[w];
        }
        if (head) {
            s.first[before + __popcll(heads & ((1ull << lane_id()) - 1))] = (uint16_t)p;
            s.sorted[p] &= 0x7FFF;
        }
        if (p == 0) s.first[all] = (uint16_t)n, s.tiles = all;
    }
    __syncthreads();
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

// A block: one tile of pairs, one group of 64 columns of v.  Wave (cw, ks): 16 of the columns (their gate rows and up
// rows, 32 weight rows), every KS-th k-tile.
template <int XR, int KS>
struct UpShape {
    static constexpr int NW = 4 * KS, kStage = 4096 + 128 * XR, kCopies = 4 + XR / 8;
    static constexpr int R = KS == 1 && XR == 8 ? 4 : 3;
    static constexpr size_t kLds = (size_t)NW * R * kStage;
    static_assert(kLds >= sizeof(PairTiles) && kLds >= 4 * 2 * 1024 * (KS - 1) + 1024, "the ring holds what comes before and after it");
};

template <typename TI, int XR, int KS, bool kOnce>
__global__ __launch_bounds__(256 * KS) void layer_up_kernel(const int8_t* __restrict__ xq, const float* __restrict__ ascale,
                                                            const TI* __restrict__ ids, int P, int topk, int E,
                                                            const int8_t* __restrict__ up, const float* __restrict__ up_scales, int H,
                                                            int I, int groups, int8_t* __restrict__ hq, float* __restrict__ hscale) {
    using S = UpShape<XR, KS>;
    constexpr int R = S::R, C = S::kCopies;
    __shared__ __attribute__((aligned(1024))) char smem[S::kLds];
    const int tile = blockIdx.x / groups, group = blockIdx.x - tile * groups;
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, kg = lane >> 4;
    const int cw = wave % 4, ks0 = wave / 4;
    PairTiles& s = *reinterpret_cast<PairTiles*>(smem);
    sort_pairs<XR>(ids, P, E, s);
    if (tile >= s.tiles) return;
    const int first = s.first[tile], rows = s.first[tile + 1] - first;
    const int expert = __builtin_amdgcn_readfirstlane(s.ids[s.sorted[first]]);
    const int pair = s.sorted[first + min(l16, rows - 1)];  // of this lane's row
    uint32_t xoff[XR / 8], woff[2];
#pragma unroll
    for (int i = 0; i < XR / 8; ++i) {
        const int r = 8 * i + lane / 8;
        xoff[i] = (uint32_t)(s.sorted[first + min(r, rows - 1)] / topk) * (uint32_t)H + 16u * copied_chunk(r);
    }
    __syncthreads();  // the lists are read: the ring may overwrite them

    const int i0 = group * kGroup + 16 * cw;
    i32x4_t acc[2] = {};
    if (i0 < I) {  // (I % 16 == 0: all of a wave's columns are there, or none)
        const int KT = (H + 127) / 128, T = (KT - ks0 + KS - 1) / KS;
        const int8_t* gate = uniform(up + ((size_t)expert * 2 * I + i0) * H);
        const int8_t* other = uniform(gate + (size_t)I * H);
#pragma unroll
        for (int i = 0; i < 2; ++i) woff[i] = (uint32_t)(8 * i + lane / 8) * (uint32_t)H + 16u * copied_chunk(8 * i + lane / 8);
        char* ring = smem + wave * R * S::kStage;
        const uint32_t ring_lds = lds_addr(ring);
        auto issue = [&](int t, int slot) __attribute__((always_inline)) {
            const bool there = t < T;
            const int kt = there ? t * KS + ks0 : 0;
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
            const int chunks = (H - (t * KS + ks0) * 128) / 16;
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
    __syncthreads();  // no copy is in flight

    // the k-tiles' sums joined (exact integers), in the ring's memory
    float* tops = reinterpret_cast<float*>(smem);  // [4][16]
    i32x4_t* sums = reinterpret_cast<i32x4_t*>(smem + 1024);
    if constexpr (KS > 1) {
        if (ks0 > 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) sums[(((ks0 - 1) * 4 + cw) * 2 + i) * 64 + lane] = acc[i];
        }
        __syncthreads();
        if (ks0 == 0) {
#pragma unroll
            for (int o = 0; o < KS - 1; ++o)
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[i] += sums[((o * 4 + cw) * 2 + i) * 64 + lane];
        }
    }
    // lane (l16, kg): row l16, columns i0 + 4 kg ..
    float v[4] = {0, 0, 0, 0};
    if (ks0 == 0) {
        uint32_t m = 0;
        if (i0 < I) {
            const float a = ascale[pair / topk];
            const float4 sg = *reinterpret_cast<const float4*>(up_scales + (size_t)expert * 2 * I + i0 + 4 * kg);
            const float4 su = *reinterpret_cast<const float4*>(up_scales + (size_t)expert * 2 * I + I + i0 + 4 * kg);
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
        if (kg == 0) tops[16 * cw + l16] = __uint_as_float(m);
    }
    __syncthreads();
    if (ks0 > 0 || l16 >= rows) return;
    uint32_t m = __float_as_uint(tops[l16]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max(m, __float_as_uint(tops[16 * i + l16]));
    const float b = scale_i8(__uint_as_float(m));
    uint32_t q = 0;
    if (b == b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q |= code_i8(v[i], b) << (8 * i);
    }
    if (i0 < I) *reinterpret_cast<uint32_t*>(hq + (size_t)pair * I + i0 + 4 * kg) = q;
    if (cw == 0 && kg == 0) hscale[(size_t)pair * groups + group] = b;
}

// ---- down products and the weighted sum ----------------------------------------------------------------

// A block: 16 columns of y for every token.  Its waves share the tiles of pairs, each cut into `parts` of K; a tile's
// part is added by one wave, kept in LDS, and the parts and choices are added at the end, in order.
constexpr int kDownWaves = 8, kDownRows = 256;  // rows of sums that LDS has room for
template <int XR>
struct DownShape {
    static constexpr int kScales = 2048 + 128 * XR, kStage = kScales + 256, kCopies = 2 + XR / 8 + 1;
    static constexpr int R = XR == 8 ? 5 : 4;
};

template <typename TO, typename TI, int XR, bool kOnce>
__global__ __launch_bounds__(64 * kDownWaves) void layer_down_kernel(const int8_t* __restrict__ hq, const float* __restrict__ hscale,
                                                                     const TI* __restrict__ ids, int T, int topk,
                                                                     const float* __restrict__ weights, int E,
                                                                     const int8_t* __restrict__ down,
                                                                     const float* __restrict__ down_scales, int H, int I, int groups,
                                                                     TO* __restrict__ y) {
    using S = DownShape<XR>;
    constexpr int R = S::R, C = S::kCopies;
    __shared__ __attribute__((aligned(1024))) char smem[kDownWaves * R * S::kStage];
    __shared__ float4 sums[kDownRows][4];
    __shared__ PairTiles s;
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.x * 16, P = T * topk, KT = (I + 127) / 128;
    sort_pairs<XR>(ids, P, E, s);
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

    struct Stream {
        int unit, kt, end;  // none left: unit >= units
        const int8_t* w;    // of the k-tile
        uint32_t xoff[XR / 8], soff;
    };
    auto begin = [&](Stream& it, int unit) __attribute__((always_inline)) {
        it.unit = unit;
        it.kt = it.end = 0;
        if (unit >= units) return;
        const int tile = unit >> log, part = unit & ((1 << log) - 1);
        it.kt = (KT * part) >> log;
        it.end = (KT * (part + 1)) >> log;
        const int first = s.first[tile], rows = s.first[tile + 1] - first;
        const int expert = __builtin_amdgcn_readfirstlane(s.ids[s.sorted[first]]);
        it.w = uniform(down + ((size_t)expert * H + n0) * I);
#pragma unroll
        for (int i = 0; i < XR / 8; ++i) {
            const int r = 8 * i + lane / 8;
            it.xoff[i] = (uint32_t)s.sorted[first + min(r, rows - 1)] * (uint32_t)I + 16u * copied_chunk(r);
        }
        it.soff = (uint32_t)s.sorted[first + min(lane / 2 % XR, rows - 1)] * (uint32_t)groups;
    };
    uint32_t woff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) woff[i] = (uint32_t)(8 * i + lane / 8) * (uint32_t)I + 16u * copied_chunk(8 * i + lane / 8);
    char* ring = smem + wave * R * S::kStage;
    const uint32_t ring_lds = lds_addr(ring);
    auto issue = [&](Stream& it, int slot) __attribute__((always_inline)) {
        const bool there = it.unit < units;
        const uint32_t lds = ring_lds + (uint32_t)(slot * S::kStage);
        const int left = I - it.kt * 128;
        const int8_t* w = there ? it.w + it.kt * 128 : down;
        const int8_t* x = there ? hq + it.kt * 128 : hq;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            copy_weights<kOnce>(there ? woff[i] - past_end(copied_chunk(8 * i + lane / 8), left) : 0, w, lds + 1024 * i);
#pragma unroll
        for (int i = 0; i < XR / 8; ++i)
            dma16(there ? it.xoff[i] - past_end(copied_chunk(8 * i + lane / 8), left) : 0, x, lds + 2048 + 1024 * i);
        dma4(there ? 4 * (it.soff + (uint32_t)min(2 * it.kt + (lane & 1), groups - 1)) : 0, hscale, lds + S::kScales);
        if (there && ++it.kt == it.end) begin(it, it.unit + kDownWaves);
    };

    Stream ahead, now;
    begin(ahead, wave);
    begin(now, wave);
#pragma unroll
    for (int t = 0; t < R - 1; ++t) issue(ahead, t);
    int slot = 0, next = R - 1;
    float acc[4] = {0, 0, 0, 0};
    while (now.unit < units) {
        issue(ahead, next);
        wait_vm<(R - 1) * C>();
        const char* w = ring + slot * S::kStage;
        const int chunks = (I - now.kt * 128) / 16;
        const float2 b = *reinterpret_cast<const float2*>(w + S::kScales + 8 * (l16 % XR));
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            i32x4_t x = fragment(w + 2048, l16 % XR, 4 * ks + kg);
            if (4 * ks + kg >= chunks) x = i32x4_t{0, 0, 0, 0};
            const i32x4_t sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(fragment(w, l16, 4 * ks + kg), x, i32x4_t{0, 0, 0, 0}, 0, 0, 0);
            // (a group past the last has no chunks: its scale, the last one's, meets a sum of zero)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf((float)sum[i], ks == 0 ? b.x : b.y, acc[i]);
        }
        reads_done();
        slot = slot + 1 == R ? 0 : slot + 1;
        next = next + 1 == R ? 0 : next + 1;
        if (++now.kt == now.end) {
            const int tile = now.unit >> log, part = now.unit & ((1 << log) - 1);
            const int first = s.first[tile], rows = s.first[tile + 1] - first;
            if (l16 < rows) sums[part * P + s.sorted[first + l16]][kg] = make_float4(acc[0], acc[1], acc[2], acc[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = 0.0f;
            now.unit += kDownWaves;
            if (now.unit < units) {
                const int p = now.unit & ((1 << log) - 1);
                now.kt = (KT * p) >> log;
                now.end = (KT * (p + 1)) >> log;
            }
        }
    }
    wait_vm<0>();
    __syncthreads();
    const int t = threadIdx.x / 16, c = threadIdx.x % 16;
    if (t >= T) return;
    const float* part_sums = reinterpret_cast<const float*>(sums);
    float out = 0.0f;
    for (int j = 0; j < topk; ++j) {
        const int p = t * topk + j, e = s.ids[p];
        if (e == INT32_MAX) continue;
        float o = part_sums[p * 16 + c];
        for (int i = 1; i < 1 << log; ++i) o += part_sums[(i * P + p) * 16 + c];
        out = __builtin_fmaf(weights[p], o * down_scales[(size_t)e * H + n0 + c], out);
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
    auto run = [&](auto id, auto xr, auto ks, auto once) {
        using TI = decltype(id);
        constexpr int XR = decltype(xr)::value, KS = decltype(ks)::value;
        constexpr bool kOnce = decltype(once)::value;
        const TI* idt = static_cast<const TI*>(ids);
        hipLaunchKernelGGL((layer_up_kernel<TI, XR, KS, kOnce>), dim3((unsigned)(expert_tiles(P, E, XR) * groups)), dim3(256 * KS), 0,
                           stream, xq, ascale, idt, (int)P, (int)topk, (int)E, up, up_scales, (int)H, (int)I, (int)groups, hq, hscale);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        return with_act_type(dtype, [&](auto t) {
            using TO = decltype(t);
            hipLaunchKernelGGL((layer_down_kernel<TO, TI, XR, kOnce>), dim3((unsigned)(H / 16)), dim3(64 * kDownWaves), 0, stream, hq,
                               hscale, idt, (int)T, (int)topk, weights, (int)E, down, down_scales, (int)H, (int)I, (int)groups,
                               static_cast<TO*>(y));
            return hipGetLastError();
        });
    };
    const double weight_bytes = 3.0 * (double)std::min(P, E) * (double)H * (double)I;
    auto with_once = [&](auto id, auto xr, auto ks) {
        return weight_bytes >= kOnceBytes ? run(id, xr, ks, std::true_type{}) : run(id, xr, ks, std::false_type{});
    };
    auto with_ks = [&](auto id, auto xr) {
        const bool few = std::min(P, E) * groups < 512;
        return few ? with_once(id, xr, std::integral_constant<int, 2>{}) : with_once(id, xr, std::integral_constant<int, 1>{});
    };
    auto with_rows = [&](auto id) {
        return T <= 8 || P <= 4 * E ? with_ks(id, std::integral_constant<int, 8>{}) : with_ks(id, std::integral_constant<int, 16>{});
    };
    return id_bits == 32 ? with_rows(int32_t{}) : with_rows(int64_t{});
}

}  // namespace w4a16

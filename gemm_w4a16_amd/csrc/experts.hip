// experts.hip -- tokens sorted by expert and back: the row movers around the experts' products.
//
// A router gives each of T tokens `topk` experts; pair p = t * topk + j is token t's j-th choice.
//   sort      off_e = #{p : id_p < e}, pos_p = off_{id_p} + #{p' < p : id_p' = id_p}; -1 for an id
//             outside [0, E)
//   gather    xs[pos_tj] = x_t, as it is or quantized to int8
//   combine   y_t = sum_j w_tj ys[pos_tj], in order of j, in fp32
//   backward  dys[pos_tj] = w_tj dy_t, dw_tj = sum_n dy_t[n] ys[pos_tj][n]
// combine without weights is the gather's gradient.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "experts.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;

// ---- sort ---------------------------------------------------------------------------------------
// A counting sort.  Keys are the ids, with every id outside [0, E) as key E.  A block takes a run of
// consecutive pairs and each of its waves a run of those, 64 at a time in order, so that a pair's rank
// among its key is (pairs of the key in earlier blocks) + (in earlier waves) + (in this wave so far) +
// (in lower lanes).  Counts are integers: no order of the additions changes them.
// Up to kSortOneBlock pairs one block does all; more take a launch that counts and one that places, each
// block adding up the others' counts for itself.  Latency bounds it (the ids are read once or twice, 4 bytes
// a pair): 2.5 us for 8 pairs, 3.6 for 1024, 6.8 for 4096 in one block; 6.1 for 8192 and 7.4 for 65536 over 64
// experts in two launches (one block took 10.8 us for 8192).  The counts' LDS atomics cost little where one expert
// takes all: 524288 pairs over 64 experts 13.4 us evenly, 14.6 so.

template <typename TI>
__device__ __forceinline__ int sort_key(const TI* ids, int64_t p, int64_t P, int E) {
    if (p >= P) return E + 1;  // past the end: no key
    const TI id = ids[p];
    return id >= 0 && id < (TI)E ? (int)id : E;
}

// Lanes of the wave with the same key.
__device__ __forceinline__ uint64_t same_key(int key, int bits) {
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((key >> b) & 1);
        same &= (key >> b) & 1 ? set : ~set;
    }
    return same;
}

// Pairs per key of this block's run, into ws[block][E + 1].
template <typename TI>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const TI* __restrict__ ids, int64_t P, int E, int64_t run,
                                                                  int32_t* __restrict__ ws) {
    extern __shared__ int32_t lds[];
    for (int e = threadIdx.x; e <= E; e += kSortThreads) lds[e] = 0;
    __syncthreads();
    const int64_t p0 = blockIdx.x * run, p1 = min(p0 + run, P);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kSortThreads) atomicAdd(&lds[sort_key(ids, p, P, E)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kSortThreads) ws[(size_t)blockIdx.x * (E + 1) + e] = lds[e];
}

// Ranks and output.  kBlocks: the run is one of several, whose counts are in ws.  kPer > 0: the run is at most kPer
// pairs a thread, whose keys and ranks stay in registers; else a wave walks its pairs twice.
template <typename TI, bool kBlocks, int kPer>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const TI* __restrict__ ids, int64_t P, int E, int64_t run,
                                                                  const int32_t* __restrict__ ws, int bits,
                                                                  int32_t* __restrict__ offsets, int32_t* __restrict__ pos,
                                                                  int32_t* __restrict__ src) {
    extern __shared__ int32_t lds[];
    const int keys = E + 1;
    int32_t* cnt = lds;                        // [kSortWaves][keys] counts, then the next rows
    int32_t* sums = lds + kSortWaves * keys;   // [kSortWaves]
    int32_t* all = sums + kSortWaves;          // [2][keys] pairs in all blocks, and in the blocks before (kBlocks)
    const int t = threadIdx.x, lane = lane_id(), wave = wave_id();
    const int64_t p0 = blockIdx.x * run;
    const int64_t wrun = run / kSortWaves;  // a multiple of 64
    const int64_t w0 = p0 + wave * wrun, w1 = min(w0 + wrun, P);
    int32_t* mine = cnt + wave * keys;

    for (int i = t; i < (kSortWaves + (kBlocks ? 2 : 0)) * keys + kSortWaves; i += kSortThreads) cnt[i] = 0;
    int key[kPer > 0 ? kPer : 1], rank[kPer > 0 ? kPer : 1];
    if constexpr (kPer > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) key[i] = sort_key(ids, w0 + kWave * i + lane, w1, E);
    }
    __syncthreads();

    // a chunk of 64 pairs: a pair's rank among its key in this wave so far, counting it
    auto rank_chunk = [&](int64_t p, int key) __attribute__((always_inline)) {
        const uint64_t same = same_key(key, bits);
        const int below = __popcll(same & ((1ull << lane) - 1));
        int rank = 0;
        if (p < w1) {
            rank = mine[key] + below;
            wave_lds_sync();
            if (below == 0) mine[key] = rank + __popcll(same);
        }
        wave_lds_sync();
        return rank;
    };
    if constexpr (kPer > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (w0 + kWave * i < w1) rank[i] = rank_chunk(w0 + kWave * i + lane, key[i]);
    } else {
        for (int64_t p = w0 + lane; p < w1; p += kWave) atomicAdd(&mine[sort_key(ids, p, P, E)], 1);
    }
    if constexpr (kBlocks) {  // the blocks' counts, over all threads
        const int rows = kSortThreads / keys, r = t / keys, e = t % keys;  // keys <= kMaxExperts + 1 < kSortThreads
        if (r < rows) {
            int total = 0, before = 0;
            for (int b = r; b < (int)gridDim.x; b += rows) {
                const int c = ws[(size_t)b * keys + e];
                total += c;
                if (b < (int)blockIdx.x) before += c;
            }
            atomicAdd(&all[e], total);
            atomicAdd(&all[keys + e], before);
        }
    }
    __syncthreads();
    // first rows of every (wave, key): one key per thread
    static_assert(kMaxExperts < kSortThreads, "a thread per key");
    int c[kSortWaves] = {}, total = 0;
    if (t < keys) {
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) c[w] = cnt[w * keys + t];
        if constexpr (kBlocks) {
            total = all[t];
        } else {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) total += c[w];
        }
    }
    int end = total;  // inclusive sum over the keys
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int v = __shfl_up(end, off);
        if (lane >= off) end += v;
    }
    if (lane == kWave - 1) sums[wave] = end;
    __syncthreads();
    if (t < keys) {
        int next = end - total;
        for (int w = 0; w < wave; ++w) next += sums[w];
        if (blockIdx.x == 0) offsets[t] = next;  // key E's first row is offsets[E]
        if constexpr (kBlocks) next += all[keys + t];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            cnt[w * keys + t] = next;
            next += c[w];
        }
    }
    __syncthreads();
    auto place = [&](int64_t p, int key, int row) __attribute__((always_inline)) {
        pos[p] = key < E ? row : -1;
        if (src != nullptr) src[row] = key < E ? (int32_t)p : -1;
    };
    if constexpr (kPer > 0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t p = w0 + kWave * i + lane;
            if (p < w1) place(p, key[i], mine[key[i]] + rank[i]);
        }
    } else {
        for (int64_t p = w0 + lane; p - lane < w1; p += kWave) {
            const int key = p < w1 ? sort_key(ids, p, P, E) : keys;
            const int row = rank_chunk(p, key);  // (mine holds the next rows now)
            if (p < w1) place(p, key, row);
        }
    }
}

// ---- row movers -----------------------------------------------------------------------------------

// A pair's sorted row, or -1: nothing outside [0, P) is followed.
__device__ __forceinline__ int64_t pair_row(const int32_t* pos, int64_t p, int64_t P) {
    const int r = pos[p];
    return r >= 0 && r < P ? r : -1;
}

// The token and unit of a row (16 bytes, or one element) that a thread moves: a block takes 256 units of a row,
// or (kShort) `tokens` whole rows where a row has at most 64.
struct RowShape {
    int width, units, tokens, blocks_per_row;  // width: elements
};
// A unit's first element.  kRagged: rows are not whole units, so units start at any element, and a row's last one is
// moved back to end with the row: its first elements are the unit's before it too.  (4096 tokens of 2 rows of 4098 bf16:
// gather 17 us against 59 by element, combine 19 against 62, backward 37 against 55; 333 of 3 rows of 1001 fp16 2.6
// against 3.3, 2.8 against 3.7, 4.3 against 6.2.)
template <int V, bool kRagged>
__device__ __forceinline__ int unit_at(int c, int width) {
    return kRagged ? min(V * c, width - V) : V * c;
}
template <bool kShort>
__device__ __forceinline__ bool row_place(const RowShape& s, int64_t b, int64_t Tn, int64_t& t, int& c) {
    if constexpr (kShort) {
        const int i = threadIdx.x / s.units;
        t = b * s.tokens + i, c = threadIdx.x - i * s.units;
        return i < s.tokens && t < Tn;
    } else {
        t = b / s.blocks_per_row, c = (int)(b - t * s.blocks_per_row) * 256 + threadIdx.x;
        return c < s.units;
    }
}

// xs[pos_tj] = x_t.  A unit is read once and stored for each of the token's pairs, so the writes bound it: 8192 tokens
// of 8 rows of 2048 bf16 (0.30 GB) take 47 us, 6.4 TB/s over what is read and written; four tokens of 2 rows
// of 4096 2.5 us, an empty launch's 1.7 and two loads' latency.
template <typename T, int V, bool kRagged, bool kStream, bool kShort>
__global__ __launch_bounds__(256) void gather_kernel(const T* __restrict__ x, int64_t Tn, int topk,
                                                     const int32_t* __restrict__ pos, RowShape s, int64_t blocks,
                                                     T* __restrict__ xs) {
    const int64_t P = Tn * topk;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        int64_t t;
        int c;
        if (!row_place<kShort>(s, b, Tn, t, c)) continue;
        const int at = unit_at<V, kRagged>(c, s.width);
        const Pack<T, V> v = load_unit<false, kRagged, V>(x + t * s.width + at);
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pair_row(pos, t * topk + j, P);
            if (r >= 0) store_unit<kStream, kRagged>(xs + r * s.width + at, v);
        }
    }
}

// The same, quantized on the way: a row is read and quantized once and its codes are stored for each pair.  kWaves
// waves per token, as in the quantizer.  4096 tokens of 2 rows of 4096 bf16 take 16.0 us (4.2 TB/s), 8192 of 8
// rows of 2048 36 us (4.6 TB/s), 200 of 8 rows of 2048 4.3 us.
template <typename T, int kWaves>
__global__ __launch_bounds__(256) void gather_i8_kernel(const T* __restrict__ x, int64_t Tn, int topk,
                                                        const int32_t* __restrict__ pos, int K, int8_t* __restrict__ xq,
                                                        float* __restrict__ ascale) {
    constexpr int kTokens = 4 / kWaves, kThreads = 64 * kWaves;
    __shared__ uint32_t red[4];
    __shared__ int32_t all_rows[kTokens][kMaxExperts];  // a token's, fetched beside its activations (topk <= kMaxExperts)
    const int64_t P = Tn * topk;
    const int tid = threadIdx.x % kThreads;
    int32_t* rows = all_rows[threadIdx.x / kThreads];
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < Tn; t0 += (int64_t)gridDim.x * kTokens) {
        const int64_t t = kWaves == 1 ? t0 + wave_id() : t0;
        if (kWaves == 1 && t >= Tn) continue;
        if constexpr (kWaves > 1) __syncthreads();  // rows may still be read
        for (int j = tid; j < topk; j += kThreads) rows[j] = (int32_t)pair_row(pos, t * topk + j, P);
        if constexpr (kWaves == 1) wave_lds_sync();
        const float a = quantize_row<kThreads>(x + t * K, K, red, [&](int c, uint4 q) __attribute__((always_inline)) {
            for (int j = 0; j < topk; ++j)
                if (rows[j] >= 0) *reinterpret_cast<uint4*>(xq + (int64_t)rows[j] * K + 16 * c) = q;
        });
        for (int j = tid; j < topk; j += kThreads)
            if (rows[j] >= 0) ascale[rows[j]] = a;
        if constexpr (kWaves == 1) wave_lds_sync();
    }
}

// The rows of kAhead pairs from j0 on, one unit of each: all requested before the first is used (a pair with no
// row reads row 0 and is left out).
template <bool kStream, bool kRagged, int kAhead, typename T, int V>
__device__ __forceinline__ void load_pairs(const T* ys, const int32_t* pos, int64_t t, int topk, int j0, int64_t P, int width,
                                           int at, Pack<T, V> (&v)[kAhead], int64_t (&row)[kAhead]) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        row[i] = j0 + i < topk ? pair_row(pos, t * topk + j0 + i, P) : -1;
        v[i] = load_unit<kStream, kRagged, V>(ys + max(row[i], (int64_t)0) * width + at);
    }
}

// y_t = sum_j w_tj ys[pos_tj] in fp32, in order of j.  A thread owns one unit of y and reads that unit of every pair's
// row, so nothing is joined and the reads bound it: 4096 tokens of 2 rows of 4096 bf16 (0.10 GB) take 17 us (5.8
// TB/s), of 8 rows of 2048 (0.15 GB) 25 us (5.9 TB/s).
template <typename T, int V, bool kRagged, int kAhead, bool kStream, bool kShort>
__global__ __launch_bounds__(256) void combine_kernel(const T* __restrict__ ys, int64_t Tn, int topk,
                                                      const int32_t* __restrict__ pos, const float* __restrict__ weights,
                                                      RowShape s, int64_t blocks, T* __restrict__ y) {
    using U = Pack<T, V>;
    const int64_t P = Tn * topk;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        int64_t t;
        int c;
        if (!row_place<kShort>(s, b, Tn, t, c)) continue;
        const int at = unit_at<V, kRagged>(c, s.width);
        float acc[V] = {};
        for (int j0 = 0; j0 < topk; j0 += kAhead) {
            U v[kAhead];
            int64_t row[kAhead];
            load_pairs<kStream, kRagged>(ys, pos, t, topk, j0, P, s.width, at, v, row);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (row[i] >= 0) {
                    const float w = weights != nullptr ? weights[t * topk + j0 + i] : 1.0f;
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = __builtin_fmaf(w, to_f32(v[i].v[k]), acc[k]);
                }
        }
        U o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(acc[i]);
        store_unit<kStream, kRagged>(y + t * s.width + at, o);
    }
}

// Pairs that the backward takes at a time: two (one, four and eight took 66, 50 and 50 us against 51 at 4096 tokens of
// 8 rows of 2048 bf16, 31, 32 and 38 against 29 at 4096 of 2 rows of 4096, and 5.5, 5.2 and 6.0 against 4.2 at 333
// of 3 rows of 1000: more rows in flight cost registers, and so waves).
constexpr int kBackwardAhead = 2;

// dys[pos_tj] = w_tj dy_t and dw_tj = <dy_t, ys[pos_tj]> in one pass over ys and dys.  kWaves waves per token (one, four
// tokens a block, for short rows); kAhead pairs at a time.  A thread's partial dot products are summed over
// the wave, then over the waves, in a fixed order.  Its bytes bound it: 4096 tokens of 8 rows of 2048 bf16 (0.29
// GB) take 51 us (5.6 TB/s).
template <typename T, int V, bool kRagged, int kAhead, int kWaves, bool kStream>
__global__ __launch_bounds__(256) void combine_backward_kernel(const T* __restrict__ dy, const T* __restrict__ ys, int64_t Tn,
                                                               int topk, const int32_t* __restrict__ pos,
                                                               const float* __restrict__ weights, int units, int width,
                                                               T* __restrict__ dys, float* __restrict__ dweights) {
    using U = Pack<T, V>;
    constexpr int kTokens = 4 / kWaves, kThreads = kWave * kWaves;
    __shared__ float red[4][kAhead];
    const int64_t P = Tn * topk;
    const int lane = threadIdx.x % kThreads;
    for (int64_t b = blockIdx.x; b * kTokens < Tn; b += gridDim.x) {
        const int64_t t = kWaves > 1 ? b : b * kTokens + wave_id();
        if (kWaves == 1 && t >= Tn) continue;
        for (int j0 = 0; j0 < topk; j0 += kAhead) {
            float dot[kAhead] = {};
            for (int c = lane; c < units; c += kThreads) {
                const int at = unit_at<V, kRagged>(c, width), seen = V * c - at;  // (the unit before has its first `seen`)
                const U g = load_unit<false, kRagged, V>(dy + t * width + at);
                U v[kAhead];
                int64_t row[kAhead];
                if (dweights != nullptr) {
                    load_pairs<kStream, kRagged>(ys, pos, t, topk, j0, P, width, at, v, row);
                } else {
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) row[i] = j0 + i < topk ? pair_row(pos, t * topk + j0 + i, P) : -1;
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (row[i] < 0) continue;
                    if (dweights != nullptr) {
#pragma unroll
                        for (int k = 0; k < V; ++k)
                            if (!kRagged || k >= seen) dot[i] = __builtin_fmaf(to_f32(g.v[k]), to_f32(v[i].v[k]), dot[i]);
                    }
                    if (dys != nullptr) {
                        const float w = weights != nullptr ? weights[t * topk + j0 + i] : 1.0f;
                        U o;
#pragma unroll
                        for (int k = 0; k < V; ++k) o.v[k] = from_f32<T>(w * to_f32(g.v[k]));
                        store_unit<kStream, kRagged>(dys + row[i] * width + at, o);
                    }
                }
            }
            if (dweights == nullptr) continue;
            if constexpr (kWaves > 1) __syncthreads();  // red may still be read
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const float sum = wave_sum(dot[i]);
                if (lane_id() == 0) red[wave_id()][i] = sum;
            }
            if constexpr (kWaves > 1)
                __syncthreads();
            else
                wave_lds_sync();
            if (lane < kAhead && j0 + lane < topk) {
                float sum = red[wave_id()][lane];
                if constexpr (kWaves > 1) sum = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
                dweights[t * topk + j0 + lane] = sum;
            }
            if constexpr (kWaves == 1) wave_lds_sync();
        }
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
dim3 row_grid(int64_t blocks) { return dim3((unsigned)std::min<int64_t>(blocks, kMaxGridBlocks)); }

}  // namespace

// ---- host ---------------------------------------------------------------------------------------

// Pairs a block sorts: all of them up to kSortOneBlock, else enough for at most 256 blocks.
static int64_t sort_run(int64_t P) {
    if (P <= kSortOneBlock) return ceil_div(P, kSortThreads) * kSortThreads;
    return std::max<int64_t>(kSortThreads, ceil_div(ceil_div(P, 256), kSortThreads) * kSortThreads);
}

size_t expert_sort_workspace_bytes(int64_t P, int64_t E) {
    return P <= kSortOneBlock ? 0 : (size_t)ceil_div(P, sort_run(P)) * (size_t)(E + 1) * 4;
}

template <typename TI>
static hipError_t launch_sort(const TI* ids, int64_t P, int E, int32_t* offsets, int32_t* pos, int32_t* src, int32_t* ws,
                              hipStream_t stream) {
    const int64_t run = sort_run(P);
    const dim3 grid((unsigned)ceil_div(P, run));
    int bits = 1;  // keys 0..E + 1
    while ((E + 1) >> bits) ++bits;
    auto place = [&](auto blocks, auto per) {
        constexpr bool kBlocks = decltype(blocks)::value;
        constexpr int kPer = decltype(per)::value;
        const size_t lds = (size_t)((kSortWaves + (kBlocks ? 2 : 0)) * (E + 1) + kSortWaves) * 4;
        hipLaunchKernelGGL((sort_place_kernel<TI, kBlocks, kPer>), grid, dim3(kSortThreads), lds, stream, ids, P, E, run, ws,
                           bits, offsets, pos, src);
        return hipGetLastError();
    };
    using std::false_type;
    using std::integral_constant;
    using std::true_type;
    constexpr int kPerBlock = kSortOneBlock / kSortThreads;
    if (P <= kSortThreads) return place(false_type{}, integral_constant<int, 1>{});
    if (P <= kSortOneBlock) return place(false_type{}, integral_constant<int, kPerBlock>{});
    hipLaunchKernelGGL((sort_count_kernel<TI>), grid, dim3(kSortThreads), (E + 1) * 4, stream, ids, P, E, run, ws);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    return run == kSortThreads ? place(true_type{}, integral_constant<int, 1>{}) : place(true_type{}, integral_constant<int, 0>{});
}

hipError_t launch_expert_sort(const void* ids, int id_bits, int64_t P, int64_t E, int32_t* offsets, int32_t* pos,
                              int32_t* src, int32_t* ws, hipStream_t stream) {
    if (id_bits == 64) return launch_sort(static_cast<const int64_t*>(ids), P, (int)E, offsets, pos, src, ws, stream);
    return launch_sort(static_cast<const int32_t*>(ids), P, (int)E, offsets, pos, src, ws, stream);
}

// Arrays of sorted rows from this size on are streamed (more than the L2s hold, 8 x 4 MiB): 4096 tokens of 2 rows of
// 8 KiB are gathered in 16.1 us against 20.5, 333 of 3 rows of 2 KB in 2.8 against 2.5.  Rows that are not whole
// units, whose ends share lines, from twice that: 4096 tokens of 2 rows of 4098 bf16 17.4 against 19.5, 6000 of 7
// rows of 609 fp16 (49 MiB) 16.7 against 12.1.
static bool streams(int64_t rows, int64_t row_bytes, bool ragged) {
    return rows * row_bytes >= ((int64_t)(ragged ? 64 : 32) << 20);
}

static RowShape row_shape(int64_t width, int64_t units) {
    return RowShape{(int)width, (int)units, units <= 64 ? (int)(256 / units) : 1, (int)ceil_div(units, 256)};
}
static int64_t row_blocks(const RowShape& s, int64_t T) { return s.tokens > 1 ? ceil_div(T, s.tokens) : T * s.blocks_per_row; }

// f(an element, the elements of a unit, whether a row is not whole units, whether rows are streamed) as constants.
// Rows shorter than a unit go by element.
template <typename E, typename F>
static hipError_t with_row_unit(E t, int64_t T, int64_t topk, int64_t N, F f) {
    using std::false_type;
    using std::integral_constant;
    using std::true_type;
    constexpr int V = 16 / sizeof(E);
    if (N < V) return f(t, integral_constant<int, 1>{}, false_type{}, false_type{});
    const bool ragged = N % V != 0, stream = streams(T * topk, N * sizeof(E), ragged);
    auto run = [&](auto r) {
        return stream ? f(t, integral_constant<int, V>{}, r, true_type{}) : f(t, integral_constant<int, V>{}, r, false_type{});
    };
    return ragged ? run(true_type{}) : run(false_type{});
}

hipError_t launch_expert_gather(int dtype, const void* x, int64_t T, int64_t topk, const int32_t* pos, int64_t K, void* xs,
                                hipStream_t stream) {
    auto run = [&](auto t, auto v, auto ragged, auto stream_rows) {
        using E = decltype(t);
        constexpr int V = decltype(v)::value;
        const RowShape s = row_shape(K, ceil_div(K, V));
        const int64_t blocks = row_blocks(s, T);
        auto launch = [&](auto is_short) {
            hipLaunchKernelGGL((gather_kernel<E, V, decltype(ragged)::value, decltype(stream_rows)::value,
                                              decltype(is_short)::value>),
                               row_grid(blocks), dim3(256), 0, stream, static_cast<const E*>(x), T, (int)topk, pos, s, blocks,
                               static_cast<E*>(xs));
            return hipGetLastError();
        };
        return s.tokens > 1 ? launch(std::true_type{}) : launch(std::false_type{});
    };
    return dtype == 2 ? with_row_unit(uint32_t{}, T, topk, K, run) : with_row_unit(uint16_t{}, T, topk, K, run);
}

hipError_t launch_expert_gather_i8(int dtype, const void* x, int64_t T, int64_t topk, const int32_t* pos, int64_t K,
                                   int8_t* xq, float* ascale, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using E = decltype(t);
        auto run = [&](auto waves) {
            constexpr int kWaves = decltype(waves)::value;
            hipLaunchKernelGGL((gather_i8_kernel<E, kWaves>), row_grid(ceil_div(T, 4 / kWaves)), dim3(256), 0, stream,
                               static_cast<const E*>(x), T, (int)topk, pos, (int)K, xq, ascale);
            return hipGetLastError();
        };
        return row_by_wave(T, K) ? run(std::integral_constant<int, 1>{}) : run(std::integral_constant<int, 4>{});
    });
}

hipError_t launch_expert_combine(int dtype, const void* ys, int64_t T, int64_t topk, const int32_t* pos,
                                 const float* weights, int64_t N, void* y, hipStream_t stream) {
    auto run = [&](auto t, auto v, auto ragged, auto stream_rows) {
        using E = decltype(t);
        constexpr int V = decltype(v)::value;
        const RowShape s = row_shape(N, ceil_div(N, V));
        const int64_t blocks = row_blocks(s, T);
        auto launch = [&](auto ahead, auto is_short) {
            hipLaunchKernelGGL((combine_kernel<E, V, decltype(ragged)::value, decltype(ahead)::value,
                                               decltype(stream_rows)::value, decltype(is_short)::value>),
                               row_grid(blocks), dim3(256), 0, stream, static_cast<const E*>(ys), T, (int)topk, pos, weights, s,
                               blocks, static_cast<E*>(y));
            return hipGetLastError();
        };
        using std::integral_constant;  // (eight pairs at a time take as long as four)
        auto pairs = [&](auto is_short) {
            return topk <= 2 ? launch(integral_constant<int, 2>{}, is_short) : launch(integral_constant<int, 4>{}, is_short);
        };
        return s.tokens > 1 ? pairs(std::true_type{}) : pairs(std::false_type{});
    };
    return with_act_type(dtype, [&](auto t) { return with_row_unit(t, T, topk, N, run); });
}

hipError_t launch_expert_combine_backward(int dtype, const void* dy, const void* ys, int64_t T, int64_t topk,
                                          const int32_t* pos, const float* weights, int64_t N, void* dys, float* dweights,
                                          hipStream_t stream) {
    auto run = [&](auto t, auto v, auto ragged, auto stream_rows) {
        using E = decltype(t);
        constexpr int V = decltype(v)::value;
        constexpr bool kRagged = decltype(ragged)::value, kStream = decltype(stream_rows)::value;
        const int64_t units = ceil_div(N, V);
        auto launch = [&](auto waves) {
            constexpr int kWaves = decltype(waves)::value;
            hipLaunchKernelGGL((combine_backward_kernel<E, V, kRagged, kBackwardAhead, kWaves, kStream>),
                               row_grid(ceil_div(T, 4 / kWaves)),
                               dim3(256), 0, stream, static_cast<const E*>(dy), static_cast<const E*>(ys), T, (int)topk, pos,
                               weights, (int)units, (int)N, static_cast<E*>(dys), dweights);
            return hipGetLastError();
        };
        return units <= 64 ? launch(std::integral_constant<int, 1>{}) : launch(std::integral_constant<int, 4>{});
    };
    // Rows that a wave's lanes hold by element: 60000 tokens of 4 rows of 64 fp16 28 us against 34, of 63 fp32 46 against
    // 57 (but of 64 fp32, whole units, 40 against 37).
    return with_act_type(dtype, [&](auto t) {
        if (N <= kWave && (sizeof(t) == 2 || N % (16 / sizeof(t)) != 0))
            return run(t, std::integral_constant<int, 1>{}, std::false_type{}, std::false_type{});
        return with_row_unit(t, T, topk, N, run);
    });
}

}  // namespace w4a16

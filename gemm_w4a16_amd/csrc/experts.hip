// experts.hip -- tokens sorted by expert and back: the row movers around the experts' products.
//
// A router gives each of T tokens `topk` experts; pair p = t * topk + j is token t's j-th choice.
//   sort      off_e = #{p : id_p < e}, pos_p = off_{id_p} + #{p' < p : id_p' = id_p}; -1 for an id
//             outside [0, E)
//   gather    xs[pos_tj] = x_t, as it is or quantized to int8
//   combine   y_t = sum_j w_tj ys[pos_tj], in order of j, in fp32
//   backward  dys[pos_tj] = w_tj dy_t, dw_tj = sum_n dy_t[n] ys[pos_tj][n]
// combine without weights is the gather's gradient.
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

// Ranks and output.  ws: the blocks' counts (null where there is one block).
template <typename TI>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const TI* __restrict__ ids, int64_t P, int E, int64_t run,
                                                                  const int32_t* __restrict__ ws, int bits,
                                                                  int32_t* __restrict__ offsets, int32_t* __restrict__ pos,
                                                                  int32_t* __restrict__ src) {
    extern __shared__ int32_t lds[];  // [kSortWaves][E + 1] counts, then next rows; [kSortWaves] sums
    int32_t* cnt = lds;
    int32_t* sums = lds + kSortWaves * (E + 1);
    const int t = threadIdx.x, lane = lane_id(), wave = wave_id();
    for (int i = t; i < kSortWaves * (E + 1); i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int64_t p0 = blockIdx.x * run;
    const int64_t wrun = run / kSortWaves;  // a multiple of 64
    const int64_t w0 = p0 + wave * wrun, w1 = min(w0 + wrun, P);
    for (int64_t p = w0 + lane; p < w1; p += kWave) atomicAdd(&cnt[wave * (E + 1) + sort_key(ids, p, P, E)], 1);
    __syncthreads();
    // first rows of every (wave, key): keys 0..E, one per thread
    static_assert(kMaxExperts < kSortThreads, "a thread per key");
    {
        const int e = t;
        int total = 0, before = 0;
        if (e <= E) {
            if (ws != nullptr) {
                for (int b = 0; b < (int)gridDim.x; ++b) {
                    const int c = ws[(size_t)b * (E + 1) + e];
                    total += c;
                    if (b < (int)blockIdx.x) before += c;
                }
            }
            int s = 0;
            for (int w = 0; w < kSortWaves; ++w) {
                const int c = cnt[w * (E + 1) + e];
                cnt[w * (E + 1) + e] = before + s;
                s += c;
            }
            if (ws == nullptr) total = s;
        }
        int end = total;  // inclusive sum over the block's keys
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int v = __shfl_up(end, off);
            if (lane >= off) end += v;
        }
        if (lane == kWave - 1) sums[wave] = end;
        __syncthreads();
        int base = 0;
        for (int w = 0; w < wave; ++w) base += sums[w];
        if (e <= E) {
            const int first = base + end - total;
            for (int w = 0; w < kSortWaves; ++w) cnt[w * (E + 1) + e] += first;
            if (blockIdx.x == 0) offsets[e] = first;  // key E's first row is offsets[E]
        }
    }
    __syncthreads();
    for (int64_t p = w0 + lane; p - lane < w1; p += kWave) {
        const int key = p < w1 ? sort_key(ids, p, P, E) : E + 1;
        const uint64_t same = same_key(key, bits);
        if (p < w1) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            int32_t* next = &cnt[wave * (E + 1) + key];
            const int row = *next + rank;
            wave_lds_sync();
            if (rank == 0) *next = row + __popcll(same);
            pos[p] = key < E ? row : -1;
            if (src != nullptr) src[row] = key < E ? (int32_t)p : -1;
        }
        wave_lds_sync();
    }
}

// ---- row movers -----------------------------------------------------------------------------------

// A pair's sorted row, or -1: nothing outside [0, P) is followed.
__device__ __forceinline__ int64_t pair_row(const int32_t* pos, int64_t p, int64_t P) {
    const int r = pos[p];
    return r >= 0 && r < P ? r : -1;
}

// One unit U (16 bytes, or one element) of a row per thread, stored once for each of the token's pairs.
template <typename U>
__global__ __launch_bounds__(256) void gather_kernel(const U* __restrict__ x, int64_t T, int topk,
                                                     const int32_t* __restrict__ pos, int units, int blocks_per_row,
                                                     U* __restrict__ xs) {
    const int64_t P = T * topk;
    for (int64_t b = blockIdx.x; b < T * blocks_per_row; b += gridDim.x) {
        const int64_t t = b / blocks_per_row;
        const int c = (int)(b % blocks_per_row) * 256 + threadIdx.x;
        if (c >= units) continue;
        const U v = x[t * units + c];
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pair_row(pos, t * topk + j, P);
            if (r >= 0) xs[r * units + c] = v;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void gather_i8_kernel(const T* __restrict__ x, int64_t Tn, int topk,
                                                        const int32_t* __restrict__ pos, int K, int8_t* __restrict__ xq,
                                                        float* __restrict__ ascale) {
    __shared__ uint32_t red[4];
    const int64_t P = Tn * topk;
    for (int64_t t = blockIdx.x; t < Tn; t += gridDim.x) {
        const T* row = x + t * K;
        const float a = row_scale_i8<256>(row, K, red);
        for (int j = threadIdx.x; j < topk; j += 256) {
            const int64_t r = pair_row(pos, t * topk + j, P);
            if (r >= 0) ascale[r] = a;
        }
        for (int c = threadIdx.x; c < K / 16; c += 256) {
            const uint4 q = quant16(row + 16 * c, a);
            for (int j = 0; j < topk; ++j) {
                const int64_t r = pair_row(pos, t * topk + j, P);
                if (r >= 0) *reinterpret_cast<uint4*>(xq + r * K + 16 * c) = q;
            }
        }
    }
}

template <typename T, int V>
__global__ __launch_bounds__(256) void combine_kernel(const T* __restrict__ ys, int64_t Tn, int topk,
                                                      const int32_t* __restrict__ pos, const float* __restrict__ weights,
                                                      int units, int blocks_per_row, T* __restrict__ y) {
    using U = Pack<T, V>;
    const int64_t P = Tn * topk;
    for (int64_t b = blockIdx.x; b < Tn * blocks_per_row; b += gridDim.x) {
        const int64_t t = b / blocks_per_row;
        const int c = (int)(b % blocks_per_row) * 256 + threadIdx.x;
        if (c >= units) continue;
        float acc[V] = {};
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pair_row(pos, t * topk + j, P);
            if (r < 0) continue;
            const float w = weights != nullptr ? weights[t * topk + j] : 1.0f;
            const U v = reinterpret_cast<const U*>(ys)[r * units + c];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w, to_f32(v.v[i]), acc[i]);
        }
        U o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(acc[i]);
        reinterpret_cast<U*>(y)[t * units + c] = o;
    }
}

// One block per token; a thread's partial dot products are summed over the block in a fixed order.
template <typename T, int V>
__global__ __launch_bounds__(256) void combine_backward_kernel(const T* __restrict__ dy, const T* __restrict__ ys, int64_t Tn,
                                                               int topk, const int32_t* __restrict__ pos,
                                                               const float* __restrict__ weights, int units,
                                                               T* __restrict__ dys, float* __restrict__ dweights) {
    using U = Pack<T, V>;
    __shared__ float red[4];
    const int64_t P = Tn * topk;
    for (int64_t t = blockIdx.x; t < Tn; t += gridDim.x) {
        for (int j = 0; j < topk; ++j) {
            const int64_t r = pair_row(pos, t * topk + j, P);
            const float w = weights != nullptr ? weights[t * topk + j] : 1.0f;
            float dot = 0.0f;
            if (r >= 0) {
                for (int c = threadIdx.x; c < units; c += 256) {
                    const U g = reinterpret_cast<const U*>(dy)[t * units + c];
                    if (dweights != nullptr) {
                        const U v = reinterpret_cast<const U*>(ys)[r * units + c];
#pragma unroll
                        for (int i = 0; i < V; ++i) dot = __builtin_fmaf(to_f32(g.v[i]), to_f32(v.v[i]), dot);
                    }
                    if (dys != nullptr) {
                        U o;
#pragma unroll
                        for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(w * to_f32(g.v[i]));
                        reinterpret_cast<U*>(dys)[r * units + c] = o;
                    }
                }
            }
            if (dweights != nullptr) {
                dot = wave_sum(dot);
                __syncthreads();
                if (lane_id() == 0) red[wave_id()] = dot;
                __syncthreads();
                if (threadIdx.x == 0) dweights[t * topk + j] = (red[0] + red[1]) + (red[2] + red[3]);
            }
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
    const size_t lds = (size_t)(kSortWaves * (E + 1) + kSortWaves) * 4;
    if (P > kSortOneBlock) {
        hipLaunchKernelGGL((sort_count_kernel<TI>), grid, dim3(kSortThreads), (E + 1) * 4, stream, ids, P, E, run, ws);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    } else {
        ws = nullptr;
    }
    hipLaunchKernelGGL((sort_place_kernel<TI>), grid, dim3(kSortThreads), lds, stream, ids, P, E, run, ws, bits, offsets, pos,
                       src);
    return hipGetLastError();
}

hipError_t launch_expert_sort(const void* ids, int id_bits, int64_t P, int64_t E, int32_t* offsets, int32_t* pos,
                              int32_t* src, int32_t* ws, hipStream_t stream) {
    if (id_bits == 64) return launch_sort(static_cast<const int64_t*>(ids), P, (int)E, offsets, pos, src, ws, stream);
    return launch_sort(static_cast<const int32_t*>(ids), P, (int)E, offsets, pos, src, ws, stream);
}

hipError_t launch_expert_gather(int dtype, const void* x, int64_t T, int64_t topk, const int32_t* pos, int64_t K, void* xs,
                                hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using E = decltype(t);
        auto run = [&](auto unit) {
            using U = decltype(unit);
            const int units = (int)(K * sizeof(E) / sizeof(U)), bpr = (int)ceil_div(units, 256);
            hipLaunchKernelGGL((gather_kernel<U>), row_grid(T * bpr), dim3(256), 0, stream, static_cast<const U*>(x), T,
                               (int)topk, pos, units, bpr, static_cast<U*>(xs));
            return hipGetLastError();
        };
        return K * sizeof(E) % 16 == 0 ? run(uint4{}) : run(E{});
    });
}

hipError_t launch_expert_gather_i8(int dtype, const void* x, int64_t T, int64_t topk, const int32_t* pos, int64_t K,
                                   int8_t* xq, float* ascale, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using E = decltype(t);
        hipLaunchKernelGGL((gather_i8_kernel<E>), row_grid(T), dim3(256), 0, stream, static_cast<const E*>(x), T, (int)topk,
                           pos, (int)K, xq, ascale);
        return hipGetLastError();
    });
}

template <typename F>
static hipError_t with_row_unit(int dtype, int64_t N, F f) {
    return with_act_type(dtype, [&](auto t) {
        using E = decltype(t);
        constexpr int V = 16 / sizeof(E);
        return N % V == 0 ? f(t, std::integral_constant<int, V>{}) : f(t, std::integral_constant<int, 1>{});
    });
}

hipError_t launch_expert_combine(int dtype, const void* ys, int64_t T, int64_t topk, const int32_t* pos,
                                 const float* weights, int64_t N, void* y, hipStream_t stream) {
    return with_row_unit(dtype, N, [&](auto t, auto v) {
        using E = decltype(t);
        constexpr int V = decltype(v)::value;
        const int units = (int)(N / V), bpr = (int)ceil_div(units, 256);
        hipLaunchKernelGGL((combine_kernel<E, V>), row_grid(T * bpr), dim3(256), 0, stream, static_cast<const E*>(ys), T,
                           (int)topk, pos, weights, units, bpr, static_cast<E*>(y));
        return hipGetLastError();
    });
}

hipError_t launch_expert_combine_backward(int dtype, const void* dy, const void* ys, int64_t T, int64_t topk,
                                          const int32_t* pos, const float* weights, int64_t N, void* dys, float* dweights,
                                          hipStream_t stream) {
    return with_row_unit(dtype, N, [&](auto t, auto v) {
        using E = decltype(t);
        constexpr int V = decltype(v)::value;
        hipLaunchKernelGGL((combine_backward_kernel<E, V>), row_grid(T), dim3(256), 0, stream, static_cast<const E*>(dy),
                           static_cast<const E*>(ys), T, (int)topk, pos, weights, (int)(N / V), static_cast<E*>(dys),
                           dweights);
        return hipGetLastError();
    });
}

}  // namespace w4a16

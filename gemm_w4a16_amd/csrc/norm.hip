// norm.hip -- RMS norm of rows with a residual added first, in the activations' type or in 8-bit integers with a
// scale per row (what the int8 products take), and its gradients.
//
// Row t of T, width N:  s = x + residual (fp32),  h = s rounded to the activations' type,
//     r = 1 / sqrt(sum_n s_n^2 / N + eps),   v_n = (s_n r) w_n   (fp32),   y = v rounded once;
// in 8 bits a = max|v| / 127, q = clamp(rint(v / a), -127, 127).  The norm is of the sum as it is in fp32, not of
// the rounded h: h is what goes on, and one rounding of y is enough.
// Gradients, of y = norm(h) for the h that was stored, which is all that a backward pass has of s (g = dy w, r from h):
//     dx = r (g - u sum_n(g u) / N) + dh,   dw_n = sum_t dy u,   u = h r:
// with u and not h r^2, whose factor leaves fp32's range long before dx does (r of 2^64 on).
//
// Bytes bound all of these for many rows, and a row's chain of loads and reductions for few.  A row stays in registers
// between its passes (kKeep units of 16 bytes a thread); what a long row has beyond that is read again, from the
// caches.  8192 x 4096 bf16 with a residual: in 8 bits 42 us (5.6 TB/s; a copy moves 5.1), in bf16 48, gradients 51 (5.3
// TB/s); one row in 8 bits 3.2 us, 1024 rows 10.  With a row's loads behind the row before instead of beside it, 59, 59
// and 89.
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "experts.h"
#include "launch.h"

namespace w4a16 {

namespace {

template <typename T>
constexpr int kUnit = 16 / (int)sizeof(T);

// Where eps leaves a row's factor to its squares (eps below kSmallEps) and these are next to fp32's smallest numbers
// (their sum below kSmallSum), the row is taken times kUp and eps times its square, exactly: then no square is below
// 2^-98, and none, nor their sum, past 2^120.  Above either bound what vanishes is below 2^-30 of the rest.  Kernels of their own
// (kTiny), since the others would lose registers to it (gradients of sixteen waves a row spilled up to 72).
constexpr float kSmallEps = 0x1p-110f, kSmallSum = 0x1p-80f, kUp = 0x1p100f;
__device__ __forceinline__ float factor(float ss, int N, float eps, float up) {
    return 1.0f / sqrtf(ss / (float)N + eps * up * up);
}

// Unit c of a row of N elements: elements past the row's end are zero.  kAny: rows start at any element; kStream: past
// the caches' usual order.
template <bool kStream, bool kAny, typename T>
__device__ __forceinline__ Pack<T, kUnit<T>> load_row_unit(const T* row, int c, int N) {
    constexpr int V = kUnit<T>;
    if (!kAny || (c + 1) * V <= N) return load_unit<kStream, kAny, V>(row + c * V);
    Pack<T, V> u;
#pragma unroll
    for (int j = 0; j < V; ++j) u.v[j] = c * V + j < N ? row[c * V + j] : from_f32<T>(0.0f);
    return u;
}
template <bool kStream, bool kAny, typename T>
__device__ __forceinline__ void store_row_unit(T* row, int c, int N, const float (&f)[kUnit<T>]) {
    constexpr int V = kUnit<T>;
    Pack<T, V> u;
#pragma unroll
    for (int j = 0; j < V; ++j) u.v[j] = from_f32<T>(f[j]);
    if (!kAny || (c + 1) * V <= N) {
        store_unit<kStream, kAny>(row + c * V, u);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c * V + j < N) row[c * V + j] = u.v[j];
    }
}
template <typename T, int V>
__device__ __forceinline__ void widen(const Pack<T, V>& u, float (&f)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = to_f32(u.v[j]);
}
template <typename T, int V>
__device__ __forceinline__ void add(const Pack<T, V>& u, float (&f)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] += to_f32(u.v[j]);
}

// A sum or maximum over the threads of a row, the same in each: lanes, then waves in order.  red: a word per wave, of
// two arrays in turn: who writes one has passed the other's barrier, behind which nobody reads the first any more.
template <int kWaves>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = wave_sum(v);
    if constexpr (kWaves > 1) {
        if (lane_id() == 0) red[wave_id()] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w];
    }
    return v;
}
// (two sums at once)
template <int kWaves>
__device__ __forceinline__ void row_sums(float& a, float& b, float2* red) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (kWaves > 1) {
        if (lane_id() == 0) red[wave_id() % kWaves] = make_float2(a, b);
        __syncthreads();
        a = red[0].x, b = red[0].y;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) a += red[w].x, b += red[w].y;
    }
}
// (of magnitudes' bits, which order like the magnitudes, infinity above every finite value and NaN above infinity)
template <int kWaves>
__device__ __forceinline__ uint32_t row_max(uint32_t m, float* red) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    if constexpr (kWaves > 1) {
        if (lane_id() == 0) red[wave_id()] = __uint_as_float(m);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) m = max(m, __float_as_uint(red[w]));
    }
    return m;
}

// The 8-bit codes of V values by a product with inv = 1 / a where that cannot differ from the division (codes16 has the
// argument); else by the division, and zero where a is NaN.
template <int V>
__device__ __forceinline__ void codes_i8(const float (&v)[V], float a, float inv, uint32_t (&w)[V / 4]) {
    constexpr float kMagic = 12582912.0f;
    float far = a >= 0x1p-100f ? 0.0f : 1.0f;  // largest distance from a code
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float t = __builtin_fmaf(v[4 * i + j], inv, kMagic);
            far = fmaxf(far, fabsf(__builtin_fmaf(v[4 * i + j], inv, kMagic - t)));
            b[j] = __float_as_uint(t);
        }
        w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u),
                                     0x05040100u);
    }
    if (!(far <= 0.4999f)) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) w[i] = 0;
        if (a != a) return;
#pragma unroll
        for (int j = 0; j < V; ++j) w[j / 4] |= code_i8(v[j], a) << (8 * (j % 4));
    }
}

// x, residual, h and y may be the same memory: a thread reads a unit of x and residual before it writes that unit of h
// and y, in each pass, and no other thread's.
template <typename T, int kWaves, int kKeep, bool kI8, bool kAny, bool kStream, bool kTiny>
__global__ __launch_bounds__(kWaves == 1 ? 256 : 64 * kWaves) void add_rmsnorm_kernel(const T* x, const T* residual, int64_t rows,
                                                                                      int N, const T* __restrict__ weight, float eps,
                                                                                      T* h, T* y, int8_t* __restrict__ xq,
                                                                                      float* __restrict__ ascale) {
    constexpr int V = kUnit<T>, kThreads = 64 * kWaves, kRows = kWaves == 1 ? 4 : 1;
    __shared__ float red[3][kWaves];
    int turn = 0;
    const int tid = kWaves == 1 ? lane_id() : (int)threadIdx.x;
    const int units = (N + V - 1) / V;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t m = (int64_t)blockIdx.x * kRows + (kWaves == 1 ? wave_id() : 0);
    // the kept units of a row, asked for while the row before is worked on
    Pack<T, V> xu[kKeep], ru[kKeep], wu[kKeep];
    auto load_row = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int c = tid + kThreads * i;
            xu[i] = c < units && row < rows ? load_row_unit<kStream, kAny>(x + row * N, c, N) : Pack<T, V>{};
            if (residual) ru[i] = c < units && row < rows ? load_row_unit<kStream, kAny>(residual + row * N, c, N) : Pack<T, V>{};
        }
    };
    load_row(m);
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = tid + kThreads * i;
        if (weight && c < units) wu[i] = load_row_unit<false, kAny>(weight, c, N);
    }
    for (; m < rows; m += step) {
        const T* xr = x + m * N;
        const T* rr = residual ? residual + m * N : nullptr;
        // s of a unit that is read again; times up, for the sum and v
        float up = 1.0f;
        auto sum_unit = [&](int c, float (&s)[V]) __attribute__((always_inline)) {
            widen(load_row_unit<false, kAny>(xr, c, N), s);
            if (rr) add(load_row_unit<false, kAny>(rr, c, N), s);
        };
        float keep[kKeep][V], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            widen(xu[i], keep[i]);
            if (rr) add(ru[i], keep[i]);
        }
        load_row(m + step);
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) ss = __builtin_fmaf(keep[i][j], keep[i][j], ss);
        for (int c = tid + kThreads * kKeep; c < units; c += kThreads) {
            float s[V];
            sum_unit(c, s);
#pragma unroll
            for (int j = 0; j < V; ++j) ss = __builtin_fmaf(s[j], s[j], ss);
        }
        ss = row_sum<kWaves>(ss, red[turn]);
        if constexpr (!kI8) turn ^= 1;
        auto raise = [&](float (&s)[V]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] *= up;
        };
        if (kTiny && ss < kSmallSum) {  // (every thread of the row)
            up = kUp, ss = 0.0f;
            auto square = [&](const float (&s)[V]) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < V; ++j) ss = __builtin_fmaf(s[j], s[j], ss);
            };
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int c = tid + kThreads * i;
                if (h && c < units) store_row_unit<kStream, kAny>(h + m * N, c, N, keep[i]);
                raise(keep[i]);
                square(keep[i]);
            }
            for (int c = tid + kThreads * kKeep; c < units; c += kThreads) {
                float s[V];
                sum_unit(c, s);
                raise(s);
                square(s);
            }
            ss = row_sum<kWaves>(ss, red[2]);  // (a barrier of another sum lies between this and the next use of red[2])
        }
        const float r = factor(ss, N, eps, up);
        // s -> v
        auto scaled = [&](const Pack<T, V>& w, float (&s)[V]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = weight ? s[j] * r * to_f32(w.v[j]) : s[j] * r;
        };
        auto weight_unit = [&](int c) __attribute__((always_inline)) {
            return weight ? load_row_unit<false, kAny>(weight, c, N) : Pack<T, V>{};
        };
        if constexpr (!kI8) {
            auto out = [&](int c, const Pack<T, V>& w, float (&s)[V]) __attribute__((always_inline)) {
                scaled(w, s);
                store_row_unit<kStream, kAny>(y + m * N, c, N, s);
            };
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int c = tid + kThreads * i;
                if (c >= units) continue;
                if (h && up == 1.0f) store_row_unit<kStream, kAny>(h + m * N, c, N, keep[i]);
                out(c, wu[i], keep[i]);
            }
            for (int c = tid + kThreads * kKeep; c < units; c += kThreads) {
                float s[V];
                sum_unit(c, s);
                if (h) store_row_unit<kStream, kAny>(h + m * N, c, N, s);
                raise(s);
                out(c, weight_unit(c), s);
            }
        } else {
            uint32_t top = 0;
            auto widest = [&](const float (&v)[V]) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            };
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int c = tid + kThreads * i;
                if (c < units) {
                    if (h && up == 1.0f) store_row_unit<kStream, kAny>(h + m * N, c, N, keep[i]);
                    scaled(wu[i], keep[i]);
                    widest(keep[i]);
                }
            }
            for (int c = tid + kThreads * kKeep; c < units; c += kThreads) {
                float s[V];
                sum_unit(c, s);
                raise(s);
                scaled(weight_unit(c), s);
                widest(s);
            }
            const float a = scale_i8(__uint_as_float(row_max<kWaves>(top, red[1]))), inv = 1.0f / a;
            auto codes = [&](int c, const float (&v)[V]) __attribute__((always_inline)) {
                uint32_t w[V / 4];
                codes_i8(v, a, inv, w);
                if constexpr (V == 8)
                    *reinterpret_cast<uint2*>(xq + m * N + c * V) = make_uint2(w[0], w[1]);
                else
                    *reinterpret_cast<uint32_t*>(xq + m * N + c * V) = w[0];
            };
#pragma unroll
            for (int i = 0; i < kKeep; ++i) {
                const int c = tid + kThreads * i;
                if (c < units) codes(c, keep[i]);
            }
            for (int c = tid + kThreads * kKeep; c < units; c += kThreads) {
                float s[V];
                sum_unit(c, s);
                if (h) store_row_unit<kStream, kAny>(h + m * N, c, N, s);
                raise(s);
                scaled(weight_unit(c), s);
                codes(c, s);
            }
            if (lane_id() == 0) ascale[m] = a;  // (every wave's is the same)
        }
    }
}

// ---- gradients ----------------------------------------------------------------------------------

// dx, and this block's part of dweight.  kWaves waves of a block take a row, rows in turn, and a thread the same
// columns of each, so that the columns' sums stay in its registers (N at most 64 kWaves kUnits V); the groups of waves
// add theirs in LDS at the end, in order.  A block's part leaves once, to part [blocks][N].  The order of additions
// does not depend on timing.
constexpr int grad_waves(int row_waves) { return row_waves > 8 ? row_waves : 8; }  // of a block
template <typename T, int kWaves, int kUnits, bool kAny, bool kStream, bool kTiny>
__global__ __launch_bounds__(64 * grad_waves(kWaves)) void add_rmsnorm_backward_kernel(const T* dy, const T* dh, const T* __restrict__ h,
                                                                               int64_t rows, int N, const T* __restrict__ weight,
                                                                               float eps, T* dx, float* __restrict__ part) {
    constexpr int V = kUnit<T>, kThreads = 64 * kWaves, kGradWaves = grad_waves(kWaves), kRows = kGradWaves / kWaves;
    __shared__ float2 red[3][kGradWaves];
    int turn = 0;
    __shared__ float sums[kRows > 1 ? kRows * kThreads * kUnits * V : 1];
    const int tid = threadIdx.x % kThreads, group = wave_id() / kWaves, units = (N + V - 1) / V;
    Pack<T, V> w[kUnits];
    float dw[kUnits][V];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int c = tid + kThreads * i;
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.0f, w[i].v[j] = from_f32<T>(1.0f);
        if (weight && c < units) w[i] = load_row_unit<false, kAny>(weight, c, N);
    }
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t m = (int64_t)blockIdx.x * kRows + group;
    // a row, asked for while the row before is worked on
    Pack<T, V> next_g[kUnits], next_h[kUnits], next_a[kUnits];
    auto load_row = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int c = tid + kThreads * i;
            const bool there = c < units && row < rows;
            next_h[i] = there ? load_row_unit<kStream, kAny>(h + row * N, c, N) : Pack<T, V>{};
            next_g[i] = there ? load_row_unit<kStream, kAny>(dy + row * N, c, N) : Pack<T, V>{};
            if (dx && dh && there) next_a[i] = load_row_unit<kStream, kAny>(dh + row * N, c, N);
        }
    };
    constexpr bool kAhead = kWaves <= 8;  // (sixteen waves a block have 128 registers a thread: they spill)
    if (kAhead) load_row(m);
    for (; m - group < rows; m += step) {  // (as often for every group: they share the barriers)
        if (!kAhead) load_row(m);
        Pack<T, V> gu[kUnits], hu[kUnits], au[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) gu[i] = next_g[i], hu[i] = next_h[i], au[i] = next_a[i];
        if (kAhead) load_row(m + step);
        float ss = 0.0f, gh = 0.0f;
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float hv = to_f32(hu[i].v[j]), g = to_f32(gu[i].v[j]) * to_f32(w[i].v[j]);
                ss = __builtin_fmaf(hv, hv, ss);
                gh = __builtin_fmaf(g, hv, gh);
            }
        row_sums<kWaves>(ss, gh, red[turn] + group * kWaves);
        turn ^= 1;
        float up = 1.0f;
        if constexpr (kTiny) {  // (every group of the block: they share the barrier)
            float ss_up = 0.0f, gh_up = 0.0f;
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float hv = to_f32(hu[i].v[j]) * kUp;
                    ss_up = __builtin_fmaf(hv, hv, ss_up);
                    gh_up = __builtin_fmaf(to_f32(gu[i].v[j]) * to_f32(w[i].v[j]), hv, gh_up);
                }
            row_sums<kWaves>(ss_up, gh_up, red[2] + group * kWaves);
            if (ss < kSmallSum) {
                up = kUp, ss = ss_up, gh = gh_up;
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) hu[i].v[j] = from_f32<T>(to_f32(hu[i].v[j]) * kUp);  // (exact: below 2^60)
            }
        }
        const float r = factor(ss, N, eps, up), c = gh * r / (float)N;  // (the mean of g u)
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int at = tid + kThreads * i;
            if (at >= units || m >= rows) continue;
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = to_f32(hu[i].v[j]) * r, g = to_f32(gu[i].v[j]);
                dw[i][j] = __builtin_fmaf(g, u, dw[i][j]);
                o[j] = r * (g * to_f32(w[i].v[j]) - u * c) * up;
            }
            if (dx && dh) add(au[i], o);
            if (dx) store_row_unit<kStream, kAny>(dx + m * N, at, N, o);
        }
    }
    if (!part) return;
    if constexpr (kRows > 1) {
        // [group][unit][V][thread]
        constexpr int kAll = kThreads * kUnits * V;
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) sums[group * kAll + (i * V + j) * kThreads + tid] = dw[i][j];
        __syncthreads();
        for (int u = threadIdx.x; u < kAll; u += 64 * kGradWaves) {
            const int n = (u % kThreads + kThreads * (u / kThreads / V)) * V + u / kThreads % V;
            float s = sums[u];
#pragma unroll
            for (int k = 1; k < kRows; ++k) s += sums[k * kAll + u];
            if (n < N) part[(int64_t)blockIdx.x * N + n] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int c = tid + kThreads * i;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c < units && c * V + j < N) part[(int64_t)blockIdx.x * N + c * V + j] = dw[i][j];
        }
    }
}

// Rows too long for that: dx row by row, each read twice, and r kept for the columns' sums below (with a minus where it is
// the factor of the row times kUp).
template <typename T, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void add_rmsnorm_backward_long_kernel(const T* dy, const T* dh, const T* __restrict__ h,
                                                                                int64_t rows, int N, const T* __restrict__ weight,
                                                                                float eps, T* dx, float* __restrict__ rstd) {
    constexpr int V = kUnit<T>, kThreads = 64 * kWaves;
    __shared__ float2 red[3][kWaves];
    int turn = 0;
    const int units = (N + V - 1) / V;
    for (int64_t m = blockIdx.x; m < rows; m += gridDim.x) {
        float ss = 0.0f, gh = 0.0f, up = 1.0f;
        auto sum = [&]() __attribute__((always_inline)) {
            ss = gh = 0.0f;
            for (int c = threadIdx.x; c < units; c += kThreads) {
                float hv[V], g[V], w[V];
                widen(load_row_unit<false, true>(h + m * N, c, N), hv);
                widen(load_row_unit<false, true>(dy + m * N, c, N), g);
                if (weight) widen(load_row_unit<false, true>(weight, c, N), w);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    hv[j] *= up;
                    ss = __builtin_fmaf(hv[j], hv[j], ss);
                    gh = __builtin_fmaf(weight ? g[j] * w[j] : g[j], hv[j], gh);
                }
            }
        };
        sum();
        row_sums<kWaves>(ss, gh, red[turn]);
        turn ^= 1;
        if (eps < kSmallEps && ss < kSmallSum) {  // (the whole block)
            up = kUp;
            sum();
            row_sums<kWaves>(ss, gh, red[2]);
        }
        const float r = factor(ss, N, eps, up), c = gh * r / (float)N;  // (the mean of g u)
        if (rstd && threadIdx.x == 0) rstd[m] = up == 1.0f ? r : -r;
        if (!dx) continue;
        for (int at = threadIdx.x; at < units; at += kThreads) {
            float hv[V], g[V], w[V];
            widen(load_row_unit<false, true>(h + m * N, at, N), hv);
            widen(load_row_unit<false, true>(dy + m * N, at, N), g);
            if (weight) widen(load_row_unit<false, true>(weight, at, N), w);
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = r * ((weight ? g[j] * w[j] : g[j]) - hv[j] * up * r * c) * up;
            if (dh) add(load_row_unit<false, true>(dh + m * N, at, N), g);
            store_row_unit<false, true>(dx + m * N, at, N, g);
        }
    }
}
template <typename T>
__global__ __launch_bounds__(256) void rmsnorm_dweight_long_kernel(const T* __restrict__ dy, const T* __restrict__ h, int64_t rows,
                                                                   int N, const float* __restrict__ rstd,
                                                                   float* __restrict__ part, int64_t each) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    const int64_t lo = blockIdx.y * each, hi = min(lo + each, rows);
    if (n >= N) return;
    float sum = 0.0f;
    for (int64_t m = lo; m < hi; ++m) {
        const float r = rstd[m], hv = to_f32(h[m * N + n]);
        sum = __builtin_fmaf(to_f32(dy[m * N + n]), r < 0.0f ? hv * kUp * -r : hv * r, sum);
    }
    part[(int64_t)blockIdx.y * N + n] = sum;
}

// dweight = the parts' sums over [parts][N], in an order of their own: kGroups threads a column take every kGroups-th
// part, and the groups are added in order.
constexpr int kJoinColumns = 32, kJoinGroups = 32;
__global__ __launch_bounds__(kJoinColumns* kJoinGroups) void join_dweight_kernel(const float* __restrict__ part, int parts, int N,
                                                                                 float* __restrict__ dweight) {
    __shared__ float sums[kJoinGroups][kJoinColumns + 1];
    const int col = threadIdx.x % kJoinColumns, group = threadIdx.x / kJoinColumns;
    const int n = blockIdx.x * kJoinColumns + col;
    float s = 0.0f;
    if (n < N) {
#pragma unroll 4
        for (int p = group; p < parts; p += kJoinGroups) s += part[(int64_t)p * N + n];
    }
    sums[group][col] = s;
    __syncthreads();
    if (group == 0 && n < N) {
        s = sums[0][col];
#pragma unroll
        for (int g = 1; g < kJoinGroups; ++g) s += sums[g][col];
        dweight[n] = s;
    }
}

// Blocks of the gradients' kernel, each with a part of dweight: one a CU.
constexpr int64_t kGradBlocks = 256;
// Longest row, in elements, whose columns' sums stay in a block's registers.
template <typename T>
constexpr int64_t kGradKept = 1024 * 2 * kUnit<T>;
constexpr int64_t kLongParts = 64;

int64_t grad_parts(int64_t rows) { return std::min(rows, kGradBlocks); }

// Waves of a launch: as many as run at once, each with rows in turn.
constexpr int64_t kNormWaves = 4096;
// Arrays from this many bytes on are read and written past the caches' usual order (gradients 16384 x 4096 bf16 92 us against
// 101, 8192 x 2048, 32 MiB, 28.4 against 30.3; of 16 MiB 17.6 against 17.2).
constexpr int64_t kNormStreamBytes = 32 << 20;

}  // namespace

hipError_t launch_add_rmsnorm(int dtype, const void* x, const void* residual, int64_t rows, int64_t N, const void* weight,
                              float eps, void* h, void* y, int8_t* xq, float* ascale, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t units = (N + kUnit<T> - 1) / kUnit<T>;
        const bool past = rows * N * (int64_t)sizeof(T) >= kNormStreamBytes;
        auto run = [&](auto waves, auto keep, auto i8, auto any, auto stream_past, auto tiny) {
            constexpr int kWaves = decltype(waves)::value, kRows = kWaves == 1 ? 4 : 1;
            const dim3 grid((unsigned)std::min<int64_t>((rows + kRows - 1) / kRows, kNormWaves / (kWaves * kRows)));
            hipLaunchKernelGGL((add_rmsnorm_kernel<T, kWaves, decltype(keep)::value, decltype(i8)::value, decltype(any)::value,
                                                   decltype(stream_past)::value, decltype(tiny)::value>),
                               grid, dim3(kWaves == 1 ? 256 : 64 * kWaves), 0, stream, static_cast<const T*>(x),
                               static_cast<const T*>(residual), rows, (int)N, static_cast<const T*>(weight), eps, static_cast<T*>(h),
                               static_cast<T*>(y), xq, ascale);
            return hipGetLastError();
        };
        // Two units a thread, so a wave for 128 of a row's units.
        auto pick_waves = [&](auto i8, auto any, auto past, auto tiny) {
            using I2 = std::integral_constant<int, 2>;
            if (units <= 128) return run(std::integral_constant<int, 1>{}, I2{}, i8, any, past, tiny);
            if (units <= 256) return run(std::integral_constant<int, 2>{}, I2{}, i8, any, past, tiny);
            if (units <= 512) return run(std::integral_constant<int, 4>{}, I2{}, i8, any, past, tiny);
            if (units <= 1024) return run(std::integral_constant<int, 8>{}, I2{}, i8, any, past, tiny);
            return run(std::integral_constant<int, 16>{}, I2{}, i8, any, past, tiny);
        };
        using No = std::false_type;
        using Yes = std::true_type;
        auto pick = [&](auto i8, auto any) { return past ? pick_waves(i8, any, Yes{}, No{}) : pick_waves(i8, any, No{}, No{}); };
        // (in 8 bits rows are whole units: N % 16 == 0)
        if (eps < kSmallEps) return xq ? pick_waves(Yes{}, No{}, No{}, Yes{}) : pick_waves(No{}, Yes{}, No{}, Yes{});
        if (xq) return pick(Yes{}, No{});
        return N % kUnit<T> == 0 ? pick(No{}, No{}) : pick(No{}, Yes{});
    });
}

size_t add_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t N) {
    // the parts of dweight, and a factor per row that the longest rows need
    const int64_t parts = N <= kGradKept<bf16_t> ? grad_parts(rows) : std::min(rows, kLongParts);
    return (size_t)parts * (size_t)N * 4 + (size_t)((rows + 3) / 4 * 16);
}

hipError_t launch_add_rmsnorm_backward(int dtype, const void* dy, const void* dh, const void* h, int64_t rows, int64_t N,
                                       const void* weight, float eps, void* dx, float* dweight, float* ws, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        const T *dyt = static_cast<const T*>(dy), *dht = static_cast<const T*>(dh), *ht = static_cast<const T*>(h),
                *wt = static_cast<const T*>(weight);
        T* dxt = static_cast<T*>(dx);
        int parts = (int)grad_parts(rows);
        if (N <= kGradKept<T>) {
            const bool stream_past = rows * N * (int64_t)sizeof(T) >= kNormStreamBytes;
            auto run = [&](auto waves, auto keep, auto any, auto past, auto tiny) {
                constexpr int kWaves = decltype(waves)::value, kUnits = decltype(keep)::value, kGradWaves = grad_waves(kWaves), kRows = kGradWaves / kWaves;
                // Up to two rows for each group one block and no join (16 x 1024 bf16 5.6 us against 6.4, 16 x 500 fp32
                // 4.1 against 5.6; at four rows each 8.0 against 6.5 and 5.7 against 5.6).
                parts = rows <= 2 * kRows ? 1 : (int)std::min((rows + kRows - 1) / kRows, kGradBlocks);
                float* part = parts == 1 ? dweight : dweight ? ws : nullptr;
                hipLaunchKernelGGL((add_rmsnorm_backward_kernel<T, kWaves, kUnits, decltype(any)::value, decltype(past)::value, decltype(tiny)::value>),
                                   dim3((unsigned)parts), dim3(64 * kGradWaves), 0, stream, dyt, dht, ht, rows, (int)N, wt, eps, dxt, part);
                return hipGetLastError();
            };
            auto pick_waves = [&](auto any, auto past, auto tiny) {
                const int64_t units = (N + kUnit<T> - 1) / kUnit<T>;
                using I2 = std::integral_constant<int, 2>;
                if (units <= 128) return run(std::integral_constant<int, 1>{}, I2{}, any, past, tiny);
                if (units <= 256) return run(I2{}, I2{}, any, past, tiny);
                if (units <= 512) return run(std::integral_constant<int, 4>{}, I2{}, any, past, tiny);
                if (units <= 1024) return run(std::integral_constant<int, 8>{}, I2{}, any, past, tiny);
                return run(std::integral_constant<int, 16>{}, I2{}, any, past, tiny);
            };
            using No = std::false_type;
            using Yes = std::true_type;
            auto pick = [&](auto any) { return stream_past ? pick_waves(any, Yes{}, No{}) : pick_waves(any, No{}, No{}); };
            const hipError_t e = eps < kSmallEps ? pick_waves(Yes{}, No{}, Yes{}) : N % kUnit<T> == 0 ? pick(No{}) : pick(Yes{});
            if (e != hipSuccess || !dweight || parts == 1) return e;
        } else {
            float* rstd = ws;
            float* part = ws + (rows + 3) / 4 * 4;
            hipLaunchKernelGGL((add_rmsnorm_backward_long_kernel<T, 16>), dim3((unsigned)std::min<int64_t>(rows, kMaxGridBlocks)),
                               dim3(1024), 0, stream, dyt, dht, ht, rows, (int)N, wt, eps, dxt, dweight ? rstd : nullptr);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess || !dweight) return e;
            const int64_t each = (rows + kLongParts - 1) / kLongParts;
            parts = (int)((rows + each - 1) / each);
            hipLaunchKernelGGL((rmsnorm_dweight_long_kernel<T>), dim3((unsigned)((N + 255) / 256), (unsigned)parts), dim3(256), 0,
                               stream, dyt, ht, rows, (int)N, rstd, part, each);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            ws = part;
        }
        hipLaunchKernelGGL(join_dweight_kernel, dim3((unsigned)((N + kJoinColumns - 1) / kJoinColumns)),
                           dim3(kJoinColumns * kJoinGroups), 0, stream, ws, parts, (int)N, dweight);
        return hipGetLastError();
    });
}

}  // namespace w4a16

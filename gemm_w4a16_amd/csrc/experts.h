// experts.h -- what the int8 product and the experts' row movers share (gfx950 only): activation
// types, per-row int8 quantization, and the search for the expert that a row tile belongs to.
#pragma once

#include <algorithm>

#include "device_common.h"

namespace w4a16 {

// Blocks a launch may have at up to 1024 threads (the grid's threads stay below 2^32); kernels with
// more items than that walk them with a stride of the grid.
constexpr int64_t kMaxGridBlocks = (int64_t)1 << 21;

// ---- activation types ---------------------------------------------------------------------------
// Raw storage types: a distinct struct per 16-bit type, so that templates tell them apart.
struct bf16_t {
    uint16_t bits;
};
struct f16_t {
    uint16_t bits;
};

__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_bits_to_f32(v.bits); }
__device__ __forceinline__ float to_f32(f16_t v) { return f16_bits_to_f32(v.bits); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
    return bf16_t{f32_to_bf16_bits(v)};
}
template <>
__device__ __forceinline__ f16_t from_f32<f16_t>(float v) {
    return f16_t{f32_to_f16_bits(v)};
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}

// Calls f with a value of the storage type of `dtype` (0 bf16, 1 fp16, 2 fp32).
template <typename F>
hipError_t with_act_type(int dtype, F f) {
    if (dtype == 0) return f(bf16_t{});
    if (dtype == 1) return f(f16_t{});
    return f(float{});
}

// V elements moved as one unit (16 bytes where V * sizeof(T) is 16).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

// A unit read or written once: with kStream past the caches' usual order (non-temporal), which large arrays
// gain by and arrays that the caches hold lose by.
typedef uint32_t unit16_t __attribute__((ext_vector_type(4)));
template <bool kStream, typename U>
__device__ __forceinline__ U load_unit(const U* p) {
    if constexpr (kStream && sizeof(U) == 16)
        return __builtin_bit_cast(U, __builtin_nontemporal_load(reinterpret_cast<const unit16_t*>(p)));
    else
        return *p;
}
template <bool kStream, typename U>
__device__ __forceinline__ void store_unit(U* p, const U& u) {
    if constexpr (kStream && sizeof(U) == 16)
        __builtin_nontemporal_store(__builtin_bit_cast(unit16_t, u), reinterpret_cast<unit16_t*>(p));
    else
        *p = u;
}

// ---- int8 quantization of a row -------------------------------------------------------------------

// Bits of |v| as an unsigned integer of the type's own width: these order like the magnitudes, with
// infinity above every finite value and NaN above infinity.
__device__ __forceinline__ uint32_t abs_bits(bf16_t v) { return v.bits & 0x7FFFu; }
__device__ __forceinline__ uint32_t abs_bits(f16_t v) { return v.bits & 0x7FFFu; }
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float from_abs_bits(uint32_t b, bf16_t) { return bf16_bits_to_f32(b); }
__device__ __forceinline__ float from_abs_bits(uint32_t b, f16_t) { return f16_bits_to_f32(b); }
__device__ __forceinline__ float from_abs_bits(uint32_t b, float) { return __uint_as_float(b); }

// A row's scale from its largest magnitude: max / 127 in fp32 (IEEE division), 1 where that is zero,
// and NaN where the row holds an infinity or NaN (its codes are then zero and its outputs NaN).
__device__ __forceinline__ float scale_i8(float amax) {
    const float a = amax / 127.0f;
    if (!(amax < INFINITY)) return __uint_as_float(0x7FC00000u);
    return a == 0.0f ? 1.0f : a;
}

// rint(v / a), ties to even, clamped to +-127; 0 where a is NaN.
__device__ __forceinline__ uint32_t code_i8(float v, float a) {
    const float r = rintf(v / a);
    return (uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f) & 0xFFu;
}

// 16 consecutive activations (16-byte aligned), their largest magnitude's bits, and their codes.
template <typename T>
struct alignas(16) Act16 {
    T v[16];
};
template <typename T>
__device__ __forceinline__ uint32_t max_bits(const Act16<T>& x, uint32_t m) {
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, abs_bits(x.v[j]));
    return m;
}
// The codes by a product with r = 1 / a where that cannot differ: r and the product are each off by at most
// 2^-24 of their value, so for |v / a| <= 127 the product is within 127.5 * 2^-23 < 1.6e-5 of v / a, and the
// division's own rounding within 0.8e-5; with the product at least 1e-4 from a midpoint both round to the
// same code.  Else (and for scales whose reciprocal is not a normal number) the 16 are divided.
template <typename T>
__device__ __forceinline__ uint4 codes16(const Act16<T>& x, float a, float r) {
    uint32_t w[4] = {};
    float far = a >= 0x1p-100f ? 0.0f : 1.0f;  // largest distance from a code (NaN scales come here too)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float t = to_f32(x.v[j]) * r, q = rintf(t);
        far = fmaxf(far, fabsf(t - q));
        w[j / 4] |= ((uint32_t)(int)fminf(fmaxf(q, -127.0f), 127.0f) & 0xFFu) << (8 * (j % 4));
    }
    if (far > 0.4999f) {
        w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) w[j / 4] |= code_i8(to_f32(x.v[j]), a) << (8 * (j % 4));
        if (a != a) return make_uint4(0, 0, 0, 0);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// row[0 .. K) (K % 16 == 0) quantized by a block of kThreads, or by one wave (kThreads = 64, red unused): store(c,
// codes) for each 16 codes c; the row's scale is returned.  A thread's first activations stay in registers
// between the two passes.  red: one word per wave of LDS.
template <int kThreads, typename T, typename F>
__device__ __forceinline__ float quantize_row(const T* row, int K, uint32_t* red, F store) {
    constexpr int kKeep = kThreads == kWave ? 3 : 2;
    const int tid = kThreads == kWave ? lane_id() : (int)threadIdx.x;
    const Act16<T>* in = reinterpret_cast<const Act16<T>*>(row);
    Act16<T> keep[kKeep];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = tid + kThreads * i;
        if (c < K / 16) {
            keep[i] = in[c];
            m = max_bits(keep[i], m);
        }
    }
    for (int c = tid + kThreads * kKeep; c < K / 16; c += kThreads) m = max_bits(in[c], m);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    if constexpr (kThreads > kWave) {
        __syncthreads();  // red may still be read from the row before
        if (lane_id() == 0) red[wave_id()] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / kWave; ++w) m = max(m, red[w]);
    }
    const float a = scale_i8(from_abs_bits(m, T{})), r = 1.0f / a;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int c = tid + kThreads * i;
        if (c < K / 16) store(c, codes16(keep[i], a, r));
    }
    for (int c = tid + kThreads * kKeep; c < K / 16; c += kThreads) store(c, codes16(in[c], a, r));
    return a;
}

// ---- row tiles of experts ----------------------------------------------------------------------

// Most row tiles of `tile` rows that R rows over E experts can make: each expert that has rows may end
// in a part of a tile.
inline int64_t expert_tiles(int64_t R, int64_t E, int64_t tile) {
    const int64_t used = std::min(R, E);
    return (R + used * (tile - 1)) / tile;
}

struct ExpertTile {
    int expert, row0, row_end;  // rows [row0, min(row0 + tile, row_end)) of this expert; none if row0 >= row_end
};

// Expert e's rows, clamped to [0, R) whatever `offsets` holds.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int R, int& lo, int& hi) {
    lo = min(max(offsets[e], 0), R);
    hi = min(max(offsets[e + 1], lo), R);
}

// Row tiles of all experts; every wave counts for itself.
__device__ __forceinline__ int count_expert_tiles(const int32_t* __restrict__ offsets, int E, int R, int tile) {
    int n = 0;
    for (int e = lane_id(); e < E; e += kWave) {
        int lo, hi;
        expert_rows(offsets, e, R, lo, hi);
        n += (hi - lo + tile - 1) / tile;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off);
    return __builtin_amdgcn_readfirstlane(n);
}

// The expert and first row of row tile `t`, counting tiles expert by expert.  Each wave looks for
// itself, 64 experts at a time: the lanes' tile counts are summed over the lanes, and the lane whose
// range of tiles holds t is the expert.  Every lane returns the same.
__device__ __forceinline__ ExpertTile find_expert_tile(const int32_t* __restrict__ offsets, int E, int R, int tile, int t) {
    const int lane = lane_id();
    int before = 0;  // tiles of the experts so far
    for (int e0 = 0; e0 < E; e0 += kWave) {
        int lo = 0, hi = 0;
        if (e0 + lane < E) expert_rows(offsets, e0 + lane, R, lo, hi);
        const int n = (hi - lo + tile - 1) / tile;
        int end = n;  // inclusive sum over the lanes
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int v = __shfl_up(end, off);
            if (lane >= off) end += v;
        }
        const uint64_t past = __ballot(before + end > t);
        if (past != 0) {
            const int src = __ffsll((unsigned long long)past) - 1;
            const int first = before + __shfl(end - n, src);
            ExpertTile r;
            r.expert = __builtin_amdgcn_readfirstlane(e0 + src);
            r.row0 = __builtin_amdgcn_readfirstlane(__shfl(lo, src) + (t - first) * tile);
            r.row_end = __builtin_amdgcn_readfirstlane(__shfl(hi, src));
            if (r.row0 < __builtin_amdgcn_readfirstlane(__shfl(lo, src))) r.row0 = r.row_end;  // offsets that fall
            return r;
        }
        before += __shfl(end, kWave - 1);
    }
    return ExpertTile{0, 0, 0};
}

}  // namespace w4a16

// experts.h -- what the int8 product and the experts' row movers share (gfx950 only): activation
// types, per-row int8 quantization, and the search for the expert that a row tile belongs to.
#pragma once

#include <type_traits>

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

// V consecutive elements.  With kStream past the caches' usual order (non-temporal), which large arrays gain by and
// arrays that the caches hold lose by; kAny: at any element (the memory unit takes 16 bytes at any address).
typedef uint32_t unit16_t __attribute__((ext_vector_type(4)));
typedef unit16_t any16_t __attribute__((aligned(2)));
template <bool kStream, bool kAny, int V, typename T>
__device__ __forceinline__ Pack<T, V> load_unit(const T* p) {
    using U = Pack<T, V>;
    if constexpr (sizeof(U) == 16 && (kStream || kAny)) {
        using V16 = std::conditional_t<kAny, any16_t, unit16_t>;
        const V16* q = reinterpret_cast<const V16*>(p);
        const unit16_t v = kStream ? __builtin_nontemporal_load(q) : *q;
        return __builtin_bit_cast(U, v);
    } else {
        return *reinterpret_cast<const U*>(p);
    }
}
template <bool kStream, bool kAny, int V, typename T>
__device__ __forceinline__ void store_unit(T* p, const Pack<T, V>& u) {
    if constexpr (sizeof(u) == 16 && (kStream || kAny)) {
        using V16 = std::conditional_t<kAny, any16_t, unit16_t>;
        V16* q = reinterpret_cast<V16*>(p);
        const V16 v = __builtin_bit_cast(unit16_t, u);
        if constexpr (kStream)
            __builtin_nontemporal_store(v, q);
        else
            *q = v;
    } else {
        *reinterpret_cast<Pack<T, V>*>(p) = u;
    }
}

// ---- int8 quantization of a row -------------------------------------------------------------------

// The value whose magnitude has these bits.
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

// rint(v / a), ties to even, clamped to +-127 (a not NaN).
__device__ __forceinline__ uint32_t code_i8(float v, float a) {
    const float r = rintf(v / a);
    return (uint32_t)(int)fminf(fmaxf(r, -127.0f), 127.0f) & 0xFFu;
}

// 16 consecutive activations (16-byte aligned), their largest magnitude's bits, and their codes.
template <typename T>
struct alignas(16) Act16 {
    T v[16];
};
// The bits of |v| as an unsigned integer of the type's own width order like the magnitudes, with infinity above every
// finite value and NaN above infinity.  (16-bit types: the two halves of a word at once; fold_max joins them.)
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <typename T>
__device__ __forceinline__ uint32_t max_bits(const Act16<T>& x, uint32_t m) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(x.v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, m),
                                                                       __builtin_bit_cast(u16x2_t, w[j] & 0x7FFF7FFFu)));
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(x.v[j]) & 0x7FFFFFFFu);
    }
    return m;
}
template <typename T>
__device__ __forceinline__ uint32_t fold_max(uint32_t m) {
    return sizeof(T) == 2 ? max(m & 0xFFFFu, m >> 16) : m;
}
// The codes by a product with r = 1 / a where that cannot differ from the division.  fma(v, r, 1.5 * 2^23) is the
// product rounded to an integer, ties to even, in its low mantissa bits, whose lowest byte is the code in two's
// complement.  r is off by at most 2^-24 of its value, so for |v / a| <= 127.1 the product is within 0.8e-5 of
// v / a, and the division's own rounding within another 0.8e-5; with the product at least 1e-4 from a midpoint
// both round to the same code.  Else (and for scales whose reciprocal is not a normal number, or NaN) the 16
// are divided.
template <typename T>
__device__ __forceinline__ uint4 codes16(const Act16<T>& x, float a, float r) {
    constexpr float kMagic = 12582912.0f;
    uint32_t w[4];
    float far = a >= 0x1p-100f ? 0.0f : 1.0f;  // largest distance from a code
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = to_f32(x.v[4 * i + j]), t = __builtin_fmaf(v, r, kMagic);
            far = fmaxf(far, fabsf(__builtin_fmaf(v, r, kMagic - t)));
            b[j] = __float_as_uint(t);
        }
        w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u),
                                     0x05040100u);
    }
    if (!(far <= 0.4999f)) {
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
    constexpr int kKeep = 2;
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
    m = fold_max<T>(m);
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

// Whether a wave quantizes a row by itself, not a block: short rows, which would leave threads of a block idle, and
// enough of them for every SIMD (16384 rows of 1024 fp16 11.6 us against 21.1, 8192 of 2048 bf16 16.5 against
// 18.2; of 4096 29.5 against 25.1).
inline bool row_by_wave(int64_t rows, int64_t K) { return K <= 2048 && rows >= 1024; }

// ---- row tiles of experts ----------------------------------------------------------------------

// Most row tiles of `tile` rows that R rows over E experts can make: each expert that has rows may end
// in a part of a tile.
__host__ __device__ constexpr int64_t expert_tiles(int64_t R, int64_t E, int64_t tile) {
    const int64_t used = R < E ? R : E;
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

// The experts' row tiles, counted expert by expert; every wave counts for itself.  A lane holds one expert of a
// run of 64, whose tiles are summed over the lanes.
struct ExpertRun {
    int lo, hi, end;  // this lane's expert: its rows, and the run's tiles up to and with it
    int tiles;        // of the run
};
__device__ __forceinline__ ExpertRun expert_run(const int32_t* __restrict__ offsets, int E, int e0, int R, int tile) {
    ExpertRun r{0, 0, 0, 0};
    const int lane = lane_id();
    if (e0 + lane < E) expert_rows(offsets, e0 + lane, R, r.lo, r.hi);
    r.end = (r.hi - r.lo + tile - 1) / tile;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int v = __shfl_up(r.end, off);
        if (lane >= off) r.end += v;
    }
    r.tiles = __builtin_amdgcn_readlane(r.end, kWave - 1);
    return r;
}

// All tiles, given the first run.
__device__ __forceinline__ int count_expert_tiles(const ExpertRun& first, const int32_t* __restrict__ offsets, int E, int R,
                                                  int tile) {
    int n = first.tiles;
    for (int e0 = kWave; e0 < E; e0 += kWave) n += expert_run(offsets, E, e0, R, tile).tiles;
    return n;
}

// The expert and first row of tile `t`, given the first run: the first lane whose tiles end past t is the expert.
// Every lane returns the same.
__device__ __forceinline__ ExpertTile find_expert_tile(const ExpertRun& first, const int32_t* __restrict__ offsets, int E,
                                                       int R, int tile, int t) {
    ExpertRun run = first;
    for (int e0 = 0, before = 0;;) {
        const uint64_t past = __ballot(before + run.end > t);
        if (past != 0) {
            const int src = __ffsll((unsigned long long)past) - 1;
            const int lo = __builtin_amdgcn_readlane(run.lo, src), hi = __builtin_amdgcn_readlane(run.hi, src);
            const int start = before + __builtin_amdgcn_readlane(run.end, src) - (hi - lo + tile - 1) / tile;
            ExpertTile r{e0 + src, lo + (t - start) * tile, hi};
            if (r.row0 < lo) r.row0 = hi;  // offsets that fall
            return r;
        }
        before += run.tiles, e0 += kWave;
        if (e0 >= E) return ExpertTile{0, 0, 0};
        run = expert_run(offsets, E, e0, R, tile);
    }
}

}  // namespace w4a16

// mx4.h -- the microscaled 4-bit format's layout and conversions (gfx950 only).
//
// A block is 32 consecutive values of a row: a power of two 2^(s - 127), s one byte (255: the block is not a number),
// and 32 elements of four bits (e2m1: a sign and the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).  codes [rows][K/2], byte j
// of a row holding value 2j in its low half.  scales [K/256 rounded up][rows / 32 rounded up][64][4]: for each 256 of K
// (a k-tile) and 32 rows, a word for each lane of a wave, in the order the matrix instructions take them.  Lane
// l of a 16 x 128 operand holds row l % 16 and block l / 16 of the instruction's four; its word has the bytes of rows
// l % 16 (bytes 0, 1) and 16 + l % 16 (bytes 2, 3), of the k-tile's first (0, 2) and second (1, 3) 128.  So a lane
// reads one word for four operands, no byte is moved, and the scales of a tile's rows are one run of memory.
#pragma once

#include "experts.h"

namespace w4a16 {

constexpr int kMx4Block = 32;   // values that share a scale
constexpr int kMx4TileK = 256;  // values of a row in a k-tile: 128 bytes of codes, 8 scales
__host__ __device__ constexpr int64_t mx4_groups(int64_t rows) { return (rows + 31) / 32; }  // of 32 rows: 256 bytes a k-tile
__host__ __device__ constexpr int64_t mx4_ktiles(int64_t K) { return (K + kMx4TileK - 1) / kMx4TileK; }
constexpr size_t mx4_scale_bytes(int64_t rows, int64_t K) { return (size_t)mx4_ktiles(K) * (size_t)mx4_groups(rows) * 256; }
// Where the scale of row r's block b lies; groups: mx4_groups of the array's rows.
__device__ __forceinline__ int64_t mx4_scale_at(int64_t groups, int64_t r, int b) {
    return ((b / 8) * groups + r / 32) * 256 + (b % 4 * 16 + r % 16) * 4 + r / 16 % 2 * 2 + b / 4 % 2;
}

// The scale's byte for a block whose largest magnitude has these fp32 bits: floor(log2 max) less 2, the largest
// element's exponent, not below -127; 255 for a block with an infinity or NaN.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t max_bits) {
    const int e = (int)(max_bits >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 2^(s - 127); NaN for 255.
__device__ __forceinline__ float mx4_factor(uint32_t s) {
    return s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s == 0 ? 0x00400000u : s << 23);
}

// The fp32 bits of the largest magnitude among kN values (an even number of 16-bit ones: two at a time, whose bits order
// like the magnitudes).
template <int kN, typename T>
__device__ __forceinline__ uint32_t mx4_max_bits(const T* v) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
        u16x2_t m = __builtin_bit_cast(u16x2_t, w[0] & 0x7FFF7FFFu);
#pragma unroll
        for (int j = 1; j < kN / 2; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[j] & 0x7FFF7FFFu));
        return __float_as_uint(from_abs_bits(fold_max<T>(__builtin_bit_cast(uint32_t, m)), T{}));
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kN; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        return m;
    }
}
// The same over groups of four lanes, or eight.
__device__ __forceinline__ uint32_t mx4_max_quad(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor1, 0xF, 0xF, false));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppQuadXor2, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t mx4_max_eight(uint32_t m) {
    m = mx4_max_quad(m);
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppRowHalfMirror, 0xF, 0xF, false));
}

// kN values (4 or 8) as elements of a block of scale s, four bits each: v / X to nearest, ties to even, magnitudes past 6
// becoming 6 (the conversion takes the exponent of its scale alone, so 2^-127 too); zero where the block is not
// a number.
template <int kN, typename T>
__device__ __forceinline__ uint32_t mx4_codes(const T* v, uint32_t s) {
    const float X = __uint_as_float(s << 23);
    uint32_t w = 0;
    auto two = [&](auto place) __attribute__((always_inline)) {
        constexpr int i = decltype(place)::value;
        if constexpr (std::is_same_v<T, bf16_t>) {
            const bf16x2v_t p = __builtin_bit_cast(bf16x2v_t, reinterpret_cast<const uint32_t*>(v)[i]);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, p, X, i);
        } else if constexpr (std::is_same_v<T, f16_t>) {
            typedef _Float16 f16x2v_t __attribute__((ext_vector_type(2)));
            const f16x2v_t p = __builtin_bit_cast(f16x2v_t, reinterpret_cast<const uint32_t*>(v)[i]);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, p, X, i);
        } else {
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2 * i], v[2 * i + 1], X, i);
        }
    };
    two(std::integral_constant<int, 0>{});
    two(std::integral_constant<int, 1>{});
    if constexpr (kN == 8) {
        two(std::integral_constant<int, 2>{});
        two(std::integral_constant<int, 3>{});
    }
    return s == 255 ? 0u : w;
}

}  // namespace w4a16

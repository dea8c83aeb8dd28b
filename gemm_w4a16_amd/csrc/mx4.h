// mx4.h -- the microscaled 4-bit format's layout and conversions (gfx950 only).
//
// A block is 32 consecutive values of a row: a power of two 2^(s - 127), s one byte (255: the block is not a number),
// and 32 elements of four bits (e2m1: a sign and the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6).  codes [rows][K/2], byte j
// of a row holding value 2j in its low half; scales [K/256 rounded up][rows rounded up to 16][8], byte b of row r in
// k-tile t belonging to block 8 t + b.  So the scales of a tile's rows are one run of memory for each 256 of K, in
// whole 128-byte lines, and 8 bytes of a row are what a matrix-core step pair of 256 takes.
#pragma once

#include "device_common.h"

namespace w4a16 {

constexpr int kMx4Block = 32;   // values that share a scale
constexpr int kMx4TileK = 256;  // values of a row in a k-tile: 128 bytes of codes, 8 scales
__host__ __device__ constexpr int64_t mx4_rows(int64_t rows) { return (rows + 15) / 16 * 16; }  // that scales has room for
__host__ __device__ constexpr int64_t mx4_ktiles(int64_t K) { return (K + kMx4TileK - 1) / kMx4TileK; }
constexpr size_t mx4_scale_bytes(int64_t rows, int64_t K) { return (size_t)mx4_ktiles(K) * (size_t)mx4_rows(rows) * 8; }

// The scale's byte for a block whose largest magnitude has these fp32 bits: floor(log2 max) less 2, the largest
// element's exponent, not below -127; 255 for a block with an infinity or NaN.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t max_bits) {
    const int e = (int)(max_bits >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
// 2^(127 - s): what a value is multiplied by before it is rounded to an element (exact, but where the product
// falls below the normal numbers, far under half the smallest element).  0 for s = 255.
__device__ __forceinline__ float mx4_inverse(uint32_t s) { return s == 255 ? 0.0f : __uint_as_float((254 - s) << 23); }
// 2^(s - 127); NaN for 255.
__device__ __forceinline__ float mx4_factor(uint32_t s) {
    return s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s == 0 ? 0x00400000u : s << 23);
}

// Eight values, already multiplied, as elements: to nearest, ties to even, magnitudes past 6 becoming 6.
__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8]) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
    return w;
}

}  // namespace w4a16

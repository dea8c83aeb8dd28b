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

#include "device_common.h"

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

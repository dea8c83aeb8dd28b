// mx4.hip -- rows and weights quantized to the microscaled 4-bit format, and back (mx4.h has the layout).
//
// Block scale and elements as the OCP Microscaling Formats specification (v1.0, "Conversion from scalar to MX") has
// them: X = 2^(floor(log2 max|v|) - 2), element = v / X rounded to nearest even, magnitudes past 6 becoming 6.  A
// power of two divides exactly, so the codes are the definition's bit for bit.  A block that holds an infinity or NaN
// becomes NaN as a whole (scale 255, codes 0); other blocks are not touched by it.
#include <algorithm>

#include "experts.h"
#include "launch.h"
#include "mx4.h"

namespace w4a16 {

namespace {

// Bytes bound both directions.  A thread takes 8 values, four threads a block.
template <typename T>
__global__ __launch_bounds__(256) void quant_mx4_kernel(const T* __restrict__ x, int64_t M, int K, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
    const int K8 = K / 8;
    const int64_t units = M * K8, groups = mx4_groups(M);
    for (int64_t u0 = (int64_t)blockIdx.x * 256; u0 < units; u0 += (int64_t)gridDim.x * 256) {
        const int64_t m0 = u0 / K8;
        const uint32_t in = (uint32_t)(u0 - m0 * K8) + threadIdx.x;  // units from row m0's first
        const int64_t m = m0 + in / (uint32_t)K8;
        const int c = (int)(in % (uint32_t)K8);
        // (K % 32 == 0: the four threads of a block are there together or not at all)
        if (m >= M) continue;
        float v[8];
        if constexpr (sizeof(T) == 2) {
            const Pack<T, 8> p = load_unit<false, false, 8>(x + m * K + 8 * c);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f32(p.v[j]);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const Pack<T, 4> p = load_unit<false, false, 4>(x + m * K + 8 * c + 4 * h);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = to_f32(p.v[j]);
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const uint32_t s = mx4_scale(top);
        const float inv = mx4_inverse(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv;
        uint32_t w = mx4_codes8(v);
        if (s == 255) w = 0;  // (infinity and NaN times zero)
        *reinterpret_cast<uint32_t*>(codes + m * (K / 2) + 4 * c) = w;
        if (c % 4 == 0) {
            const int b = c / 4;
            scales[mx4_scale_at(groups, m, b)] = (uint8_t)s;
            if (b + 1 == K / 32) {  // the last k-tile's blocks past K
                for (int i = b + 1; i % 8 != 0; ++i) scales[mx4_scale_at(groups, m, i)] = 0;
            }
        }
    }
}

// A thread takes 8 codes of a block.
template <typename T>
__global__ __launch_bounds__(256) void dequant_mx4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                          int64_t M, int K, T* __restrict__ out) {
    const int K8 = K / 8;
    const int64_t units = M * K8, groups = mx4_groups(M);
    for (int64_t u0 = (int64_t)blockIdx.x * 256; u0 < units; u0 += (int64_t)gridDim.x * 256) {
        const int64_t m0 = u0 / K8;
        const uint32_t in = (uint32_t)(u0 - m0 * K8) + threadIdx.x;
        const int64_t m = m0 + in / (uint32_t)K8;
        const int c = (int)(in % (uint32_t)K8);
        if (m >= M) continue;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + m * (K / 2) + 4 * c);
        const float f = mx4_factor(scales[mx4_scale_at(groups, m, c / 4)]);
        float v[8];
        auto two = [&](int j, f32x2_t p) __attribute__((always_inline)) { v[2 * j] = p.x * f, v[2 * j + 1] = p.y * f; };
        two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0));
        two(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1));
        two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2));
        two(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3));
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
            Pack<T, V> p;
#pragma unroll
            for (int j = 0; j < V; ++j) p.v[j] = from_f32<T>(v[V * h + j]);
            store_unit<false, false>(out + m * K + 8 * c + V * h, p);
        }
    }
}

dim3 unit_blocks(int64_t M, int64_t K) { return dim3((unsigned)std::min<int64_t>((M * (K / 8) + 255) / 256, kMaxGridBlocks)); }

}  // namespace

hipError_t launch_quant_mx4(int dtype, const void* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((quant_mx4_kernel<T>), unit_blocks(M, K), dim3(256), 0, stream, static_cast<const T*>(x), M, (int)K,
                           codes, scales);
        return hipGetLastError();
    });
}

hipError_t launch_dequant_mx4(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, int dtype, void* out,
                              hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((dequant_mx4_kernel<T>), unit_blocks(M, K), dim3(256), 0, stream, codes, scales, M, (int)K,
                           static_cast<T*>(out));
        return hipGetLastError();
    });
}

}  // namespace w4a16

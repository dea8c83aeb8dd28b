// w4a4.hip -- W4A4: activations and weights both in the microscaled 4-bit format (mx4.h), on the scaled matrix
// instructions.
//
//     y[m][n] = sum_b 2^(sx[m][b] + sw[n][b] - 254) sum_{k in block b} p[m][k] q[n][k]
// with the products of elements exact and the sums in fp32, rounded once to the output type.
#include <algorithm>

#include "experts.h"
#include "launch.h"
#include "mx4.h"

namespace w4a16 {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4v_t __attribute__((ext_vector_type(4)));

// A wave computes 16 rows x 64 columns from operands in global memory.
template <typename TO>
__global__ __launch_bounds__(256) void w4a4_simple_kernel(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xscales, int M,
                                                          const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                          int N, int K, TO* __restrict__ y) {
    const int lane = lane_id(), l16 = lane & 15, kg = lane >> 4;
    const int64_t n_tiles = (N + 63) / 64, tiles = n_tiles * ((M + 15) / 16);
    const int64_t Mp = mx4_rows(M), Np = mx4_rows(N);
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave_id(); t < tiles; t += (int64_t)gridDim.x * 4) {
        const int m0 = (int)(t / n_tiles) * 16, n0 = (int)(t % n_tiles) * 64;
        const int m = min(m0 + l16, M - 1);
        f32x4v_t acc[4] = {};
        for (int k0 = 0; k0 < K; k0 += 128) {
            const int b = k0 / 32 + kg;
            const bool there = b < K / 32;
            auto frag = [&](const uint8_t* rows, int64_t r) __attribute__((always_inline)) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (there) v = *reinterpret_cast<const uint4*>(rows + r * (K / 2) + b * 16);
                return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
            };
            auto scale = [&](const uint8_t* s, int64_t rows, int64_t r) __attribute__((always_inline)) {
                return there ? (int)s[((int64_t)(b / 8) * rows + r) * 8 + b % 8] : 127;
            };
            const i32x8_t xf = frag(xq, m);
            const int xs = scale(xscales, Mp, m);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const int n = min(n0 + 16 * a + l16, N - 1);
                acc[a] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(codes, n), xf, acc[a], 4, 4, 0, scale(scales, Np, n), 0,
                                                                         xs);
            }
        }
        if (m0 + l16 >= M) continue;
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int n = n0 + 16 * a + 4 * kg + e;
                if (n < N) y[(int64_t)(m0 + l16) * N + n] = from_f32<TO>(acc[a][e]);
            }
    }
}

}  // namespace

hipError_t launch_gemm_w4a4(int dtype, const uint8_t* xq, const uint8_t* xscales, int64_t M, const uint8_t* codes,
                            const uint8_t* scales, int64_t N, int64_t K, void* y, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t tiles = ((N + 63) / 64) * ((M + 15) / 16);
        hipLaunchKernelGGL((w4a4_simple_kernel<T>), dim3((unsigned)std::min<int64_t>((tiles + 3) / 4, kMaxGridBlocks)), dim3(256), 0,
                           stream, xq, xscales, (int)M, codes, scales, (int)N, (int)K, static_cast<T*>(y));
        return hipGetLastError();
    });
}

}  // namespace w4a16

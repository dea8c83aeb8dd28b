// w8a8.hip -- W8A8: int8 activations (quantized per row) against the W8 format's int8 weights, on the
// int8 matrix cores; for one weight matrix and for one matrix per expert.
//
// With a_m = max_k |x[m][k]| / 127 and q[m][k] = clamp(rint(x[m][k] / a_m), -127, 127),
//     y[m][n] = a_m * s_n * sum_k q[m][k] w[n][k].
// The integer sum is exact in 32 bits (K < 2^17 keeps |sum| below 2^31 for any int8 codes), so it does
// not depend on the order of additions or on how K is divided; the two scales are applied once, in
// fp32, and the result is rounded once to the output type.
//
// With experts the rows are sorted by expert (offsets[e] is the first row of expert e) and row r of
// expert e is multiplied by that expert's weights.
#include "device_common.h"
#include "experts.h"
#include "launch.h"

namespace w4a16 {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// ---- activation quantization ------------------------------------------------------------------

template <typename T>
__global__ __launch_bounds__(256) void quant_rows_i8_kernel(const T* __restrict__ x, int64_t M, int K,
                                                            int8_t* __restrict__ xq, float* __restrict__ ascale) {
    __shared__ uint32_t red[4];
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const T* row = x + m * K;
        const float a = row_scale_i8<256>(row, K, red);
        if (threadIdx.x == 0) ascale[m] = a;
        for (int c = threadIdx.x; c < K / 16; c += 256) *reinterpret_cast<uint4*>(xq + m * K + 16 * c) = quant16(row + 16 * c, a);
    }
}

// ---- product ----------------------------------------------------------------------------------

// One wave: 16 rows x 64 columns; the MFMA's A operand is the weights, so a lane ends with four
// consecutive columns of one row.
template <typename TO, bool kExperts>
__global__ __launch_bounds__(256) void w8a8_simple_kernel(const int8_t* __restrict__ xq, const float* __restrict__ ascale,
                                                          const int8_t* __restrict__ codes,
                                                          const float* __restrict__ scales, TO* __restrict__ y, int M,
                                                          int N, int K, const int32_t* __restrict__ offsets, int E,
                                                          int n_tiles) {
    const int lane = lane_id(), wave = wave_id();
    const int l16 = lane & 15, kg = lane >> 4;
    const int tn = blockIdx.x % n_tiles, tm = blockIdx.x / n_tiles;
    int row0 = tm * 64, row_end = M, expert = 0;
    if constexpr (kExperts) {
        const ExpertTile t = find_expert_tile(offsets, E, M, 64, tm);
        if (t.row0 >= t.row_end) return;
        row0 = t.row0, row_end = t.row_end, expert = t.expert;
    }
    const int m = row0 + 16 * wave + l16, n0 = tn * 64;
    const int8_t* w = codes + (size_t)expert * N * K;
    const int8_t* xr = xq + (size_t)min(m, row_end - 1) * K;
    i32x4_t acc[4] = {};
    for (int k = 16 * kg; k < K + 16 * kg; k += 64) {
        i32x4_t b = {};
        if (k < K) b = *reinterpret_cast<const i32x4_t*>(xr + k);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            i32x4_t a = {};
            if (k < K) a = *reinterpret_cast<const i32x4_t*>(w + (size_t)min(n0 + 16 * c + l16, N - 1) * K + k);
            acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc[c], 0, 0, 0);
        }
    }
    if (m >= row_end) return;
    const float am = ascale[m];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = n0 + 16 * c + 4 * kg + e;
            if (n < N) y[(size_t)m * N + n] = from_f32<TO>((float)acc[c][e] * scales[(size_t)expert * N + n] * am);
        }
}

template <typename TO>
hipError_t launch_product(const int8_t* xq, const float* ascale, int64_t M, const int8_t* codes, const float* scales,
                          int64_t N, int64_t K, TO* y, const int32_t* offsets, int64_t E, hipStream_t stream) {
    const int64_t tn = (N + 63) / 64, tm = offsets ? expert_tiles(M, E, 64) : (M + 63) / 64;
    const dim3 grid((unsigned)(tn * tm));
    if (offsets)
        hipLaunchKernelGGL((w8a8_simple_kernel<TO, true>), grid, dim3(256), 0, stream, xq, ascale, codes, scales, y, (int)M,
                           (int)N, (int)K, offsets, (int)E, (int)tn);
    else
        hipLaunchKernelGGL((w8a8_simple_kernel<TO, false>), grid, dim3(256), 0, stream, xq, ascale, codes, scales, y, (int)M,
                           (int)N, (int)K, nullptr, 1, (int)tn);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows_i8(int dtype, const void* x, int64_t M, int64_t K, int8_t* xq, float* ascale,
                                hipStream_t stream) {
    const dim3 grid((unsigned)std::min<int64_t>(M, kMaxGridBlocks));
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((quant_rows_i8_kernel<T>), grid, dim3(256), 0, stream, static_cast<const T*>(x), M, (int)K, xq,
                           ascale);
        return hipGetLastError();
    });
}

bool w8a8_fits_grid(int64_t M, int64_t N, int64_t E) {
    return ((N + 63) / 64) * expert_tiles(M, E, 64) <= kMaxGridBlocks * 8;
}

hipError_t launch_gemm_w8a8(int dtype, const int8_t* xq, const float* ascale, int64_t M, const int8_t* codes,
                            const float* scales, int64_t N, int64_t K, void* y, const int32_t* offsets, int64_t E,
                            hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_product<T>(xq, ascale, M, codes, scales, N, K, static_cast<T*>(y), offsets, E, stream);
    });
}

}  // namespace w4a16

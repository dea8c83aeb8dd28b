// mx4.hip -- rows and weights quantized to the microscaled 4-bit format, and back (mx4.h has the layout).
//
// Block scale and elements as the OCP Microscaling Formats specification (v1.0, "Conversion from scalar to MX") has
// them: X = 2^(floor(log2 max|v|) - 2), element = v / X rounded to nearest even, magnitudes past 6 becoming 6.  A
// power of two divides exactly, so the codes are the definition's bit for bit.  A block that holds an infinity or NaN
// becomes NaN as a whole (scale 255, codes 0); other blocks are not touched by it.
#include <algorithm>
#include <type_traits>

#include "experts.h"
#include "launch.h"
#include "mx4.h"

namespace w4a16 {

namespace {

// Bytes bound both directions.  A block takes 32 rows of a k-tile, so that its scales, one group of 256 bytes, pass through
// LDS and are whole lines of memory (written byte by byte they cost as much as the codes); a half wave takes a row
// at a time, 8 values a lane, four lanes a block of the format.  14336 x 4096 fp32
// 51 us (5.2 TB/s; a copy moves 5.0), bf16 28; back to bf16 24-31; 333 x 2080 3.2.

// Tile `tile`: k-tile kt of rows 32 g ..
struct Tile {
    int kt;
    int64_t g;
    __device__ __forceinline__ Tile(int64_t tile, int KT) : kt((int)(tile % KT)), g(tile / KT) {}
};

template <typename T, int kWaves, bool kStream>
__global__ __launch_bounds__(64 * kWaves) void quant_mx4_kernel(const T* __restrict__ x, int64_t M, int K, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
    constexpr int V = 16 / sizeof(T), kLoads = 8 / V, kRowsOfWave = 32 / kWaves;
    __shared__ uint32_t group[2][64];
    const int lane = lane_id(), wave = wave_id();
    const int KT = (int)mx4_ktiles(K);
    const int64_t groups = mx4_groups(M), tiles = groups * KT;
    int which = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, which ^= 1) {
        const Tile at(tile, KT);
        const int k = at.kt * kMx4TileK + 8 * (lane % 32);
        const int64_t m0 = 32 * at.g + kRowsOfWave * wave + lane / 32;
        // (K % 32 == 0: the four lanes of a block are there together or not at all; what is not there has scale 0)
        Pack<T, V> p[kRowsOfWave / 2][kLoads];
#pragma unroll
        for (int i = 0; i < kRowsOfWave / 2; ++i)
#pragma unroll
            for (int h = 0; h < kLoads; ++h) {
                const int64_t m = m0 + 2 * i;
                p[i][h] = m < M && k < K ? load_unit<kStream, false, V>(x + m * K + k + V * h) : Pack<T, V>{};
            }
#pragma unroll
        for (int i = 0; i < kRowsOfWave / 2; ++i) {
            const int64_t m = m0 + 2 * i;
            const T* v = p[i][0].v;  // (a row's packs are one array of 8)
            const uint32_t s = mx4_scale(mx4_max_quad(mx4_max_bits<8>(v))), w = mx4_codes<8>(v, s);
            if (m < M && k < K) *reinterpret_cast<uint32_t*>(codes + m * (K / 2) + k / 2) = w;
            if (lane % 4 == 0)
                reinterpret_cast<uint8_t*>(group[which])[mx4_scale_at(1, kRowsOfWave * wave + 2 * i + lane / 32, lane % 32 / 4)] = (uint8_t)s;
        }
        __syncthreads();  // (the other half of `group` takes the next tile's)
        if (threadIdx.x < 64)
            reinterpret_cast<uint32_t*>(scales)[(at.kt * groups + at.g) * 64 + threadIdx.x] = group[which][threadIdx.x];
    }
}

template <typename T, int kWaves, bool kStream>
__global__ __launch_bounds__(64 * kWaves) void dequant_mx4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                          int64_t M, int K, T* __restrict__ out) {
    constexpr int V = 16 / sizeof(T), kRowsOfWave = 32 / kWaves;
    __shared__ uint32_t group[2][64];
    const int lane = lane_id(), wave = wave_id();
    const int KT = (int)mx4_ktiles(K);
    const int64_t groups = mx4_groups(M), tiles = groups * KT;
    int which = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, which ^= 1) {
        const Tile at(tile, KT);
        const int k = at.kt * kMx4TileK + 8 * (lane % 32);
        const int64_t m0 = 32 * at.g + kRowsOfWave * wave + lane / 32;
        if (threadIdx.x < 64)
            group[which][threadIdx.x] = reinterpret_cast<const uint32_t*>(scales)[(at.kt * groups + at.g) * 64 + threadIdx.x];
        uint32_t w[kRowsOfWave / 2];
#pragma unroll
        for (int i = 0; i < kRowsOfWave / 2; ++i)
            w[i] = m0 + 2 * i < M && k < K ? *reinterpret_cast<const uint32_t*>(codes + (m0 + 2 * i) * (K / 2) + k / 2) : 0u;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowsOfWave / 2; ++i) {
            const int64_t m = m0 + 2 * i;
            if (m >= M || k >= K) continue;
            const float f = mx4_factor(reinterpret_cast<const uint8_t*>(
                group[which])[mx4_scale_at(1, kRowsOfWave * wave + 2 * i + lane / 32, lane % 32 / 4)]);
            float v[8];
            auto two = [&](int j, f32x2_t q) __attribute__((always_inline)) { v[2 * j] = q.x * f, v[2 * j + 1] = q.y * f; };
            two(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0));
            two(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1));
            two(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2));
            two(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3));
#pragma unroll
            for (int h = 0; h < 8 / V; ++h) {
                Pack<T, V> p;
#pragma unroll
                for (int j = 0; j < V; ++j) p.v[j] = from_f32<T>(v[V * h + j]);
                store_unit<kStream, false>(out + m * K + k + V * h, p);
            }
        }
    }
}

// Few tiles by sixteen waves each, for the shorter chain (333 x 2080 fp16 3.2 us against 3.9 by four); else by eight (14336 x
// 4096 fp32 51 against 56 by four, bf16 28 against 34 by sixteen); arrays from 64 MiB on past the caches' usual order.
template <typename T, typename F>
hipError_t with_shape(int64_t M, int64_t K, F f) {
    const int64_t tiles = mx4_groups(M) * mx4_ktiles(K);
    const dim3 grid((unsigned)std::min<int64_t>(tiles, kMaxGridBlocks));
    if (tiles <= 1024) return f(grid, std::integral_constant<int, 16>{}, std::false_type{});
    if (M * K * (int64_t)sizeof(T) >= (64 << 20)) return f(grid, std::integral_constant<int, 8>{}, std::true_type{});
    return f(grid, std::integral_constant<int, 8>{}, std::false_type{});
}

}  // namespace

hipError_t launch_quant_mx4(int dtype, const void* x, int64_t M, int64_t K, uint8_t* codes, uint8_t* scales, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        return with_shape<T>(M, K, [&](dim3 grid, auto waves, auto past) {
            constexpr int kWaves = decltype(waves)::value;
            hipLaunchKernelGGL((quant_mx4_kernel<T, kWaves, decltype(past)::value>), grid, dim3(64 * kWaves), 0, stream,
                               static_cast<const T*>(x), M, (int)K, codes, scales);
            return hipGetLastError();
        });
    });
}

hipError_t launch_dequant_mx4(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, int dtype, void* out,
                              hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        return with_shape<T>(M, K, [&](dim3 grid, auto waves, auto past) {
            constexpr int kWaves = decltype(waves)::value;
            hipLaunchKernelGGL((dequant_mx4_kernel<T, kWaves, decltype(past)::value>), grid, dim3(64 * kWaves), 0, stream, codes,
                               scales, M, (int)K, static_cast<T*>(out));
            return hipGetLastError();
        });
    });
}

}  // namespace w4a16

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
// LDS and are whole lines of memory (written byte by byte they cost as much as the codes); a lane takes 16 bytes
// of a row, so a wave two rows of 16-bit values or one of 32-bit ones.  14336 x 4096 fp32
// 43-44 us (6.1 TB/s; a copy moves 5.1), bf16 28; back to bf16 24-31; 333 x 2080 fp16 3.0.  (32 bytes a lane of fp32: 50-53.)

// Tile `tile`: k-tile kt of rows 32 g ..
struct Tile {
    int kt;
    int64_t g;
    __device__ __forceinline__ Tile(int64_t tile, int KT) : kt((int)(tile % KT)), g(tile / KT) {}
};

template <typename T, int kWaves, bool kStream>
__global__ __launch_bounds__(64 * kWaves) void quant_mx4_kernel(const T* __restrict__ x, int64_t M, int K, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
    constexpr int V = 16 / sizeof(T), kLanes = kMx4TileK / V, kAtOnce = kWave / kLanes;  // lanes a row, rows at once
    constexpr int kBlockLanes = kMx4Block / V, kSteps = 32 / kWaves / kAtOnce;
    static_assert(kSteps * kWaves * kAtOnce == 32, "a tile's rows");
    __shared__ uint32_t group[2][64];
    const int lane = lane_id(), wave = wave_id();
    const int KT = (int)mx4_ktiles(K);
    const int64_t groups = mx4_groups(M), tiles = groups * KT;
    int which = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, which ^= 1) {
        const Tile at(tile, KT);
        const int k = at.kt * kMx4TileK + V * (lane % kLanes);
        const int r0 = kSteps * kAtOnce * wave + lane / kLanes;
        const int64_t m0 = 32 * at.g + r0;
        // (K % 32 == 0: the lanes of a block are there together or not at all; what is not there has scale 0)
        Pack<T, V> p[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t m = m0 + kAtOnce * i;
            p[i] = m < M && k < K ? load_unit<kStream, false, V>(x + m * K + k) : Pack<T, V>{};
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t m = m0 + kAtOnce * i;
            const uint32_t top = mx4_max_bits<V>(p[i].v);
            const uint32_t s = mx4_scale(kBlockLanes == 8 ? mx4_max_eight(top) : mx4_max_quad(top));
            uint32_t w = mx4_codes<V>(p[i].v, s);
            if constexpr (V == 4)  // two lanes' codes in the first one's word
                w |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, kDppQuadXor1, 0xF, 0xF, false) << 16;
            if (m < M && k < K && lane % (8 / V) == 0) *reinterpret_cast<uint32_t*>(codes + m * (K / 2) + k / 2) = w;
            if (lane % kBlockLanes == 0)
                reinterpret_cast<uint8_t*>(group[which])[mx4_scale_at(1, r0 + kAtOnce * i, lane % kLanes / kBlockLanes)] = (uint8_t)s;
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
// 4096 bf16 28 us against 34 by sixteen); arrays from 64 MiB on past the caches' usual order.
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

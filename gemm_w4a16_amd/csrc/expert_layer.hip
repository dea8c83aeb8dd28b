// expert_layer.hip -- a few tokens' whole pass through their experts in two launches: up products and SwiGLU, then
// down products and the weighted sum, on the int8 matrix cores, from rows already in 8 bits.
//
// Token t's choice j is pair p = t topk + j, of expert e = ids[p]; a pair whose id is outside [0, E) adds nothing.
//     g_i = a_t s_i sum_k xq[t][k] up[e][i][k],  u_i the same with row I + i   (integer sums exact)
//     v_i = g_i / (1 + exp(-g_i)) u_i            (fp32)
//     b = max |v| / 127 over each group of 64 columns (1 where 0, NaN where not finite), hq = clamp(rint(v / b))
//     o_n = s_n sum_groups b (sum_{i in group} hq_i down[e][n][i])            (integer sums exact, the rest fp32)
//     y[t][n] = sum_j weights[t][j] o_n          (in order of j, rounded once)
// A scale for 64 columns instead of one for the row: the first launch then finishes its codes by itself (a row's
// largest magnitude would need all of its blocks), and small values keep more bits.
#include <algorithm>

#include "experts.h"
#include "launch.h"

namespace w4a16 {

namespace {

constexpr int kGroup = 64;  // columns of v that share a scale

template <typename TI>
__device__ __forceinline__ int expert_of(const TI* ids, int p, int E) {
    const TI e = ids[p];
    return e >= 0 && e < E ? (int)e : -1;
}

__device__ __forceinline__ int dot16(uint4 a, uint4 b, int c) {
    c = __builtin_amdgcn_sdot4((int)a.x, (int)b.x, c, false);
    c = __builtin_amdgcn_sdot4((int)a.y, (int)b.y, c, false);
    c = __builtin_amdgcn_sdot4((int)a.z, (int)b.z, c, false);
    return __builtin_amdgcn_sdot4((int)a.w, (int)b.w, c, false);
}

// A block: one pair, one group.  Thread = (column of the group, gate or up, half of K).
template <typename TI>
__global__ __launch_bounds__(256) void layer_up_simple_kernel(const int8_t* __restrict__ xq, const float* __restrict__ ascale,
                                                              const TI* __restrict__ ids, int topk, int E,
                                                              const int8_t* __restrict__ up, const float* __restrict__ up_scales,
                                                              int H, int I, int8_t* __restrict__ hq, float* __restrict__ hscale) {
    __shared__ int sums[2][2][kGroup];
    const int p = blockIdx.y, e = expert_of(ids, p, E), t = p / topk;
    if (e < 0) return;
    const int c = threadIdx.x % kGroup, which = threadIdx.x / kGroup % 2, half = threadIdx.x / (2 * kGroup);
    const int i = min((int)blockIdx.x * kGroup + c, I - 1);
    const uint4* row = reinterpret_cast<const uint4*>(up + ((size_t)e * 2 * I + (size_t)which * I + i) * H);
    const uint4* x = reinterpret_cast<const uint4*>(xq + (size_t)t * H);
    int sum = 0;
    for (int k = half; k < H / 16; k += 2) sum = dot16(row[k], x[k], sum);
    sums[half][which][c] = sum;
    __syncthreads();
    if (threadIdx.x >= kGroup) return;
    const float a = ascale[t];
    const float* s = up_scales + (size_t)e * 2 * I;
    const float g = (float)(sums[0][0][c] + sums[1][0][c]) * s[i] * a, u = (float)(sums[0][1][c] + sums[1][1][c]) * s[I + i] * a;
    const float v = g / (1.0f + expf(-g)) * u;
    uint32_t m = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    const float b = scale_i8(__uint_as_float(m));
    if ((int)blockIdx.x * kGroup + c < I) hq[(size_t)p * I + i] = b != b ? 0 : (int8_t)code_i8(v, b);
    if (c == 0) hscale[(size_t)p * gridDim.x + blockIdx.x] = b;
}

// A block: one token, 256 columns of y.
template <typename TO, typename TI>
__global__ __launch_bounds__(256) void layer_down_simple_kernel(const int8_t* __restrict__ hq, const float* __restrict__ hscale,
                                                                const TI* __restrict__ ids, int topk,
                                                                const float* __restrict__ weights, int E,
                                                                const int8_t* __restrict__ down,
                                                                const float* __restrict__ down_scales, int H, int I,
                                                                TO* __restrict__ y) {
    const int t = blockIdx.y, n = blockIdx.x * 256 + threadIdx.x, groups = (I + kGroup - 1) / kGroup;
    if (n >= H) return;
    float sum = 0.0f;
    for (int j = 0; j < topk; ++j) {
        const int p = t * topk + j, e = expert_of(ids, p, E);
        if (e < 0) continue;
        const uint4* row = reinterpret_cast<const uint4*>(down + ((size_t)e * H + n) * I);
        const uint4* h = reinterpret_cast<const uint4*>(hq + (size_t)p * I);
        float o = 0.0f;
        for (int g = 0; g < groups; ++g) {
            int part = 0;
            for (int k = g * (kGroup / 16); k < min((g + 1) * (kGroup / 16), I / 16); ++k) part = dot16(row[k], h[k], part);
            o = __builtin_fmaf((float)part, hscale[(size_t)p * groups + g], o);
        }
        sum = __builtin_fmaf(weights[p], o * down_scales[(size_t)e * H + n], sum);
    }
    y[(size_t)t * H + n] = from_f32<TO>(sum);
}

}  // namespace

size_t expert_layer_scale_bytes(int64_t pairs, int64_t I) {
    return (size_t)pairs * (size_t)((I + kGroup - 1) / kGroup) * 4;
}

hipError_t launch_expert_layer_w8a8(int dtype, const int8_t* xq, const float* ascale, int64_t T, const void* ids, int id_bits,
                                    int64_t topk, const float* weights, int64_t E, const int8_t* up, const float* up_scales,
                                    const int8_t* down, const float* down_scales, int64_t H, int64_t I, void* y, int8_t* hq,
                                    float* hscale, hipStream_t stream) {
    auto run = [&](auto id) {
        using TI = decltype(id);
        const TI* idt = static_cast<const TI*>(ids);
        hipLaunchKernelGGL((layer_up_simple_kernel<TI>), dim3((unsigned)((I + kGroup - 1) / kGroup), (unsigned)(T * topk)), dim3(256),
                           0, stream, xq, ascale, idt, (int)topk, (int)E, up, up_scales, (int)H, (int)I, hq, hscale);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        return with_act_type(dtype, [&](auto t) {
            using TO = decltype(t);
            hipLaunchKernelGGL((layer_down_simple_kernel<TO, TI>), dim3((unsigned)((H + 255) / 256), (unsigned)T), dim3(256), 0,
                               stream, hq, hscale, idt, (int)topk, weights, (int)E, down, down_scales, (int)H, (int)I,
                               static_cast<TO*>(y));
            return hipGetLastError();
        });
    };
    return id_bits == 32 ? run(int32_t{}) : run(int64_t{});
}

}  // namespace w4a16

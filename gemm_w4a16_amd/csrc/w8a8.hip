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
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "device_common.h"
#include "experts.h"
#include "launch.h"
#include "lds_dma.h"

namespace w4a16 {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// ---- activation quantization ------------------------------------------------------------------

// One pass for the largest magnitude, one for the codes, the row held in registers between them.  Bytes and
// latency bound it: 8192 rows of 4096 fp32 take 31 us (5.4 TB/s), bf16 25 us (4.0 TB/s), 1024 rows 5.4 us, 37 rows
// 3.3 us.  kWaves waves per row (4, or 1: four rows a block).
template <typename T, int kWaves>
__global__ __launch_bounds__(256) void quant_rows_i8_kernel(const T* __restrict__ x, int64_t M, int K,
                                                            int8_t* __restrict__ xq, float* __restrict__ ascale) {
    constexpr int kRows = 4 / kWaves;
    __shared__ uint32_t red[4];
    for (int64_t m0 = (int64_t)blockIdx.x * kRows; m0 < M; m0 += (int64_t)gridDim.x * kRows) {
        const int64_t m = kWaves == 1 ? m0 + wave_id() : m0;
        if (kWaves == 1 && m >= M) continue;
        const float a = quantize_row<64 * kWaves>(x + m * K, K, red, [&](int c, uint4 q) __attribute__((always_inline)) {
            *reinterpret_cast<uint4*>(xq + m * K + 16 * c) = q;
        });
        if (lane_id() == 0) ascale[m] = a;
    }
}

// ---- product ----------------------------------------------------------------------------------

// A block computes BM rows x BN columns in WM x WN waves of (16 TM) x (16 TN), each doubled WK times
// along K.  K is taken in stages of WK k-tiles of 128; the waves of index wk along K multiply k-tile wk of a
// stage, and their sums are added at the end.  Operands reach LDS by direct copies into a ring of R
// units: a unit is a whole stage (U = 1), or a stage's weights or its rows of x (U = 2, BM = BN).
// kX = false: x is not staged (the ring holds weights alone).
//
// What bounds it.  Many rows: the matrix cores at the clock the power limit leaves.  At 1024 x 14336 x 4096 (T256x256,
// 53 us, 2.27 POP/s; hipBLASLt's int8 product 73 us) timing-only copies took 43 us without the copies inside the
// loop and 49 with all of them reading one line, and the matrix instructions alone on such data take 36; waiting
// for the copies costs nothing.  8192 rows: 376-393 us (2.45-2.56 POP/s; hipBLASLt 426-430).  Eight waves of 128 x 64
// rather than four of 128 x 128 (64 us): two waves per SIMD fill each other's gaps.  16x16x64 instructions rather
// than 32x32x32: 3.8 POP/s against 3.3 on random codes.  Few rows: the weights' bytes.  One row, 14336 x 4096:
// 14.1 us from HBM (4.2 TB/s), 11 from the Infinity Cache (5.3 TB/s); two rows for each of eight such matrices 79
// us (5.9 TB/s).  Few columns: each block's own chain of k-tiles, which K in parts shortens (launch_parts).  Short
// rows (K of 500 to 1000): a block's first copies and its outputs, which nothing hides (1621 x 19712 x 512 36 us).
template <int WM_, int WN_, int WK_, int TM_, int TN_, int R_, int U_ = 1, bool kX = true>
struct Tiling {
    static constexpr int WM = WM_, WN = WN_, WK = WK_, TM = TM_, TN = TN_, R = R_, U = U_;
    static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, NW = WM * WN * WK;
    static_assert(U == 1 || (U == 2 && WK == 1 && BM == BN), "units of one size");
    static constexpr int kXRows = kX ? BM : 0;
    static constexpr int kTileBytes = (kXRows + BN) * 128;  // one k-tile: BN rows of weights, then BM rows of x
    static constexpr int kUnitBytes = WK * kTileBytes / U;
    static constexpr int kCopies = kUnitBytes / 1024;      // of 8 rows x 128 bytes
    static constexpr int kWaveCopies = (kCopies + NW - 1) / NW;  // (the last ones may be made twice)
};

// An output before its last rounding: the sum times the weight row's scale, then the activation row's, each
// rounded to fp32.  The empty statement keeps the last product out of an instruction that multiplies and
// rounds to 16 bits at once, which the compiler would use in some kernels only: every kernel stores the
// same bits.
__device__ __forceinline__ float scaled_sum(int32_t sum, float sn, float am) {
    float v = (float)sum * sn * am;
    asm("" : "+v"(v));
    return v;
}

// Weights that one row tile reads (a tile of at most kOnceRows rows holds them all) and that take more than a
// quarter of the Infinity Cache's 256 MiB, so that they would hardly be there at the next call, are copied
// past it (kOnce): eight matrices of 14336 x 4096 for two rows each take 79 us against 87, two of them, from HBM, 25.8
// against 28.6, and one row of 28672 x 4096 26.6 against 29.0 (while the cache holds it 25.8 against 21.1).  Below, one
// row of 14336 x 4096 (56 MiB) takes 12.6 us so against 14.2 from HBM, and 11.9 against 11.0 where it shares the cache
// with two more such matrices.
constexpr int kOnceRows = 64;

// What x is: int8 rows; int8 rows sorted by expert; or a few rows of activations (TO) that every block
// quantizes for itself (kFused: no other launch, and x stays in LDS whole, behind the ring).
enum XKind { kRows, kExpertRows, kFused };

// LDS behind the ring for kFused: the tile's rows (16, or M if fewer) of codes, Kp (K up to whole stages) bytes
// each, and their activations as they are, in whole 1-KB copies.
__host__ __device__ constexpr int64_t fused_codes_bytes(int64_t M, int64_t K, int wk) {
    return M * ((K + 128 * wk - 1) / (128 * wk) * (128 * wk));
}
constexpr int64_t fused_raw_bytes(int64_t M, int64_t K, int element) {
    return (M * K * element + 1023) / 1024 * 1024;
}

// TO int32_t: y takes the sums of one part of K (split_k columns of it, a multiple of 128) per block, [parts][M][N].
template <typename TO, XKind kX, typename C, bool kOnce>
__global__ __launch_bounds__(64 * C::NW) void w8a8_tile_kernel(const void* __restrict__ x, const float* __restrict__ ascale,
                                                               const int8_t* __restrict__ codes,
                                                               const float* __restrict__ scales, TO* __restrict__ y, int M,
                                                               int N, int stride, const int32_t* __restrict__ offsets, int E,
                                                               int n_tiles, int group, int split_k) {
    constexpr int TM = C::TM, TN = C::TN, R = C::R, U = C::U, BM = C::BM, BN = C::BN, CW = C::kWaveCopies;
    constexpr int kTileCopies = C::kTileBytes / 1024 / U;  // of a unit's part of one k-tile
    constexpr bool kExperts = kX == kExpertRows, kFuse = kX == kFused, kSums = std::is_same_v<TO, int32_t>;
    static_assert(!kFuse || (U == 1 && BM == 16 && C::kXRows == 0), "a fused ring holds weights alone");
    __shared__ __attribute__((aligned(1024))) char smem[R * C::kUnitBytes];
    extern __shared__ __attribute__((aligned(1024))) char fused_lds[];
    const int8_t* xq = static_cast<const int8_t*>(x);
    const int lane = lane_id(), wave = wave_id();
    const int l16 = lane & 15, kg = lane >> 4;
    const int wn = wave % C::WN, wk = wave / C::WN % C::WK, wm = wave / (C::WN * C::WK);

    // This block's tile.  Blocks go to the XCDs in turn: each XCD takes a contiguous eighth of the tile
    // sequence, which walks `group` row tiles at a time, rows first, so that the blocks of one XCD share
    // operands in its L2.
    int row0, row_end = M, expert = 0, tn;
    int K = stride, k0 = 0;  // kSums: of this block's part of K
    {
        int m_tiles = (M + BM - 1) / BM;
        ExpertRun first;
        if constexpr (kExperts) {
            first = expert_run(offsets, E, 0, M, BM);
            // (offsets that fall can name rows more than once: no more tiles than the launch counted with)
            m_tiles = min((uint32_t)count_expert_tiles(first, offsets, E, M, BM), (uint32_t)expert_tiles(M, E, BM));
        }
        const int total = kSums ? gridDim.x : m_tiles * n_tiles, b = blockIdx.x;
        if (b >= total) return;
        const int xcd = b & 7, each = total >> 3, rest = total & 7;
        int s = xcd * each + min(xcd, rest) + (b >> 3);
        if constexpr (kSums) {  // the sequence once for each part
            const int part = s / (m_tiles * n_tiles);
            s -= part * m_tiles * n_tiles;
            k0 = part * split_k, K = min(split_k, stride - k0);
            y += (size_t)part * M * N;
        }
        const int g = s / (group * n_tiles), in = s - g * group * n_tiles;
        const int rows = min(group, m_tiles - g * group);
        tn = in / rows;
        const int tm = g * group + in - tn * rows;
        row0 = tm * BM;
        if constexpr (kExperts) {
            const ExpertTile t = find_expert_tile(first, offsets, E, M, BM, tm);
            if (t.row0 >= t.row_end) return;
            row0 = t.row0, row_end = t.row_end, expert = t.expert;
        }
    }
    const int n0 = tn * BN;
    const int KT = (K + 127) / 128, T = (KT + C::WK - 1) / C::WK;
    const int8_t* wbase = codes + ((size_t)expert * N + n0) * stride + k0;
    const int8_t* xbase = xq + (size_t)row0 * stride + k0;
    const uint32_t lds0 = lds_addr(smem);

    // This wave's copies j = CW wave + i of a unit: copy jj = j % kTileCopies of k-tile j / kTileCopies, rows
    // 8 jj + lane / 8 of [weights; x].  LDS slot lane % 8 of a row takes its 16-byte chunk
    // slot ^ ((row >> 1) & 7), so that the fragment reads below meet no bank twice.  Rows past the end
    // read the last row; they are never stored.
    auto is_w = [&](int part, int jj) __attribute__((always_inline)) { return U == 2 ? part == 0 : jj < BN / 8; };
    uint32_t voff[U][CW];
#pragma unroll
    for (int part = 0; part < U; ++part)
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            const int jj = min(CW * wave + i, C::kCopies - 1) % kTileCopies;
            const int r = 8 * jj + lane / 8, chunk = (lane % 8) ^ ((r >> 1) & 7);
            const int row = is_w(part, jj) ? min(r, N - 1 - n0) : min(U == 2 ? r : r - BN, row_end - 1 - row0);
            voff[part][i] = (uint32_t)row * (uint32_t)stride + 16u * chunk;
        }
    // copy i of stage t's unit `part` into ring slot `slot`; the last k-tile's chunks past K, and k-tiles past the
    // last, read what is there (their products are masked).  Stages past the last read one line over
    // and over: each unit is then the same number of copies, and every wait below is a constant.
    auto copy = [&](int t, int part, int slot, int i) __attribute__((always_inline)) {
        const int j = min(CW * wave + i, C::kCopies - 1), jj = j % kTileCopies;
        const int kt = min(t * C::WK + j / kTileCopies, KT - 1);
        const int8_t* base = (is_w(part, jj) ? wbase : xbase) + (size_t)kt * 128;
        uint32_t off = voff[part][i];
        const int left = K - kt * 128;
        if (left < 128) {
            const int r = 8 * jj + lane / 8, chunk = (lane % 8) ^ ((r >> 1) & 7);
            off -= (uint32_t)max(16 * chunk - (left - 16), 0);
        }
        if (t >= T) base = wbase, off = 0;
        const uint32_t lds = lds0 + (uint32_t)(slot * C::kUnitBytes + 1024 * j);
        if (kOnce && is_w(part, jj))
            dma16_once(off, base, lds);
        else
            dma16(off, base, lds);
    };

    // fragment of row tile rt at k-step ks of a k-tile: chunk 4 ks + kg of row 16 rt + l16 (the unit's own
    // rows; slot: the ring slot of its weights' unit)
    const char* frag0 = smem + wk * C::kTileBytes + 128 * l16;
    const int sw = (l16 >> 1) & 7;
    auto next_slot = [](int s, int n) __attribute__((always_inline)) { return s + n >= R ? s + n - R : s + n; };
    auto read = [&](int slot, int ks, int rt) __attribute__((always_inline)) {
        return *reinterpret_cast<const i32x4_t*>(frag0 + slot * C::kUnitBytes + 2048 * rt + 16 * ((4 * ks + kg) ^ sw));
    };
    const int w_rt = TN * wn, x_rt = (U == 2 ? 0 : BN / 16) + TM * wm;

    i32x4_t acc[TN][TM];
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};
    i32x4_t wf[2][TN], xf[2][TM];

    // the products of k-step ks, with `reads` fragment reads spread over the first three quarters of them and
    // `copies` copies over all; a wave at its products goes before one that waits or copies (1-5% faster at
    // 256 to 8192 rows)
    auto multiply = [&](int ks, auto reads, auto read, auto copies, auto copy) __attribute__((always_inline)) {
        constexpr int H = TM * TN, HR = (3 * H + 3) / 4;
        constexpr int nr = decltype(reads)::value, nc = decltype(copies)::value;
#pragma unroll
        for (int i = 0; i < H; ++i) {
#pragma unroll
            for (int u = (i * nr + HR - 1) / HR; u < min(nr, ((i + 1) * nr + HR - 1) / HR); ++u) read(u);
#pragma unroll
            for (int u = (i * nc + H - 1) / H; u < ((i + 1) * nc + H - 1) / H; ++u) copy(u);
            const int a = i / TM, b = i % TM;
            acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[ks][a], xf[ks][b], acc[a][b], 0, 0, 0);
            if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            if (i == 0) __builtin_amdgcn_s_setprio(1);
            if (i == H - 1) __builtin_amdgcn_s_setprio(0);
        }
    };
    const int Kp = T * C::WK * 128, fm = min(M - row0, 16);  // (kFuse: the tile's rows)
    const char* fused_x = fused_lds + min(l16, fm - 1) * Kp + wk * 128 + 16 * kg;
    // read u of stage t (in ring slot `slot`)
    auto read_step = [&](int t, int slot, int ks, int u) __attribute__((always_inline)) {
        if (kFuse && u < TM)
            xf[ks][u] = *reinterpret_cast<const i32x4_t*>(fused_x + t * (C::WK * 128) + 64 * ks);
        else if (u < TM)
            xf[ks][u] = read(U == 2 ? next_slot(slot, 1) : slot, ks, x_rt + u);
        else
            wf[ks][u - TM] = read(slot, ks, w_rt + u - TM);
    };
    constexpr int kReads = TM + TN;
    // Behind stage t's barrier its U units take the next ones of the ring's order, G copies: kEarly of them under
    // the stage's second k-step, the others under the next stage's first (where the ring holds more than
    // two stages; else the next barrier would wait for copies just made).
    constexpr int G = U * CW, kEarly = R > 2 * U ? G / 2 : G, kLate = G - kEarly;
    using NReads = std::integral_constant<int, kReads>;
    using NEarly = std::integral_constant<int, kEarly>;
    using NLate = std::integral_constant<int, kLate>;
    using None = std::integral_constant<int, 0>;
    auto none = [](int) {};

    static_assert(R * CW < 64, "the wait counts");
    char* raw = fused_lds + fused_codes_bytes(min(M, 16), K, C::WK);
    if constexpr (kFuse) {  // the tile's rows of x, ahead of the weights
        const TO* rows = static_cast<const TO*>(x) + (size_t)row0 * K;
        const int last = fm * K * (int)sizeof(TO) - 16, copies = (last + 16 + 1023) / 1024;
        for (int c = wave; c < copies; c += C::NW)
            dma16((uint32_t)min(1024 * c + 16 * lane, last), rows, lds_addr(raw) + (uint32_t)(1024 * c));
    }
#pragma unroll
    for (int u = 0; u < R * CW - kLate; ++u) copy(u / CW / U, u / CW % U, u / CW, u % CW);
    __shared__ float fused_scale[kFuse ? 16 : 1];
    if constexpr (kFuse) {  // codes and scales, while the first weights are on their way
        __shared__ uint32_t red[C::NW];
        wait_vm<R * CW - kLate>();
        __syncthreads();
        auto quantize = [&](int m, auto threads) __attribute__((always_inline)) {
            const float a = quantize_row<decltype(threads)::value>(
                reinterpret_cast<const TO*>(raw) + m * K, K, red, [&](int c, uint4 q) __attribute__((always_inline)) {
                    *reinterpret_cast<uint4*>(fused_lds + m * Kp + 16 * c) = q;
                });
            if (lane == 0) fused_scale[m] = a;  // (every wave's is the same)
        };
        if (fm <= 2) {  // a row by all waves, or each wave its own rows
            for (int m = 0; m < fm; ++m) quantize(m, std::integral_constant<int, 64 * C::NW>{});
        } else {
            for (int m = wave; m < fm; m += C::NW) quantize(m, std::integral_constant<int, kWave>{});
        }
    }
    wait_vm<(R - U) * CW - kLate>();
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kReads; ++u) read_step(0, 0, 0, u);

    // Stage t: its first k-step's fragments are in registers.  The second's are read under the first's
    // products; then stage t's units are no longer needed: behind the barrier, which also waits for stage
    // t + 1, they take the next units, and the next stage's first fragments are read, under the second
    // k-step's products.
    auto late = [&](int t, int slot, int v) __attribute__((always_inline)) {
        const int u = R * CW - kLate + v, q = u / CW;  // of the ring's order, from stage t's first unit
        copy(t + q / U, q % U, next_slot(slot, q), u % CW);
    };
    auto early = [&](int t, int slot, int u) __attribute__((always_inline)) {
        const int q = R + u / CW;
        copy(t + q / U, q % U, next_slot(slot, u / CW), u % CW);
    };
    int slot = 0;
    if (row0 + 16 * TM * wm < row_end) {
        for (int t = 0; t + 1 < T; ++t) {
            const int next = next_slot(slot, U);
            multiply(0, NReads{}, [&](int u) __attribute__((always_inline)) { read_step(t, slot, 1, u); }, NLate{},
                     [&](int u) __attribute__((always_inline)) { late(t, slot, u); });
            wait_vm<(R - 2 * U) * CW>();
            __syncthreads();
            multiply(1, NReads{}, [&](int u) __attribute__((always_inline)) { read_step(t + 1, next, 0, u); }, NEarly{},
                     [&](int u) __attribute__((always_inline)) { early(t, slot, u); });
            slot = next;
        }
        // the last stage: chunks past K (and k-tiles past the last) count as zero
#pragma unroll
        for (int u = 0; u < kReads; ++u) read_step(T - 1, slot, 1, u);
        const int chunks = (K - ((T - 1) * C::WK + wk) * 128) / 16;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            if (chunks < 8) {
#pragma unroll
                for (int b = 0; b < TM; ++b)
                    if (4 * ks + kg >= chunks) xf[ks][b] = i32x4_t{0, 0, 0, 0};
            }
        multiply(0, None{}, none, None{}, none);
        multiply(1, None{}, none, None{}, none);
    } else {  // no row of this wave's is there: it only makes its copies
        for (int t = 0; t + 1 < T; ++t) {
#pragma unroll
            for (int u = 0; u < kLate; ++u) late(t, slot, u);
            wait_vm<(R - 2 * U) * CW>();
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kEarly; ++u) early(t, slot, u);
            slot = next_slot(slot, U);
        }
    }

    wait_vm<0>();
    __syncthreads();  // no copy is in flight, and every wave is done with the stages
    if constexpr (C::WK > 1) {
        constexpr int kWaves = C::WM * C::WN;
        static_assert((C::WK - 1) * kWaves * TM * TN * 1024 <= R * C::kUnitBytes, "the sums fit in the stages");
        i32x4_t* sums = reinterpret_cast<i32x4_t*>(smem);
        const int w = wm * C::WN + wn;
        if (wk > 0) {
#pragma unroll
            for (int i = 0; i < TM * TN; ++i) sums[(((wk - 1) * kWaves + w) * TM * TN + i) * 64 + lane] = acc[i / TM][i % TM];
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int o = 0; o < C::WK - 1; ++o)
#pragma unroll
            for (int i = 0; i < TM * TN; ++i) acc[i / TM][i % TM] += sums[((o * kWaves + w) * TM * TN + i) * 64 + lane];
    }

    // y = sum * s_n * a_m, 16 rows at a time through this wave's own part of LDS
    constexpr int kPitch = 16 * TN * sizeof(TO) + 16;
    constexpr int kOut0 = C::WK > 1 ? (C::WK - 1) * C::WM * C::WN * TM * TN * 1024 : 0;  // behind the waves' sums
    static_assert(kOut0 + C::WM * C::WN * 16 * kPitch <= R * C::kUnitBytes, "the rows fit in the stages");
    char* buf = smem + kOut0 + (wm * C::WN + wn) * 16 * kPitch;
    const int nw = n0 + 16 * TN * wn;
    float sn[TN][4];
    if constexpr (!kSums) {
#pragma unroll
        for (int a = 0; a < TN; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) sn[a][e] = scales[(size_t)expert * N + min(nw + 16 * a + 4 * kg + e, N - 1)];
    }
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int mb = row0 + 16 * (TM * wm + b);
        if (mb >= row_end) break;
        float am = 1.0f;
        if constexpr (!kSums) am = kFuse ? fused_scale[min(l16, fm - 1)] : ascale[min(mb + l16, row_end - 1)];
#pragma unroll
        for (int a = 0; a < TN; ++a) {
            Pack<TO, 4> o;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kSums)
                    o.v[e] = acc[a][b][e];
                else
                    o.v[e] = from_f32<TO>(scaled_sum(acc[a][b][e], sn[a][e], am));
            }
            *reinterpret_cast<Pack<TO, 4>*>(buf + l16 * kPitch + (16 * a + 4 * kg) * sizeof(TO)) = o;
        }
        wave_lds_sync();
        store_rows<TO, TN>(buf, y, N, mb, nw, row_end);
        wave_lds_sync();
    }
}

// Reads bound it (512 x 4096 in two parts: 3-4 us).  y = (the parts' sums, [parts][M N]) * s_n * a_m: exactly what the
// unsplit product stores.  V columns a thread.
template <typename TO, int V>
__global__ __launch_bounds__(256) void w8a8_join_kernel(const int32_t* __restrict__ sums, int parts,
                                                        const float* __restrict__ ascale, const float* __restrict__ scales,
                                                        int64_t M, int N, TO* __restrict__ y) {
    const int64_t units = M * N / V, step = (int64_t)gridDim.x * 256;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += step) {
        Pack<int32_t, V> sum = load_unit<true, false, V>(sums + V * u);
        for (int p = 1; p < parts; ++p) {
            const Pack<int32_t, V> more = load_unit<true, false, V>(sums + V * (p * units + u));
#pragma unroll
            for (int i = 0; i < V; ++i) sum.v[i] += more.v[i];
        }
        const int64_t m = V * u / N;
        const int n = (int)(V * u - m * N);
        Pack<TO, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = from_f32<TO>(scaled_sum(sum.v[i], scales[n + i], ascale[m]));
        reinterpret_cast<Pack<TO, V>*>(y)[u] = o;
    }
}

struct Product {
    const void* x;  // int8 rows, or activations (fused)
    const float* ascale;
    const int8_t* codes;
    const float* scales;
    int64_t M, N, K;
    const int32_t* offsets;
    int64_t E;
    hipStream_t stream;
    int32_t* sums = nullptr;  // for K in parts, or null
    size_t sums_bytes = 0;
};

// Blocks of a launch: the experts' row tiles are counted on the device, at most this many.
template <typename C>
int64_t launch_blocks(int64_t M, int64_t N, bool experts, int64_t E) {
    return ((N + C::BN - 1) / C::BN) * (experts ? expert_tiles(M, E, C::BM) : (M + C::BM - 1) / C::BM);
}
template <typename C>
bool fits_grid(int64_t M, int64_t N, bool experts, int64_t E) {
    return launch_blocks<C>(M, N, experts, E) < ((int64_t)1 << 31) / (64 * C::NW);  // the grid's threads
}

// The experts that can have rows, and the rows of each if they share them evenly.
struct Share {
    int64_t M, experts, rows;
    Share(int64_t M, int64_t E) : M(M), experts(std::min(M, E)), rows(E == 1 ? M : (M + experts - 1) / experts) {}
    // Row tiles: of several experts whose counts differ, each ends half a tile past its share.
    double row_tiles(int BM) const {
        if (experts == 1) return (double)((M + BM - 1) / BM);
        return std::max((double)experts, (double)M / BM + 0.5 * (double)experts);
    }
};
template <typename C>
bool weights_once(const Share& s, int64_t N, int64_t K) {
    return C::BM <= kOnceRows && s.rows <= C::BM && (double)s.experts * (double)N * (double)K >= kOnceBytes;
}

template <typename C, typename TO>
hipError_t launch_tiles(const Product& p, TO* y) {
    const int64_t tn = (p.N + C::BN - 1) / C::BN;
    const dim3 grid((unsigned)launch_blocks<C>(p.M, p.N, p.offsets != nullptr, p.E)), block(64 * C::NW);
    constexpr int kGroup = C::BM < 256 ? 1024 / C::BM : 4;  // row tiles walked together: about 1024 rows
    auto launch = [&](auto once) {
        constexpr bool kOnce = decltype(once)::value;
        if (p.offsets)
            hipLaunchKernelGGL((w8a8_tile_kernel<TO, kExpertRows, C, kOnce>), grid, block, 0, p.stream, p.x, p.ascale, p.codes,
                               p.scales, y, (int)p.M, (int)p.N, (int)p.K, p.offsets, (int)p.E, (int)tn, kGroup, 0);
        else
            hipLaunchKernelGGL((w8a8_tile_kernel<TO, kRows, C, kOnce>), grid, block, 0, p.stream, p.x, p.ascale, p.codes,
                               p.scales, y, (int)p.M, (int)p.N, (int)p.K, nullptr, 1, (int)tn, kGroup, 0);
        return hipGetLastError();
    };
    if constexpr (C::BM <= kOnceRows) {
        if (weights_once<C>(Share(p.M, p.E), p.N, p.K)) return launch(std::true_type{});
    }
    return launch(std::false_type{});
}

// K in `parts`, one launch for the sums and one that joins them: 100 / 512 rows of 4096 x 14336, weights from HBM, 22.2 /
// 45.1 us against 30.2 / 54.7 unsplit.
template <typename C, typename TO>
hipError_t launch_parts(const Product& p, TO* y, int parts) {
    const int64_t tn = (p.N + C::BN - 1) / C::BN;
    const int64_t split = (p.K + 128 * parts - 1) / (128 * parts) * 128;
    const dim3 grid((unsigned)(launch_blocks<C>(p.M, p.N, false, 1) * parts)), block(64 * C::NW);
    constexpr int kGroup = C::BM < 256 ? 1024 / C::BM : 4;
    hipLaunchKernelGGL((w8a8_tile_kernel<int32_t, kRows, C, false>), grid, block, 0, p.stream, p.x, nullptr, p.codes, nullptr, p.sums,
                       (int)p.M, (int)p.N, (int)p.K, nullptr, 1, (int)tn, kGroup, (int)split);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    auto join = [&](auto v) {
        constexpr int V = decltype(v)::value;
        const int64_t blocks = (p.M * p.N / V + 255) / 256;
        hipLaunchKernelGGL((w8a8_join_kernel<TO, V>), dim3((unsigned)std::min<int64_t>(blocks, kMaxGridBlocks)), dim3(256), 0,
                           p.stream, p.sums, parts, p.ascale, p.scales, p.M, (int)p.N, y);
        return hipGetLastError();
    };
    return p.N % 4 == 0 ? join(std::integral_constant<int, 4>{}) : join(std::integral_constant<int, 1>{});
}

// A join costs a launch and its bytes.
constexpr double kJoinUs = 3.0, kJoinBytesPerUs = 5e6;

// The tilings, and what one costs.  A CU's first block takes `us_ktile` for each 128 of K and `us_first`
// besides, each further one `next_ktile` and `us_next`; `blocks` of them fit a CU.  The weights arrive at 5.6
// TB/s, or 7.3 where they are read once, and neither hides all of the other; a stream of more blocks than run at
// once ends with some of the GPU idle.  Fitted to the tilings' times at 200 shapes of one matrix of 3 to 4096
// rows and 290 of 4 to 256 experts: the choice is on average 1% slower than the fastest tiling for one matrix
// and 2% for experts, whose row counts are not known here, and within 10% of it in 464 of the 490.  (With
// us_first also for further blocks, and time as the larger of the two, 2% and 11%, and up to 2.9 times the
// fastest where K is short.)  It ranks tilings and does not predict times: the clock falls under large products
// (1024 x 14336 x 4096 39.8 us by it, 54 measured), and 7.3 counts the weights of experts that have no rows.
struct Cost {
    double us_ktile, us_first, next_ktile, us_next;
    int blocks;
    double us(double tiles, int64_t K, double weight_bytes, bool once) const {
        const double waves = tiles / 256, up = std::ceil(waves), slots = 256.0 * blocks, ktiles = (double)((K + 127) / 128);
        const double rounds = blocks == 1 ? up : waves <= 1 ? 1.0 : std::max(waves, 0.9 * up);
        const double work = ktiles * us_ktile + us_first + (rounds - 1) * (ktiles * next_ktile + us_next);
        const double tail = tiles > slots ? 1.0 + 0.2 * slots / tiles : 1.0;
        const double stream = weight_bytes / (once ? 7.3e6 : 5.6e6) * tail;
        return 2.6 + std::sqrt(work * work + stream * stream);
    }
};
using T256x256 = Tiling<2, 4, 1, 8, 4, 5, 2>;
using T128x256 = Tiling<2, 4, 1, 4, 4, 3>;
using T128x128 = Tiling<2, 4, 1, 4, 2, 5, 2>;
using T64x128 = Tiling<2, 4, 1, 2, 2, 3>;
using T32x128 = Tiling<2, 4, 1, 1, 2, 4>;
using T64x64 = Tiling<2, 2, 1, 2, 2, 4>;
using T32x32 = Tiling<2, 2, 2, 1, 1, 4>;
using T16x64 = Tiling<1, 4, 1, 1, 1, 4>;
using T16x32 = Tiling<1, 2, 2, 1, 1, 4>;
using T16x16 = Tiling<1, 1, 4, 1, 1, 6>;

// The tiling for a product and the parts K is taken in (1 where `sums` has no room for more).  Parts are whole
// k-tiles, none empty, of at least 16.
struct Plan {
    int tiling, parts;
};
template <typename F>
void each_tiling(F f) {
    f(0, T256x256{}, Cost{1.06, 1.8, 1.27, 5.5, 1});
    f(1, T128x256{}, Cost{0.73, 1.5, 0.81, 5.9, 1});
    f(2, T128x128{}, Cost{0.51, 0.1, 0.49, 2.3, 2});
    f(3, T64x128{}, Cost{0.36, 0.3, 0.38, 1.6, 2});
    f(4, T32x128{}, Cost{0.31, 0.5, 0.3, 1.8, 2});
    f(5, T64x64{}, Cost{0.25, 0.5, 0.23, 1.3, 2});
    f(6, T32x32{}, Cost{0.12, 0.6, 0.098, 1.4, 2});
    f(7, T16x64{}, Cost{0.22, 0.2, 0.12, 0.7, 4});
    f(8, T16x32{}, Cost{0.11, 0.3, 0.062, 0.9, 3});
    f(9, T16x16{}, Cost{0.066, 0.8, 0.051, 2.8, 1});
}
size_t sums_bytes(int64_t M, int64_t N, int parts) { return parts > 1 ? (size_t)parts * (size_t)M * (size_t)N * 4 : 0; }

Plan plan_product(int64_t M, int64_t N, int64_t K, bool experts, int64_t E, size_t room) {
    const Share share(M, E);
    const int64_t ktiles = (K + 127) / 128;
    const double weight_bytes = (double)share.experts * (double)N * (double)K;
    Plan plan{-1, 1};
    double least = 0;
    each_tiling([&](int i, auto tiling, Cost cost) {
        using C = decltype(tiling);
        if (!fits_grid<C>(M, N, experts, E)) return;
        const double tiles = share.row_tiles(C::BM) * (double)((N + C::BN - 1) / C::BN);
        const bool once = weights_once<C>(share, N, K);
        const int most = experts || C::WK > 1 || C::BM * C::BN < 64 * 64 || room == 0 || ktiles < 32 ? 0 : 3;
        for (int log = 0; log <= most; ++log) {  // (a plan takes 0.1 us of host time, a launch 3.4)
            const int parts = 1 << log;
            const int64_t part = (ktiles + parts - 1) >> log;
            if (parts > 1 && (tiles * parts > 512 || part < 16 || part * (parts - 1) >= ktiles || sums_bytes(M, N, parts) > room))
                break;
            // the parts' sums are written and read once, and joined by a second launch; a part's weights are copied
            // in the caches' usual order (launch_parts)
            const double join = parts > 1 ? kJoinUs + 2.0 * sums_bytes(M, N, parts) / kJoinBytesPerUs : 0.0;
            const double us = cost.us(tiles * parts, part * 128, weight_bytes, once && parts == 1) + join;
            if (plan.tiling < 0 || us < least) plan = Plan{i, parts}, least = us;
        }
    });
    return plan;
}

template <typename TO>
hipError_t launch_product(const Product& p, TO* y) {
    const Plan plan = plan_product(p.M, p.N, p.K, p.offsets != nullptr, p.E, p.sums != nullptr ? p.sums_bytes : 0);
    hipError_t e = hipErrorInvalidConfiguration;
    each_tiling([&](int i, auto tiling, Cost) {
        using C = decltype(tiling);
        if (i != plan.tiling) return;
        if constexpr (C::WK == 1 && C::BM * C::BN >= 64 * 64) {
            if (plan.parts > 1) {
                e = launch_parts<C>(p, y, plan.parts);
                return;
            }
        }
        e = launch_tiles<C>(p, y);
    });
    return e;
}

// x quantized by every block for itself: its tile's rows.
template <typename TO>
size_t fused_bytes(const Product& p, int wk) {
    const int64_t rows = std::min<int64_t>(p.M, 16);
    return (size_t)(fused_codes_bytes(rows, p.K, wk) + fused_raw_bytes(rows, p.K, sizeof(TO)));
}
template <typename C, typename TO>
hipError_t launch_fused_tiles(const Product& p, TO* y) {
    const int64_t tn = (p.N + C::BN - 1) / C::BN, tm = (p.M + 15) / 16;
    auto launch = [&](auto once) {
        hipLaunchKernelGGL((w8a8_tile_kernel<TO, kFused, C, decltype(once)::value>), dim3((unsigned)(tn * tm)), dim3(64 * C::NW),
                           fused_bytes<TO>(p, C::WK), p.stream, p.x, nullptr, p.codes, p.scales, y, (int)p.M, (int)p.N,
                           (int)p.K, nullptr, 1, (int)tn, 64, 0);
        return hipGetLastError();
    };
    return weights_once<C>(Share(p.M, 1), p.N, p.K) ? launch(std::true_type{}) : launch(std::false_type{});
}
using F16x32 = Tiling<1, 2, 2, 1, 1, 4, 1, false>;
using F16x16 = Tiling<1, 1, 4, 1, 1, 6, 1, false>;
using F16x16K8 = Tiling<1, 1, 8, 1, 1, 2, 1, false>;

// One launch for activations where quantizing them in every block costs less than a launch of its own (weights from
// HBM; us of one launch against two):
//  - one or two rows, in tiles as wide as leave no CU more than one block (16 columns up to N = 4096: K = 4096, N =
//    4096, bf16 6.4 against 9.8, two rows 7.6 against 9.5), else 32 columns (N = 14336 14.1 against 18.1, two rows
//    15.0 against 19.1).  More than one block a CU wants room for two at once (two rows of K = 8192, one block at a
//    time: N = 14336 31.1 against 25.6, N = 28672 59.1 against 48.6), and a CU that quantizes at most eight rows
//    in all (two rows of K = 1024, N = 57344 18.5 against 16.1, N = 131072 34.5 against 26.1; K = 4096, N = 28672
//    25.1 against 28.9);
//  - up to 256 tiles of 16 rows x 16 columns, a CU each.  A wave quantizes whole rows, so beyond two rows short ones
//    and few activations in all (bf16, N = 4096: 4 rows of K = 2048 6.5 against 8.1, of 4096 9.7 against 9.4, of 8192
//    16.6 against 13.8; 8 of 2048 7.5 against 8.4; 16 of 1024 6.9 against 7.3, of 1360 10.0 against 8.5; fp32 16 of
//    1360 7.4 against 7.9, 3 of 8192 19.7 against 12.7); one or two rows, by all eight waves, up to 96 KB (bf16
//    32768 of K, N = 2048 30.2 against 37.6, fp32 16384 15.5 against 18.8, 24576 25.9 against 22.6).
constexpr int64_t kFusedRows = 2, kFusedRowsPerCU = 8;
constexpr size_t kFusedBytes = 48 << 10, kFusedLongBytes = 96 << 10;
constexpr int64_t kFusedTileK = 2816;
constexpr size_t kLdsBytes = 160 << 10, kFusedLdsMore = 1 << 10;  // (scales and maxima)
template <typename TO>
auto fused_launch(const Product& p) -> hipError_t (*)(const Product&, TO*) {
    // Blocks that fit a CU at once, by their LDS.
    auto blocks = [&](auto tiling) {
        using C = decltype(tiling);
        return kLdsBytes / (fused_bytes<TO>(p, C::WK) + C::R * C::kUnitBytes + kFusedLdsMore);
    };
    if (p.M <= kFusedRows) {
        if (p.N <= 16 * 256) {
            if (fused_bytes<TO>(p, F16x16::WK) <= kFusedBytes) return launch_fused_tiles<F16x16, TO>;
        } else if (fused_bytes<TO>(p, F16x32::WK) <= kFusedBytes) {
            const int64_t tiles = launch_blocks<F16x32>(p.M, p.N, false, 1);
            if (blocks(F16x32{}) >= (tiles > 256 ? 2 : 1) && tiles * p.M <= 256 * kFusedRowsPerCU)
                return launch_fused_tiles<F16x32, TO>;
        }
    }
    using C = F16x16K8;
    const int64_t rows = std::min<int64_t>(p.M, 16), acts = rows * p.K;
    const bool few = rows <= kFusedRows ? fused_bytes<TO>(p, C::WK) <= kFusedLongBytes
                                        : p.K <= kFusedTileK && acts <= (sizeof(TO) == 2 ? 16 : 24) << 10;
    if (few && launch_blocks<C>(p.M, p.N, false, 1) <= 256 && blocks(C{}) >= 1) return launch_fused_tiles<C, TO>;
    return nullptr;
}

}  // namespace

hipError_t launch_quant_rows_i8(int dtype, const void* x, int64_t M, int64_t K, int8_t* xq, float* ascale,
                                hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        auto run = [&](auto waves) {
            constexpr int kWaves = decltype(waves)::value;
            const dim3 grid((unsigned)std::min<int64_t>((M + 4 / kWaves - 1) / (4 / kWaves), kMaxGridBlocks));
            hipLaunchKernelGGL((quant_rows_i8_kernel<T, kWaves>), grid, dim3(256), 0, stream, static_cast<const T*>(x), M,
                               (int)K, xq, ascale);
            return hipGetLastError();
        };
        return row_by_wave(M, K) ? run(std::integral_constant<int, 1>{}) : run(std::integral_constant<int, 4>{});
    });
}

bool w8a8_fits_grid(int64_t M, int64_t N, bool experts, int64_t E) { return fits_grid<T256x256>(M, N, experts, E); }

size_t w8a8_sums_bytes(int64_t M, int64_t N, int64_t K) {
    return sums_bytes(M, N, plan_product(M, N, K, false, 1, ~(size_t)0).parts);
}

hipError_t launch_matmul_w8a8(int dtype, const void* x, int64_t M, const int8_t* codes, const float* scales, int64_t N,
                              int64_t K, void* y, int8_t* xq, float* ascale, int32_t* sums, size_t sums_bytes,
                              hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        const Product fused{x, nullptr, codes, scales, M, N, K, nullptr, 1, stream};
        if (const auto launch = fused_launch<T>(fused)) return launch(fused, static_cast<T*>(y));
        if (const hipError_t e = launch_quant_rows_i8(dtype, x, M, K, xq, ascale, stream); e != hipSuccess) return e;
        return launch_product<T>(Product{xq, ascale, codes, scales, M, N, K, nullptr, 1, stream, sums, sums_bytes},
                                 static_cast<T*>(y));
    });
}

hipError_t launch_gemm_w8a8(int dtype, const int8_t* xq, const float* ascale, int64_t M, const int8_t* codes,
                            const float* scales, int64_t N, int64_t K, void* y, const int32_t* offsets, int64_t E,
                            int32_t* sums, size_t sums_bytes, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        return launch_product<T>(Product{xq, ascale, codes, scales, M, N, K, offsets, E, stream, sums, sums_bytes},
                                 static_cast<T*>(y));
    });
}

}  // namespace w4a16

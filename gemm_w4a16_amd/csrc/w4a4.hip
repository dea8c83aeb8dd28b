// w4a4.hip -- W4A4: activations and weights both in the microscaled 4-bit format (mx4.h), on the scaled matrix
// instructions.
//
//     y[m][n] = sum_b 2^(sx[m][b] + sw[n][b] - 254) sum_{k in block b} p[m][k] q[n][k]
// with the products of elements exact and the sums in fp32, rounded once to the output type.  An instruction
// multiplies 16 rows by 16 columns over 128 of K, each lane's 32 elements with the scale of their block; the order of
// additions follows from the sizes alone, so results are bitwise reproducible.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>
#include <utility>

#include "experts.h"
#include "launch.h"
#include "lds_dma.h"
#include "mx4.h"

namespace w4a16 {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4v_t __attribute__((ext_vector_type(4)));

template <int... I, typename F>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>{}), ...);
}

// acc += the product of 16 weight rows and 16 activation rows over 128 of K; byte kWSel of a lane's word of scales is
// that of its weight block, kXSel alike.
template <int kWSel, int kXSel>
__device__ __forceinline__ f32x4v_t mfma(i32x4_t w, i32x4_t x, f32x4v_t acc, int wscale, int xscale) {
    const i32x8_t a = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8_t b = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, 4, kWSel, wscale, kXSel, xscale);  // (4: e2m1)
}
constexpr int kOnes = 0x7F7F7F7F;  // scales of one, for blocks past K (their elements are zero)

// ---- tiles --------------------------------------------------------------------------------------

// A block computes BM rows x BN columns in WM x WN waves of (16 TM) x (16 TN), each doubled WK times along K.  K is
// taken in stages of WK k-tiles of 256 (128 bytes of codes a row); the waves of index wk along K multiply k-tile wk of a
// stage, and their sums are added at the end, in order.  Operands and scales reach LDS by direct copies into a ring
// of R stages.  kX = false: x is not in the ring (which holds weights alone) but whole in LDS behind it, quantized by
// the block from activations.
//
// What bounds it.  1024 x 14336 x 4096 takes 32-35 us in 256 x 256 tiles (3.4-3.7 PFLOP/s; the instructions alone reach 9.0 on
// zeros and 6.3-6.9 on random bits), 8192 rows 240-257 (3.7-4.0), 8192 cubed 245-265 (4.15-4.5; hipBLASLt's product of this format
// 314-327).  A k-tile is 2048 cycles of matrix instructions a SIMD
// beside 2080 of LDS reads and writes a CU, so neither hides all of the other: 1.3 us a k-tile without copies, 1.7 with
// (timing-only copies; 0.9 by the products alone).  The outputs, which all blocks write at once, are 5 us of the 32,
// scale copies 1.  Four waves of 128 x 128, one a SIMD, read a third less from LDS and take 40.  Few rows: the weights'
// stream and a block's chain of k-tiles (64 rows 8.8 us, 256 rows 14).
template <int WM_, int WN_, int WK_, int TM_, int TN_, int R_, bool kX_ = true>
struct Tiling {
    static constexpr int WM = WM_, WN = WN_, WK = WK_, TM = TM_, TN = TN_, R = R_;
    static constexpr bool kX = kX_;
    static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, NW = WM * WN * WK;
    static constexpr int kTileBytes = ((kX ? BM : 0) + BN) * 128;  // one k-tile: BN rows of weights, then BM rows of x
    static constexpr int GW = (BN + 31) / 32, GX = (BM + 31) / 32;  // groups of scales: weights', then x's
    static constexpr int kGroups = GW + (kX ? GX : 0), kScaleBytes = kGroups * 256;
    static constexpr int kCodes = WK * kTileBytes;  // of a stage; the scales of its k-tiles lie behind them
    static constexpr int kScaleCopies = (WK * kScaleBytes + 1023) / 1024;
    static constexpr int kStage = kCodes + 1024 * kScaleCopies;
    static constexpr int CW = (kCodes / 1024 + NW - 1) / NW;      // copies of 1 KB by a wave (the last ones may be made twice)
    static constexpr int SW = (kScaleCopies + NW - 1) / NW;
};

constexpr int kFusedUnits = 4;  // of 8 activations that a lane asks for at a time
// LDS behind the ring for activations quantized by the block: codes and scales of its rows, K up to whole stages.
template <typename C>
constexpr size_t fused_bytes(int64_t K) {
    return (size_t)((mx4_ktiles(K) + C::WK - 1) / C::WK * C::WK) * (C::BM * 128 + C::GX * 256);
}

// TX: uint8_t for rows in the format, or the type of activations (C::kX false).
template <typename TO, typename TX, typename C>
__global__ __launch_bounds__(64 * C::NW) void w4a4_tile_kernel(const TX* __restrict__ x, const uint8_t* __restrict__ xscales,
                                                               int M, const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int N, int stride,
                                                               TO* __restrict__ y, int n_tiles, int group) {
    constexpr int TM = C::TM, TN = C::TN, R = C::R, BM = C::BM, BN = C::BN, CW = C::CW, SW = C::SW, G = CW + SW;
    constexpr int kTileCopies = C::kTileBytes / 1024;  // of one k-tile
    static_assert(C::kX == std::is_same_v<TX, uint8_t>, "activations are quantized by the block");
    static_assert(C::kX || BM % 32 == 0, "whole groups of scales");
    __shared__ __attribute__((aligned(1024))) char smem[R * C::kStage];
    extern __shared__ __attribute__((aligned(1024))) char fused_lds[];
    const int lane = lane_id(), wave = wave_id();
    const int l16 = lane & 15, kg = lane >> 4;
    const int wn = wave % C::WN, wk = wave / C::WN % C::WK, wm = wave / (C::WN * C::WK);

    // This block's tile.  Blocks go to the XCDs in turn: each XCD takes a contiguous eighth of the tile
    // sequence, which walks `group` row tiles at a time, rows first, so that the blocks of one XCD share
    // operands in its L2.
    int row0, tn;
    {
        const int m_tiles = (M + BM - 1) / BM, total = m_tiles * n_tiles, b = blockIdx.x;
        const int xcd = b & 7, each = total >> 3, rest = total & 7;
        const int s = xcd * each + min(xcd, rest) + (b >> 3);
        const int g = s / (group * n_tiles), in = s - g * group * n_tiles;
        const int rows = min(group, m_tiles - g * group);
        tn = in / rows;
        row0 = (g * group + in - tn * rows) * BM;
    }
    const int n0 = tn * BN;
    const int S = stride;  // bytes of a row of codes
    const int KT = (S + 127) / 128, T = (KT + C::WK - 1) / C::WK;
    const uint8_t* wbase = codes + (size_t)n0 * S;
    const uint8_t* xbase = C::kX ? reinterpret_cast<const uint8_t*>(x) + (size_t)row0 * S : nullptr;
    const uint32_t lds0 = lds_addr(smem);

    // This wave's copies j = CW wave + i of a stage's codes: copy jj = j % kTileCopies of k-tile j / kTileCopies, rows
    // 8 jj + lane / 8 of [weights; x].  LDS slot lane % 8 of a row takes its 16-byte chunk
    // slot ^ ((row >> 1) & 7), so that the fragment reads below meet no bank twice.  Rows past the end
    // read the last row; they are never stored.
    uint32_t voff[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        const int jj = min(CW * wave + i, C::kCodes / 1024 - 1) % kTileCopies;
        const int r = 8 * jj + lane / 8, chunk = (lane % 8) ^ ((r >> 1) & 7);
        const int row = !C::kX || jj < BN / 8 ? min(r, N - 1 - n0) : min(r - BN, M - 1 - row0);
        voff[i] = (uint32_t)row * (uint32_t)S + 16u * chunk;
    }
    // ... and its 16 bytes of the stage's scales: groups past the last read the last one
    const char* sptr[SW];
    int64_t sstep[SW];
    int stile[SW];
#pragma unroll
    for (int i = 0; i < SW; ++i) {
        const int c = min(64 * min(SW * wave + i, C::kScaleCopies - 1) + lane, C::WK * C::kScaleBytes / 16 - 1);
        const int g = c / 16 % C::kGroups;
        const int64_t gw = mx4_groups(N), gx = mx4_groups(M);
        stile[i] = c / 16 / C::kGroups;
        const bool w = !C::kX || g < C::GW;
        const int64_t at = w ? min((int64_t)(n0 / 32 + g), gw - 1) : min((int64_t)(row0 / 32 + g - C::GW), gx - 1);
        sptr[i] = reinterpret_cast<const char*>(w ? scales : xscales) + at * 256 + c % 16 * 16;
        sstep[i] = (w ? gw : gx) * 256;
    }
    // copy i of stage t into ring slot `slot`; the last k-tile's chunks past K, and k-tiles past the last, read what is there
    // (their products are masked).  Stages past the last read one line over and over: each stage is then the same
    // number of copies, and every wait below is a constant.
    auto copy = [&](int t, int slot, int i) __attribute__((always_inline)) {
        if (i < CW) {
            const int j = min(CW * wave + i, C::kCodes / 1024 - 1), jj = j % kTileCopies;
            const int kt = min(t * C::WK + j / kTileCopies, KT - 1);
            const uint8_t* base = (!C::kX || jj < BN / 8 ? wbase : xbase) + (size_t)kt * 128;
            // (no branches: the compiler would move products across them, and past the barriers)
            const int over = 16 * ((lane % 8) ^ ((4 * jj + lane / 16) & 7)) + 16 - (S - kt * 128);
            const uint32_t off = (voff[i] - (uint32_t)max(over, 0)) & (t < T ? ~0u : 0u);
            dma16(off, base, lds0 + (uint32_t)(slot * C::kStage + 1024 * j));
        } else {
            const int s = i - CW, j = min(SW * wave + s, C::kScaleCopies - 1);
            const int kt = min(t * C::WK + stile[s], KT - 1);
            dma16_at(sptr[s] + kt * sstep[s], lds0 + (uint32_t)(slot * C::kStage + C::kCodes + 1024 * j));
        }
    };

    // fragment of row tile rt at k-step ks of a k-tile: chunk 4 ks + kg of row 16 rt + l16
    const char* frag0 = smem + wk * C::kTileBytes + 128 * l16;
    const int sw = (l16 >> 1) & 7;
    auto next_slot = [](int s) __attribute__((always_inline)) { return s + 1 >= R ? s + 1 - R : s + 1; };
    auto read = [&](int slot, int ks, int rt) __attribute__((always_inline)) {
        return *reinterpret_cast<const i32x4_t*>(frag0 + slot * C::kStage + 2048 * rt + 16 * ((4 * ks + kg) ^ sw));
    };
    const int w_rt = TN * wn, x_rt = BN / 16 + TM * wm;
    // x quantized by the block: codes [k-tile][BM] as above, then scales [k-tile][GX][64]
    const int KTp = T * C::WK;
    char* fused_scales = fused_lds + (size_t)KTp * BM * 128;
    auto read_fused = [&](int t, int ks, int b) __attribute__((always_inline)) {
        return *reinterpret_cast<const i32x4_t*>(fused_lds + ((t * C::WK + wk) * BM + 16 * (TM * wm + b) + l16) * 128 + 16 * ((4 * ks + kg) ^ sw));
    };
    // words of scales: of two row tiles each (TN, TM even), or the half of one that is this row tile's
    constexpr int NS = (TN + 1) / 2, MS = (TM + 1) / 2;
    const char* scale0 = smem + C::kCodes + wk * C::kScaleBytes + 4 * lane;
    auto read_scale = [&](int t, int slot, int i) __attribute__((always_inline)) {
        if (!C::kX && i >= NS)
            return *reinterpret_cast<const int*>(fused_scales + ((t * C::WK + wk) * C::GX + TM * wm / 2 + i - NS) * 256 + 4 * lane);
        const int g = i < NS ? TN * wn / 2 + i : C::GW + TM * wm / 2 + i - NS;
        return *reinterpret_cast<const int*>(scale0 + slot * C::kStage + 256 * g);
    };
    const int w_shift = TN == 1 ? 16 * ((n0 / 16 + wn) & 1) : 0, x_shift = TM == 1 ? 16 * ((row0 / 16 + wm) & 1) : 0;

    f32x4v_t acc[TN][TM];
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) acc[a][b] = f32x4v_t{0, 0, 0, 0};
    // Activation fragments of wide wave tiles are read in place, each behind the products that take it; narrow ones
    // are read a step ahead into registers of their own.  (Both for 128 x 64 spill.)
    constexpr bool kInPlace = TM >= 4;
    i32x4_t wf[2][TN], xf[kInPlace ? 1 : 2][TM];
    int sc[NS + MS], sc_next[NS + MS];  // of this stage's k-tile (both k-steps), and of the next's

    // The products of k-step ks, rows of x one after another, with `reads` reads and `copies` copies among them: the copies
    // and, where fragments have registers of their own, the reads spread over all and over the first three quarters;
    // else x fragment b behind its products, the others within the first half.
    auto multiply = [&](auto step, auto reads, auto read, auto copies, auto copy) __attribute__((always_inline)) {
        constexpr int ks = decltype(step)::value, H = TM * TN, HR = kInPlace ? (H + 1) / 2 : (3 * H + 3) / 4;
        constexpr int nr = decltype(reads)::value, nc = decltype(copies)::value;
        constexpr int first = kInPlace && nr > 0 ? TM : 0;  // (reads 0.. TM - 1 are the x fragments)
        each(std::make_integer_sequence<int, H>{}, [&](auto index) __attribute__((always_inline)) {
            constexpr int i = decltype(index)::value, a = i % TN, b = i / TN, n = nr - first;
#pragma unroll
            for (int u = (i * n + HR - 1) / HR; u < min(n, ((i + 1) * n + HR - 1) / HR); ++u) read(first + u);
#pragma unroll
            for (int u = (i * nc + H - 1) / H; u < ((i + 1) * nc + H - 1) / H; ++u) copy(u);
            acc[a][b] = mfma<(TN == 1 ? 0 : a % 2 * 2) + ks, (TM == 1 ? 0 : b % 2 * 2) + ks>(
                wf[ks][a], xf[kInPlace ? 0 : ks][b], acc[a][b], sc[a / 2], sc[NS + b / 2]);
            if (first > 0 && a == TN - 1) read(b);
            if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            if (i == 0) __builtin_amdgcn_s_setprio(1);
            if (i == H - 1) __builtin_amdgcn_s_setprio(0);
        });
    };
    // read u of stage t, in ring slot `slot`: fragments, and with the first k-step's the scales
    auto read_step = [&](int t, int slot, int ks, int u) __attribute__((always_inline)) {
        if (u < TM) {
            if constexpr (C::kX)
                xf[kInPlace ? 0 : ks][u] = read(slot, ks, x_rt + u);
            else
                xf[kInPlace ? 0 : ks][u] = read_fused(t, ks, u);
        } else if (u < TM + TN) {
            wf[ks][u - TM] = read(slot, ks, w_rt + u - TM);
        } else {
            const int i = u - TM - TN;
            sc_next[i] = read_scale(t, slot, i) >> (i < NS ? w_shift : x_shift);
        }
    };
    auto take_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NS + MS; ++i) sc[i] = sc_next[i];
    };
    constexpr int kReads = TM + TN, kFirst = kReads + NS + MS;
    // Behind stage t's barrier its slot takes stage t + R, G copies: kEarly of them under the stage's second k-step,
    // the others under the next stage's first (where the ring holds more than two stages; else the next barrier
    // would wait for copies just made).
    constexpr int kEarly = R > 2 ? G / 2 : G, kLate = G - kEarly;
    using NReads = std::integral_constant<int, kReads>;
    using NFirst = std::integral_constant<int, kFirst>;
    using NEarly = std::integral_constant<int, kEarly>;
    using NLate = std::integral_constant<int, kLate>;
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    auto none = [](int) {};

    static_assert(R * G < 64, "the wait counts");
#pragma unroll
    for (int u = 0; u < R * G - kLate; ++u) copy(u / G, u / G, u % G);
    if constexpr (!C::kX) {  // a wave a row, 8 values a lane, four lanes a block of the format; four units' loads
                           // before the first is waited for
        constexpr int V = 16 / sizeof(TX), kLoads = 8 / V, kAtOnce = kFusedUnits;
        const int K8 = S / 4, rows = min(BM, M - row0);
        const TX* rows_of_x = x + (size_t)row0 * (2 * S);
        for (int r = wave, c = lane; r < rows;) {
            Pack<TX, V> p[kAtOnce][kLoads];
            int rr[kAtOnce], cc[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                rr[i] = r, cc[i] = c;
#pragma unroll
                for (int h = 0; h < kLoads; ++h)
                    p[i][h] = r < rows && c < K8 ? load_unit<false, false, V>(rows_of_x + (size_t)r * (2 * S) + 8 * c + V * h) : Pack<TX, V>{};
                c += 64;
                if (c - lane >= K8) c = lane, r += C::NW;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const TX* v = p[i][0].v;  // (a unit's packs are one array of 8)
                const uint32_t s = mx4_scale(mx4_max_quad(mx4_max_bits<8>(v))), w = mx4_codes<8>(v, s);
                if (rr[i] < rows && cc[i] < K8) {
                    const int b = cc[i] / 4, kt = b / 8, chunk = b % 8 ^ ((rr[i] >> 1) & 7);
                    *reinterpret_cast<uint32_t*>(fused_lds + (kt * BM + rr[i]) * 128 + 16 * chunk + 4 * (cc[i] % 4)) = w;
                    if (cc[i] % 4 == 0) fused_scales[mx4_scale_at(C::GX, rr[i], b)] = (char)s;
                }
            }
        }
    }
    wait_vm<(R - 1) * G - kLate>();
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kFirst; ++u) read_step(0, 0, 0, u);
    take_scales();

    // Stage t: its first k-step's fragments and its scales are in registers.  The second's are read under the first's
    // products; then the stage is no longer needed: behind the barrier, which also waits for stage t + 1, its slot takes the
    // next copies, and the next stage's first fragments are read, under the second k-step's products.
    int slot = 0;
    if (row0 + 16 * TM * wm < M) {
        for (int t = 0; t + 1 < T; ++t) {
            const int next = next_slot(slot);
            const int before = slot == 0 ? R - 1 : slot - 1;  // stage t + R - 1's slot
            multiply(Zero{}, NReads{}, [&](int u) __attribute__((always_inline)) { read_step(t, slot, 1, u); }, NLate{},
                     [&](int u) __attribute__((always_inline)) { copy(t + R - 1, before, kEarly + u); });
            wait_vm<(R - 2) * G>();
            __syncthreads();
            multiply(One{}, NFirst{}, [&](int u) __attribute__((always_inline)) { read_step(t + 1, next, 0, u); }, NEarly{},
                     [&](int u) __attribute__((always_inline)) { copy(t + R, slot, u); });
            take_scales();
            slot = next;
        }
        // the last stage: blocks past K (and k-tiles past the last) count as zero
        if constexpr (!kInPlace) {
#pragma unroll
            for (int u = 0; u < kReads; ++u) read_step(T - 1, slot, 1, u);
        }
        const int chunks = (S - ((T - 1) * C::WK + wk) * 128) / 16;
        auto mask = [&](int ks) __attribute__((always_inline)) {
            if (4 * ks + kg < chunks) return;
#pragma unroll
            for (int b = 0; b < TM; ++b) xf[kInPlace ? 0 : ks][b] = i32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NS + MS; ++i) sc[i] = kOnes;  // (a lane's second block lies past its first)
        };
        mask(0);
        if constexpr (kInPlace)
            multiply(Zero{}, NReads{}, [&](int u) __attribute__((always_inline)) { read_step(T - 1, slot, 1, u); }, Zero{}, none);
        else
            multiply(Zero{}, Zero{}, none, Zero{}, none);
        mask(1);
        multiply(One{}, Zero{}, none, Zero{}, none);
    } else {  // no row of this wave's is there: it only makes its copies
        for (int t = 0; t + 1 < T; ++t) {
            const int before = slot == 0 ? R - 1 : slot - 1;
#pragma unroll
            for (int u = 0; u < kLate; ++u) copy(t + R - 1, before, kEarly + u);
            wait_vm<(R - 2) * G>();
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kEarly; ++u) copy(t + R, slot, u);
            slot = next_slot(slot);
        }
    }

    wait_vm<0>();
    __syncthreads();  // no copy is in flight, and every wave is done with the stages
    if constexpr (C::WK > 1) {
        constexpr int kWaves = C::WM * C::WN;
        static_assert((C::WK - 1) * kWaves * TM * TN * 1024 <= R * C::kStage, "the sums fit in the stages");
        f32x4v_t* sums = reinterpret_cast<f32x4v_t*>(smem);
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

    // 16 rows at a time through this wave's own part of LDS
    constexpr int kPitch = 16 * TN * sizeof(TO) + 16;
    constexpr int kOut0 = C::WK > 1 ? (C::WK - 1) * C::WM * C::WN * TM * TN * 1024 : 0;  // behind the waves' sums
    static_assert(kOut0 + C::WM * C::WN * 16 * kPitch <= R * C::kStage, "the rows fit in the stages");
    char* buf = smem + kOut0 + (wm * C::WN + wn) * 16 * kPitch;
    const int nw = n0 + 16 * TN * wn;
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int mb = row0 + 16 * (TM * wm + b);
        if (mb >= M) break;
#pragma unroll
        for (int a = 0; a < TN; ++a) {
            Pack<TO, 4> o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o.v[e] = from_f32<TO>(acc[a][b][e]);
            *reinterpret_cast<Pack<TO, 4>*>(buf + l16 * kPitch + (16 * a + 4 * kg) * sizeof(TO)) = o;
        }
        wave_lds_sync();
        store_rows<TO, TN>(buf, y, N, mb, nw, M);
        wave_lds_sync();
    }
}

// ---- few rows -----------------------------------------------------------------------------------

// Up to 16 rows: a block computes 16 columns, its waves every kWaves-th k-tile each, from a ring of its own in LDS (R
// stages of one k-tile), with no barrier until their sums are added, in the order of waves.  TX uint8_t: rows in
// the format (kRows of them staged).  Else activations, one or two rows, that each lane quantizes as the block
// that it multiplies: a block's 32 values are one lane's part of an operand, so nothing is exchanged.
template <typename TX, int kRows>
struct RowShape {
    static constexpr bool kFused = !std::is_same_v<TX, uint8_t>;
    static constexpr int kXBytes = kFused ? kRows * kMx4TileK * (int)sizeof(TX) : kRows * 128;
    static constexpr int kScales = 2048, kX = kScales + 1024, kStage = kX + kXBytes;  // weights, scales, rows
    static constexpr int kOwn = kFused ? kRows * 256 : 0;  // a wave's codes [row][128] and scales, behind the ring
    static constexpr int kXCopies = kXBytes / 1024, kCopies = 2 + 1 + kXCopies;
    static constexpr int R = kFused && kRows > 4 ? 1 : 2;  // (three or four: fewer blocks a CU, 0-20% slower)
    static_assert(kXBytes % 1024 == 0, "whole copies");
};

template <typename TO, typename TX, int kRows, int kWaves, bool kOnce>
__global__ __launch_bounds__(64 * kWaves) void w4a4_rows_kernel(const TX* __restrict__ x, const uint8_t* __restrict__ xscales,
                                                                   int M, const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales, int N, int S,
                                                                   TO* __restrict__ y) {
    using C = RowShape<TX, kRows>;
    constexpr int R = C::R;
    __shared__ __attribute__((aligned(1024))) char smem[kWaves * (R * C::kStage + C::kOwn)];
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, kg = lane >> 4;
    const int n0 = blockIdx.x * 16, KT = (S + 127) / 128, T = (KT - wave + kWaves - 1) / kWaves;
    char* ring = smem + wave * R * C::kStage;
    const uint32_t ring_lds = lds_addr(ring);
    const uint8_t* wbase = codes + (size_t)n0 * S;
    // this lane's 16 bytes of the scales: the weights' in lanes 0..15, x's in the others
    const int64_t gw = mx4_groups(N);
    const bool of_x = !C::kFused && lane >= 16;
    const char* sptr = reinterpret_cast<const char*>(of_x ? xscales : scales + n0 / 32 * (int64_t)256) + lane % 16 * 16;
    const int64_t sstep = of_x ? 256 : gw * 256;  // (one group of rows)

    // LDS slot lane % 8 of a row takes its 16-byte chunk slot ^ ((row >> 1) & 7)
    auto chunk_of = [&](int r) __attribute__((always_inline)) { return (lane % 8) ^ ((r >> 1) & 7); };
    auto issue = [&](int t, int slot) __attribute__((always_inline)) {
        const int kt = min(t * kWaves + wave, KT - 1);  // (past the last: as many copies of the last)
        const uint32_t lds = ring_lds + (uint32_t)(slot * C::kStage);
        const int last = S - 16;  // of a row; chunks past K read it (their products are masked)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 8 * i + lane / 8;
            const uint32_t off = (uint32_t)min(r, N - 1 - n0) * (uint32_t)S + (uint32_t)min(kt * 128 + 16 * chunk_of(r), last);
            if constexpr (kOnce)
                dma16_once(off, wbase, lds + 1024 * i);
            else
                dma16(off, wbase, lds + 1024 * i);
        }
        dma16_at(sptr + kt * sstep, lds + C::kScales);
        if constexpr (C::kFused) {
            constexpr int kRowBytes = kMx4TileK * sizeof(TX);  // of a row in a k-tile
#pragma unroll
            for (int i = 0; i < C::kXCopies; ++i) {
                const int b = 1024 * i + 16 * lane, r = min(b / kRowBytes, M - 1);
                const int at = min(kt * kRowBytes + b % kRowBytes, 2 * S * (int)sizeof(TX) - 16);
                dma16((uint32_t)r * (uint32_t)(2 * S * sizeof(TX)) + (uint32_t)at, x, lds + C::kX + 1024 * i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < C::kXCopies; ++i) {
                const int r = 8 * i + lane / 8;
                dma16((uint32_t)min(r, M - 1) * (uint32_t)S + (uint32_t)min(kt * 128 + 16 * chunk_of(r), last), x, lds + C::kX + 1024 * i);
            }
        }
    };
    f32x4v_t acc = {0, 0, 0, 0};
    const int w_shift = 16 * ((n0 / 16) & 1), sw = (l16 >> 1) & 7;
#pragma unroll
    for (int t = 0; t < R - 1; ++t) issue(t, t);
    int slot = 0;
    for (int t = 0; t < T; ++t) {
        issue(t + R - 1, slot + R - 1 >= R ? slot - 1 : slot + R - 1);
        wait_vm<(R - 1) * C::kCopies>();
        const char* w = ring + slot * C::kStage;
        const int chunks = (S - (t * kWaves + wave) * 128) / 16;
        int ws = *reinterpret_cast<const int*>(w + C::kScales + 4 * lane) >> w_shift;
        int xs = 0;
        char* own = smem + kWaves * R * C::kStage + wave * C::kOwn;
        if constexpr (C::kFused) {
            for (int r = 0; r < min(M, kRows); ++r) {
                const Pack<TX, 4> v = *reinterpret_cast<const Pack<TX, 4>*>(w + C::kX + r * (int)(kMx4TileK * sizeof(TX)) + lane * (int)(4 * sizeof(TX)));
                const uint32_t s = mx4_scale(mx4_max_eight(mx4_max_bits<4>(v.v)));
                *reinterpret_cast<uint16_t*>(own + 256 * r + 2 * lane) = (uint16_t)mx4_codes<4>(v.v, s);
                if (lane % 8 == 0) own[256 * r + 128 + lane / 8 % 4 * 2 + lane / 32] = (char)s;
            }
            wave_lds_sync();
            xs = *reinterpret_cast<const uint16_t*>(own + 256 * min(l16, kRows - 1) + 128 + 2 * kg);
        } else {
            xs = *reinterpret_cast<const int*>(w + C::kScales + 256 + 4 * lane);
        }
        each(std::make_integer_sequence<int, 2>{}, [&](auto step) __attribute__((always_inline)) {
            constexpr int ks = decltype(step)::value;
            const i32x4_t wf = *reinterpret_cast<const i32x4_t*>(w + 128 * l16 + 16 * ((4 * ks + kg) ^ sw));
            i32x4_t xf;
            if constexpr (C::kFused) {
                xf = *reinterpret_cast<const i32x4_t*>(own + 256 * min(l16, kRows - 1) + 16 * (4 * ks + kg));
            } else {
                const int r = l16 % kRows;
                xf = *reinterpret_cast<const i32x4_t*>(w + C::kX + 128 * r + 16 * ((4 * ks + kg) ^ ((r >> 1) & 7)));
            }
            if (4 * ks + kg >= chunks) xf = i32x4_t{0, 0, 0, 0}, xs = ws = kOnes;  // (a lane's second block lies past its first)
            acc = mfma<ks, ks>(wf, xf, acc, ws, xs);
        });
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the stage is read, copies may overwrite it
        slot = slot + 1 == R ? 0 : slot + 1;
    }
    wait_vm<0>();
    __syncthreads();
    f32x4v_t* sums = reinterpret_cast<f32x4v_t*>(smem);
    sums[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave > 0 || l16 >= M) return;
    acc = sums[lane];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) acc += sums[i * 64 + lane];
    TO* out = y + (size_t)l16 * N + n0 + 4 * kg;
    Pack<TO, 4> o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o.v[e] = from_f32<TO>(acc[e]);
    if (N % 4 == 0) {
        if (n0 + 4 * kg < N) *reinterpret_cast<Pack<TO, 4>*>(out) = o;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n0 + 4 * kg + e < N) out[e] = o.v[e];
    }
}

// Up to 16 rows; of them quantized inside the product: one or two, and up to eight where a wave has few to quantize (one
// launch against two: 8 x 1000 x 2048 4.2 us against 5.5, 4 x 4096 x 4096 4.9 against 5.5; but 8 x 4096 x 4096 6.3
// against 5.9, 4 x 14336 x 4096 11.8 against 10.3: every block quantizes them).
constexpr int64_t kFewRows = 16;
bool fused_rows(int64_t M, int64_t N, int64_t K) {
    return M <= 2 || (N <= 16 * 512 && M * ((mx4_ktiles(K) + 7) / 8) <= 8);
}

struct Product {
    const uint8_t *xq, *xscales;
    int64_t M;
    const uint8_t *codes, *scales;
    int64_t N, K;
    hipStream_t stream;
};

template <typename C>
int64_t launch_blocks(int64_t M, int64_t N) {
    return ((N + C::BN - 1) / C::BN) * ((M + C::BM - 1) / C::BM);
}
template <typename C>
bool fits_grid(int64_t M, int64_t N) {
    return launch_blocks<C>(M, N) < ((int64_t)1 << 31) / (64 * C::NW);  // the grid's threads
}

template <typename C, typename TX, typename TO>
hipError_t launch_tiles(const Product& p, const TX* x, TO* y) {
    constexpr int kGroup = C::BM < 256 ? 1024 / C::BM : 4;  // row tiles walked together: about 1024 rows
    hipLaunchKernelGGL((w4a4_tile_kernel<TO, TX, C>), dim3((unsigned)launch_blocks<C>(p.M, p.N)), dim3(64 * C::NW),
                       C::kX ? 0 : fused_bytes<C>(p.K), p.stream, x, p.xscales, (int)p.M, p.codes, p.scales, (int)p.N, (int)(p.K / 2), y, (int)((p.N + C::BN - 1) / C::BN), kGroup);
    return hipGetLastError();
}

// Few rows x, in the format or as activations.  Eight waves a block where they leave each CU two blocks at the most, for
// the shorter chain of k-tiles (one row of 4096 x 14336 8.5 us against 10.1), else four, of which more blocks fit a CU
// (14336 x 4096 9.1 against 9.8).
template <typename TO, typename TX, int kRows>
hipError_t launch_rows(const Product& p, const TX* x, TO* y) {
    const int64_t blocks = (p.N + 15) / 16;
    auto run = [&](auto waves, auto once) {
        constexpr int kWaves = decltype(waves)::value;
        hipLaunchKernelGGL((w4a4_rows_kernel<TO, TX, kRows, kWaves, decltype(once)::value>), dim3((unsigned)blocks), dim3(64 * kWaves), 0,
                           p.stream, x, p.xscales, (int)p.M, p.codes, p.scales, (int)p.N, (int)(p.K / 2), y);
        return hipGetLastError();
    };
    if (blocks <= 512) return run(std::integral_constant<int, 8>{}, std::false_type{});
    const bool once = (double)p.N * (double)p.K / 2 >= kOnceBytes;
    return once ? run(std::integral_constant<int, 4>{}, std::true_type{}) : run(std::integral_constant<int, 4>{}, std::false_type{});
}

using T256x256 = Tiling<2, 4, 1, 8, 4, 2>;
using T128x256 = Tiling<2, 4, 1, 4, 4, 3>;
using T128x128 = Tiling<2, 4, 1, 4, 2, 4>;
using T64x128 = Tiling<2, 4, 1, 2, 2, 3>;
using T64x64 = Tiling<2, 2, 1, 2, 2, 4>;
using T32x64 = Tiling<2, 4, 1, 1, 1, 4>;
using T32x32 = Tiling<2, 2, 2, 1, 1, 4>;
// ... of which these quantize x themselves
using F32x64 = Tiling<2, 4, 1, 1, 1, 4, false>;
using F32x32 = Tiling<2, 2, 2, 1, 1, 4, false>;

// What a tiling costs.  A CU's first block takes `us_ktile` for each 256 of K and `us_first` besides, each further one
// `next_ktile` and `us_next`; `blocks` of them fit a CU.  The weights arrive at 5.6 TB/s, and neither hides all of the
// other; a stream of more blocks than run at once ends with some of the GPU idle.  Fitted to the tilings' times at 180
// shapes of 17 to 4096 rows, 64 to 30000 columns and K of 64 to 16384: the choice is on average 0.2% slower than the
// fastest tiling, 7% at most.  It ranks tilings and does not predict times.
struct Cost {
    double us_ktile, us_first, next_ktile, us_next;
    int blocks;
    double us(double tiles, int64_t K, double weight_bytes) const {
        const double waves = tiles / 256, up = std::ceil(waves), slots = 256.0 * blocks, ktiles = (double)mx4_ktiles(K);
        const double rounds = blocks == 1 ? up : waves <= 1 ? 1.0 : std::max(waves, 0.9 * up);
        const double work = ktiles * us_ktile + us_first + (rounds - 1) * (ktiles * next_ktile + us_next);
        const double tail = tiles > slots ? 1.0 + 0.2 * slots / tiles : 1.0;
        const double stream = weight_bytes / 5.6e6 * tail;
        return std::sqrt(work * work + stream * stream);
    }
};

template <typename F>
void each_tiling(F f) {
    f(0, T256x256{}, Cost{1.11, 5.1, 1.94, 7.4, 1});
    f(1, T128x256{}, Cost{0.68, 3.6, 1.41, 4.4, 2});
    f(2, T128x128{}, Cost{0.44, 2.9, 0.72, 3.3, 1});
    f(3, T64x128{}, Cost{0.35, 2.2, 0.42, 1.3, 1});
    f(4, T64x64{}, Cost{0.265, 2.1, 0.27, 0.93, 4});
    f(5, T32x64{}, Cost{0.243, 2.1, 0.216, 0.74, 1});
    f(6, T32x32{}, Cost{0.13, 2.4, 0.11, 1.06, 1});
}

int choose_tiling(int64_t M, int64_t N, int64_t K) {
    int choice = -1;
    double least = 0;
    each_tiling([&](int i, auto tiling, Cost cost) {
        using C = decltype(tiling);
        if (!fits_grid<C>(M, N)) return;
        const double us = cost.us((double)launch_blocks<C>(M, N), K, (double)N * (double)K * 17 / 32);
        if (choice < 0 || us < least) choice = i, least = us;
    });
    return choice;
}

template <typename TO>
hipError_t launch_product(const Product& p, TO* y) {
    if (p.M <= 8) return launch_rows<TO, uint8_t, 8>(p, p.xq, y);
    if (p.M <= kFewRows) return launch_rows<TO, uint8_t, 16>(p, p.xq, y);
    const int choice = choose_tiling(p.M, p.N, p.K);
    hipError_t e = hipErrorInvalidConfiguration;
    each_tiling([&](int i, auto tiling, Cost) {
        if (i == choice) e = launch_tiles<decltype(tiling)>(p, p.xq, y);
    });
    return e;
}

// Rows quantized by every block for itself, in the tiling that the product takes and so to the same bits: where a
// wave has few units of it and the blocks are few (one launch against two: 37 x 1001 x 512 4.9 us against 6.4, 100 x 4000 x
// 512 5.1 against 6.4, 20 x 5000 x 1024 5.3 against 6.2; but 37 x 1001 x 2080, 17 units a wave, 11.2 against 7.5, and 300 x
// 2000 x 512, 16 units, 8.0 against 6.4).
constexpr int64_t kFusedBlocks = 512;
template <typename T>
bool launch_fused(const Product& p, const T* x, T* y, hipError_t& e) {
    const int choice = choose_tiling(p.M, p.N, p.K);
    bool done = false;
    auto attempt = [&](int i, auto tiling) {
        using C = decltype(tiling);
        const int64_t units = (std::min<int64_t>(p.M, C::BM) + C::NW - 1) / C::NW * ((p.K + 511) / 512);  // of a wave
        if (i != choice || units > 2 * kFusedUnits || launch_blocks<C>(p.M, p.N) > kFusedBlocks) return;
        e = launch_tiles<C>(p, x, y), done = true;  // (K is at most 1024 here: 17 KB of LDS behind the ring)
    };
    attempt(5, F32x64{});
    attempt(6, F32x32{});
    return done;
}

}  // namespace

bool w4a4_fits_grid(int64_t M, int64_t N) { return fits_grid<T256x256>(M, N); }

hipError_t launch_gemm_w4a4(int dtype, const uint8_t* xq, const uint8_t* xscales, int64_t M, const uint8_t* codes,
                            const uint8_t* scales, int64_t N, int64_t K, void* y, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using TO = decltype(t);
        return launch_product<TO>(Product{xq, xscales, M, codes, scales, N, K, stream}, static_cast<TO*>(y));
    });
}

hipError_t launch_matmul_w4a4(int dtype, const void* x, int64_t M, const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t K,
                              void* y, uint8_t* xq, uint8_t* xscales, hipStream_t stream) {
    return with_act_type(dtype, [&](auto t) {
        using T = decltype(t);
        const Product p{xq, xscales, M, codes, scales, N, K, stream};
        if (M <= 2) return launch_rows<T, T, 2>(p, static_cast<const T*>(x), static_cast<T*>(y));
        if (fused_rows(M, N, K)) {
            const T* xt = static_cast<const T*>(x);
            return M <= 4 ? launch_rows<T, T, 4>(p, xt, static_cast<T*>(y)) : launch_rows<T, T, 8>(p, xt, static_cast<T*>(y));
        }
        hipError_t e = hipSuccess;
        if (M > kFewRows && launch_fused(p, static_cast<const T*>(x), static_cast<T*>(y), e)) return e;
        if (e = launch_quant_mx4(dtype, x, M, K, xq, xscales, stream); e != hipSuccess) return e;
        return launch_product<T>(p, static_cast<T*>(y));
    });
}

}  // namespace w4a16

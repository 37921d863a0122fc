// ops_adapters.hpp -- low-rank adapters of many requests beside a shared
// projection:  y_t += s_i B_i (A_i x_t)  with i = ids[t], A_i of rank x cols,
// B_i of rows x rank.
//
// Two launches on the matrix cores, both over tiles of 16 (few tokens) or 64
// consecutive tokens and, within a tile, one adapter after the other: the
// tokens of a prompt lie side by side and share their adapter, the tokens of
// a batch of single requests differ and take one turn each, spread over the
// grid's z.
//   k_adapters_down  u_t = s_i A_i x_t (fp32), the columns split over the
//                    waves of a block and, for few tokens, over blocks
//   k_adapters_up    y_t += B_i u_t
// What bounds it: x read once, y read and written once.  u stays in 32 bits:
// it enters the matrix cores as a sum of 16-bit numbers, three of BF16 (8
// significant bits each), or two of FP16 (11 each) after a scaling by a power
// of two per token that brings its largest value to 2^14..2^15; products with
// the 16-bit B are exact and summed in fp32, so y is rounded once, to its own
// type.
//
// MFMA 16x16x32 (lane l = 16 g + i): A operand row i, k = 8 g .. 8 g + 7;
// B operand column i, the same k; D column i, rows 4 g .. 4 g + 3.  Here A is
// the adapter (a row of A_i or B_i) and B's columns are 16 tokens.
#pragma once

#include "ops_common.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kAdapterMaxRank = 256;

struct AdapterArgs {
    const uint16_t *x;
    uint64_t x_stride;
    void *y;
    uint64_t y_stride;
    const uint16_t *a, *b;  // n x rank x cols, n x rows x rank
    const int64_t *ids;
    const float *scales;    // n, or null: 1
    uint64_t m;
    uint32_t n, rank, cols, rows;
    float *u;               // splits x m x padded rank
    uint32_t rank_pad, splits, steps;  // steps: of 32 columns, per split
    uint32_t row_block;                // rows of y per block of k_adapters_up
    uint32_t *err;
};

// The adapters of a tile of up to 64 tokens, one by one: lane l looks after
// token tile + l.
struct TileIds {
    int32_t id;        // the lane's token's adapter, -1: none
    uint64_t pending;  // tokens whose adapter was not taken yet

    __device__ TileIds(const AdapterArgs &g, uint64_t tile, uint32_t tokens)
    {
        const uint32_t lane = threadIdx.x & 63;
        id = -1;
        if (lane < tokens && tile + lane < g.m) {
            const int64_t v = g.ids[tile + lane];
            if (v >= 0 && v < (int64_t)g.n) id = (int32_t)v;
            else if (v != -1 && threadIdx.x < 64) report(g.err, WC_EF_BAD_INDEX);
        }
        pending = __ballot(id >= 0);
    }
    // the next adapter and its tokens; false when there is none
    __device__ bool next(uint32_t &adapter, uint64_t &mask)
    {
        if (!pending) return false;
        adapter = (uint32_t)__builtin_amdgcn_readlane(id, __builtin_ctzll(pending));
        mask = __ballot(id == (int32_t)adapter);
        pending &= ~mask;
        return true;
    }
};

// u = s A x.  Grid: x = tiles x splits, y = blocks of 16 RT ranks, z = turns.
template <int T, int TT, int RT>
__global__ __launch_bounds__(256) void k_adapters_down(AdapterArgs g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    __shared__ f32x4 part[4][RT * TT][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint64_t tile = (uint64_t)(blockIdx.x / g.splits) * (16 * TT);
    const uint32_t split = blockIdx.x % g.splits;
    const uint32_t r0 = blockIdx.y * (16 * RT);
    const uint32_t s0 = split * g.steps, s1 = min((g.cols + 31) / 32, s0 + g.steps), full = min(g.cols / 32, s1);
    TileIds ids(g, tile, 16 * TT);
    const uint16_t *xr[TT];
#pragma unroll
    for (int t = 0; t < TT; t++) xr[t] = g.x + min(tile + 16 * t + i, g.m - 1) * g.x_stride;
    uint32_t adapter, turn = 0;
    uint64_t mask;
    while (ids.next(adapter, mask)) {
        if (turn++ % gridDim.z != blockIdx.z) continue;
        const uint16_t *ar[RT];
#pragma unroll
        for (int r = 0; r < RT; r++)
            ar[r] = g.a + ((uint64_t)adapter * g.rank + min(r0 + 16 * r + i, g.rank - 1)) * g.cols;
        f32x4 acc[RT][TT];
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int t = 0; t < TT; t++) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto step = [&](uint32_t st, bool in) {  // 32 columns; a lane's 8 are all there or all not
            X8 av[RT], xv[TT];
            const uint32_t k = 32 * st + 8 * gr;
#pragma unroll
            for (int r = 0; r < RT; r++)
                av[r] = __builtin_bit_cast(X8, in ? load16<16>(ar[r] + k) : u32x4{0u, 0u, 0u, 0u});
#pragma unroll
            for (int t = 0; t < TT; t++)
                xv[t] = __builtin_bit_cast(X8, in ? load16<16>(xr[t] + k) : u32x4{0u, 0u, 0u, 0u});
#pragma unroll
            for (int r = 0; r < RT; r++)
#pragma unroll
                for (int t = 0; t < TT; t++) acc[r][t] = Ty::mfma(av[r], xv[t], acc[r][t]);
        };
        uint32_t st = s0 + wave;
#pragma unroll 4
        for (; st < full; st += 4) step(st, true);
        if (st < s1) step(st, 32 * st + 8 * gr < g.cols);  // the columns' end is a multiple of 8, not of 32
#pragma unroll
        for (int r = 0; r < RT; r++)
#pragma unroll
            for (int t = 0; t < TT; t++) part[wave][r * TT + t][lane] = acc[r][t];
        __syncthreads();
        const float s = g.scales ? g.scales[adapter] : 1.f;
#pragma unroll
        for (int q = 0; q < (RT * TT + 3) / 4; q++) {
            const uint32_t c = 4 * q + wave;
            if (c < RT * TT) {
                const uint32_t t = c % TT, row = r0 + 16 * (c / TT) + 4 * gr;
                f32x4 v = (part[0][c][lane] + part[1][c][lane]) + (part[2][c][lane] + part[3][c][lane]);
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = row + e < g.rank ? s * v[e] : 0.f;
                if (((mask >> (16 * t + i)) & 1) && row < g.rank_pad)
                    *reinterpret_cast<f32x4 *>(g.u + ((uint64_t)split * g.m + tile + 16 * t + i) * g.rank_pad + row) = v;
            }
        }
        __syncthreads();
    }
}

// A 16-bit operand's 32-bit numbers as sums of 16-bit ones.
template <int T>
struct Terms;
template <>
struct Terms<WC_T_BF16> {
    static constexpr int kCount = 3;
    __device__ static void split(const float *f, bf16x8 *out)
    {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const __bf16 a = (__bf16)f[e];
            const float r1 = fabsf((float)a) < kInf ? f[e] - (float)a : 0.f;  // an infinity is its own first term
            const __bf16 b = (__bf16)r1;
            out[0][e] = a;
            out[1][e] = b;
            out[2][e] = (__bf16)(r1 - (float)b);
        }
    }
};
template <>
struct Terms<WC_T_FP16> {
    static constexpr int kCount = 2;
    __device__ static void split(const float *f, f16x8 *out)
    {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const _Float16 a = (_Float16)f[e];
            out[0][e] = a;
            out[1][e] = (_Float16)(fabsf((float)a) < kInf ? f[e] - (float)a : 0.f);
        }
    }
};

// y += B u.  Grid: x = tiles x row blocks, z = turns.  A wave takes 64 rows
// at a time as four tiles whose rows are dealt out so that a lane ends with
// 16 consecutive elements of its token's y: row i of tile p is row
// 16 (i / 4) + 4 p + i % 4 of the 64.
template <int T, int YT, int TT, int KS>
__global__ __launch_bounds__(256) void k_adapters_up(AdapterArgs g)
{
    using Ty = Type<T>;
    using Y = Type<YT>;
    using YE = typename Y::elem;
    using X8 = typename Ty::x8;
    constexpr int kTerms = Terms<T>::kCount, kYVecs = 16 / Y::kPer16;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t row_blocks = (g.rows + g.row_block - 1) / g.row_block;
    const uint64_t tile = (uint64_t)(blockIdx.x / row_blocks) * (16 * TT);
    const uint32_t n0 = (blockIdx.x % row_blocks) * g.row_block, n1 = min(g.rows, n0 + g.row_block);
    TileIds ids(g, tile, 16 * TT);
    uint32_t adapter, turn = 0;
    uint64_t mask;
    while (ids.next(adapter, mask)) {
        if (turn++ % gridDim.z != blockIdx.z) continue;
        X8 u[TT][KS][kTerms];
        float unscale[TT];
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const uint64_t token = min(tile + 16 * t + i, g.m - 1);
            float f[KS][8];
            float most = 0.f;
#pragma unroll
            for (int s = 0; s < KS; s++) {
                const uint32_t k = 32 * s + 8 * gr;
#pragma unroll
                for (int e = 0; e < 8; e++) f[s][e] = 0.f;
                if (k < g.rank_pad && ((mask >> (16 * t + i)) & 1)) {
                    for (uint32_t sp = 0; sp < g.splits; sp++) {
                        const float *p = g.u + ((uint64_t)sp * g.m + token) * g.rank_pad + k;
                        const f32x4 v = *reinterpret_cast<const f32x4 *>(p), w = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            f[s][e] += v[e];
                            f[s][4 + e] += w[e];
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; e++) most = fmaxf(most, fabsf(f[s][e]));
            }
            unscale[t] = 1.f;
            if constexpr (T == WC_T_FP16) {
                most = fmaxf(most, __shfl_xor(most, 16, 64));
                most = fmaxf(most, __shfl_xor(most, 32, 64));
                if (most > 0.f && most < kInf) {
                    const int ex = max(-100, min(100, 15 - __builtin_amdgcn_frexp_expf(most)));
                    unscale[t] = __builtin_ldexpf(1.f, -ex);
#pragma unroll
                    for (int s = 0; s < KS; s++)
#pragma unroll
                        for (int e = 0; e < 8; e++) f[s][e] = __builtin_ldexpf(f[s][e], ex);
                }
            }
#pragma unroll
            for (int s = 0; s < KS; s++) Terms<T>::split(f[s], u[t][s]);
        }
        const uint16_t *b = g.b + (uint64_t)adapter * g.rows * g.rank;
        for (uint32_t nb = n0 + 64 * wave; nb < n1; nb += 256) {
            X8 bv[4][KS];
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const uint32_t row = min(nb + 16 * (i >> 2) + 4 * p + (i & 3), g.rows - 1);
                const uint16_t *br = b + (uint64_t)row * g.rank;
#pragma unroll
                for (int s = 0; s < KS; s++) {
                    const uint32_t k = 32 * s + 8 * gr;
                    u32x4 v{0u, 0u, 0u, 0u};
                    if (k + 8 <= g.rank) {
                        v = load16<2>(br + k);
                    } else {
                        for (uint32_t e = 0; e < 8; e++)
                            if (k + e < g.rank) v[e >> 1] |= (uint32_t)br[k + e] << (16 * (e & 1));
                    }
                    bv[p][s] = __builtin_bit_cast(X8, v);
                }
            }
            const uint32_t n = nb + 16 * gr;
#pragma unroll
            for (int t = 0; t < TT; t++) {
                if (!((mask >> (16 * t)) & 0xFFFFu)) continue;
                const bool mine = (mask >> (16 * t + i)) & 1;
                YE *yp = static_cast<YE *>(g.y) + (tile + 16 * t + i) * g.y_stride + n;
                float f[16];
                const bool whole = mine && n + 16 <= n1;
                if (whole) {
#pragma unroll
                    for (int v = 0; v < kYVecs; v++)
                        Y::unpack(load16<Y::kBytes>(yp + v * Y::kPer16), f + v * Y::kPer16);
                }
                f32x4 acc[4];
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    acc[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < KS; s++)
#pragma unroll
                        for (int c = kTerms - 1; c >= 0; c--) acc[p] = Ty::mfma(bv[p][s], u[t][s][c], acc[p]);
                }
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 16; e++) f[e] += acc[e >> 2][e & 3] * unscale[t];
#pragma unroll
                    for (int v = 0; v < kYVecs; v++)
                        store16<Y::kBytes>(yp + v * Y::kPer16, Y::pack(f + v * Y::kPer16));
                } else if (mine) {
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        if (n + e < n1) yp[e] = Y::from_f32(Y::to_f32(yp[e]) + acc[e >> 2][e & 3] * unscale[t]);
                }
            }
        }
    }
}

}  // namespace ops
}  // namespace wc

// ops_adapters.hpp -- low-rank adapters of many requests beside a shared
// projection:  y_t += s_i B_i (A_i x_t)  with i = ids[t], A_i of rank x cols,
// B_i of rows x rank.
//
// On the matrix cores, over tiles of 16 (few tokens) or 128 consecutive tokens
// and, within a tile, one adapter after the other: the tokens of a prompt lie
// side by side and share their adapter, the tokens of a batch of single
// requests differ and take one turn each, spread over the grid.
//   k_adapters_few    few tokens: both products in one launch
//   k_adapters_down   A_i x_t in parts along the columns; for many tokens
//                     k_adapters_down_many
//   k_adapters_terms  u_t = s_i times the sum of the parts, as terms (below)
//   k_adapters_up     y_t += B_i u_t, u from the parts up to rank 64; for many
//                     tokens k_adapters_up_many
// What bounds it: x read once, y read and written once.  u stays in 32 bits:
// it enters the matrix cores as a sum of 16-bit numbers (Terms), for FP16
// after a scaling by a power of two per token that brings its largest value
// to 2^14..2^15; products with the 16-bit B are exact and summed in fp32, so y
// is rounded once, to its own type.  (Two BF16 terms, 16 bits, for a 16-bit y
// would save 3% of 8192 tokens at rank 64 and 7% of 2048 at rank 256.)
//
// MFMA 16x16x32 (lane l = 16 g + i): A operand row i, k = 8 g .. 8 g + 7;
// B operand column i, the same k; D column i, rows 4 g .. 4 g + 3.  Here A is
// the adapter (a row of A_i or B_i) and B's columns are 16 tokens.
#pragma once

#include "ops_common.hpp"
#include "wc_common.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kAdapterMaxRank = 256;
constexpr int kDownWaves = 8;

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
    float *part;            // splits x m x rank_pad: A x in parts
    uint16_t *u;            // terms x m x rank_pad: k_adapters_terms' result
    float *unscale;         // m x rank blocks: what the products of the terms are multiplied by
    uint32_t rank_pad;      // the rank rounded up to 32
    uint32_t splits, split_cols;
    uint32_t row_block;     // rows of y per block of k_adapters_up and k_adapters_few
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
        take(adapter, mask);
        return true;
    }
    // the tokens of an adapter
    __device__ void take(uint32_t adapter, uint64_t &mask)
    {
        mask = __ballot(id == (int32_t)adapter);
        pending &= ~mask;
    }
};

// Eight values of u of one token, from rank k, as terms.
template <int T>
__device__ __forceinline__ void put_terms(const AdapterArgs &g, uint64_t token, uint32_t k, const float *f)
{
    constexpr int kTerms = Terms<T>::kCount;
    typename Type<T>::x8 u[kTerms];
    Terms<T>::split(f, u);
#pragma unroll
    for (int c = 0; c < kTerms; c++)
        *reinterpret_cast<u32x4 *>(g.u + (c * g.m + token) * g.rank_pad + k) = __builtin_bit_cast(u32x4, u[c]);
}

// A x of tiles of 16 tokens, without the scales, in parts along the columns.
// Grid: x = tiles x splits, y = blocks of 64 ranks (RT tiles of 16), z = turns.
// The columns go round the waves of the block, four steps of 32 (of which a
// lane has 8: all there, or none) on their way at once.  What bounds it is the
// latency of its loads, so that a block takes no more columns than are on
// their way at once where there are compute units for it: 61 tokens of 32
// adapters of rank 16, 4096 columns, take 5.4 us in four parts, 12.2 in one
// with every token's row read for every adapter.
template <int T, int RT>
__global__ __launch_bounds__(64 * kDownWaves, 2) void k_adapters_down(AdapterArgs g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    constexpr int Q = 4, W = kDownWaves;
    __shared__ f32x4 part[W][RT][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint64_t tile = (uint64_t)(blockIdx.x / g.splits) * 16;
    const uint32_t split = blockIdx.x % g.splits, c0 = split * g.split_cols, c1 = min(g.cols, c0 + g.split_cols);
    const uint32_t r0 = blockIdx.y * 64, steps = (c1 - c0 + 31) / 32;
    TileIds ids(g, tile, 16);
    uint32_t adapter, turn = 0;
    uint64_t mask;
    while (ids.next(adapter, mask)) {
        if (turn++ % gridDim.z != blockIdx.z) continue;
        // lanes of other tokens repeat the first one's loads
        const uint16_t *xr = g.x + (tile + ((mask >> i) & 1 ? i : (uint32_t)__builtin_ctzll(mask))) * g.x_stride;
        const uint16_t *ar[RT];
        f32x4 acc[RT];
#pragma unroll
        for (int r = 0; r < RT; r++) {
            ar[r] = g.a + ((uint64_t)adapter * g.rank + min(r0 + 16 * r + i, g.rank - 1)) * g.cols;
            acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        for (uint32_t j = 0; wave_step<W>(wave, j) < steps; j += Q) {
            X8 av[Q][RT], xv[Q];
#pragma unroll
            for (int q = 0; q < Q; q++) {
                const uint32_t c = c0 + 32 * wave_step<W>(wave, j + q) + 8 * gr, k = min(c, g.cols - 8);
                const bool in = c < c1;
                xv[q] = __builtin_bit_cast(X8, only(in, load16<16>(xr + k)));
#pragma unroll
                for (int r = 0; r < RT; r++) av[q][r] = __builtin_bit_cast(X8, only(in, load16<16>(ar[r] + k)));
            }
#pragma unroll
            for (int q = 0; q < Q; q++)
#pragma unroll
                for (int r = 0; r < RT; r++) acc[r] = Ty::mfma(av[q][r], xv[q], acc[r]);
        }
#pragma unroll
        for (int r = 0; r < RT; r++) part[wave][r][lane] = acc[r];
        __syncthreads();
        for (uint32_t q = threadIdx.x; q < 64 * RT; q += 64 * W) {  // four ranks of a token
            const uint32_t c = q >> 6, l = q & 63, t = l & 15, r = r0 + 16 * c + 4 * (l >> 4);
            f32x4 v = part[0][c][l];
#pragma unroll
            for (int w = 1; w < W; w++) v += part[w][c][l];
            if (((mask >> t) & 1) && r < g.rank_pad)
                *reinterpret_cast<f32x4 *>(g.part + ((uint64_t)split * g.m + tile + t) * g.rank_pad + r) = v;
        }
        __syncthreads();
    }
}

// A x of many tokens, without the scales, in parts along the columns.  Grid:
// x = tiles of 128 tokens x splits, y = blocks of 64 ranks (RT tiles of 16),
// z = turns.
// The four waves of a block take 32 tokens each; their rows and those of A
// are read in whole lines and come to operand order in LDS (Strip), A once
// for the block.  With 32 tokens a block and all columns, A passed through
// the L1 cache twice as often as x, and that took 75 us where this takes 37
// (8192 tokens, 4096 columns, rank 64).  The next columns are on their way
// while these are multiplied.
template <int T, int RT>
__global__ __launch_bounds__(256) void k_adapters_down_many(AdapterArgs g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    __shared__ Strip sa[RT], sx[4][2];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t hi = lane >> 5, lo = lane & 31;
    const uint32_t block = xcd_block(), split = block % g.splits, r0 = blockIdx.y * 64;
    const uint64_t tile = (uint64_t)(block / g.splits) * 128, first = tile + 32 * wave;
    const uint32_t c0 = split * g.split_cols, c1 = min(g.cols, c0 + g.split_cols);
    TileIds low(g, tile, 64), high(g, tile + 64, 64);
    const uint16_t *xr[2][8];  // the rows of the lane's loads
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int u = 0; u < 8; u++) xr[t][u] = g.x + min(first + 16 * t + 2 * u + hi, g.m - 1) * g.x_stride;
    uint64_t mlow, mhigh;
    uint32_t adapter, turn = 0;
    while (low.pending | high.pending) {
        if (low.next(adapter, mlow)) {
            high.take(adapter, mhigh);
        } else {
            mlow = 0;
            high.next(adapter, mhigh);
        }
        if (turn++ % gridDim.z != blockIdx.z) continue;
        const uint32_t mask = (uint32_t)((wave & 2 ? mhigh : mlow) >> (32 * (wave & 1)));  // the wave's tokens
        const uint16_t *a = g.a + (uint64_t)adapter * g.rank * g.cols;
        f32x4 acc[RT][2];
#pragma unroll
        for (int r = 0; r < RT; r++) acc[r][0] = acc[r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        u32x4 xv[2][8], av[2 * RT];
        auto fetch = [&](uint32_t c) {
            const uint32_t k = min(c + 8 * lo, g.cols - 8);
            if (mask) {
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int u = 0; u < 8; u++) xv[t][u] = read16<16, true>(xr[t][u] + k);
            }
#pragma unroll
            for (int u = 0; u < 2 * RT; u++)  // a quarter of A's rows
                av[u] = load16<16>(a + (uint64_t)min(r0 + 4 * RT * wave + 2 * u + hi, g.rank - 1) * g.cols + k);
        };
        if (c0 < c1) fetch(c0);
        for (uint32_t c = c0; c < c1; c += kStripCols) {
            const bool there = c + 8 * lo < c1;
            __syncthreads();  // the last columns' readers are done
            if (mask) {
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int u = 0; u < 8; u++) sx[wave][t].q[(2 * u + hi) * kStripPitch + lo] = only(there, xv[t][u]);
            }
#pragma unroll
            for (int u = 0; u < 2 * RT; u++) {
                const uint32_t r = 4 * RT * wave + 2 * u + hi;
                sa[r >> 4].q[(r & 15) * kStripPitch + lo] = only(there, av[u]);
            }
            __syncthreads();
            if (c + kStripCols < c1) fetch(c + kStripCols);
            if (!mask) continue;
#pragma unroll
            for (int s = 0; s < (int)kStripCols / 32; s++) {
                X8 xo[2];
#pragma unroll
                for (int t = 0; t < 2; t++) xo[t] = __builtin_bit_cast(X8, sx[wave][t].q[i * kStripPitch + 4 * s + gr]);
#pragma unroll
                for (int r = 0; r < RT; r++) {
                    const X8 ao = __builtin_bit_cast(X8, sa[r].q[i * kStripPitch + 4 * s + gr]);
#pragma unroll
                    for (int t = 0; t < 2; t++) acc[r][t] = Ty::mfma(ao, xo[t], acc[r][t]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; t++) {
            if (!((mask >> (16 * t + i)) & 1)) continue;
            float *p = g.part + ((uint64_t)split * g.m + first + 16 * t + i) * g.rank_pad + r0 + 4 * gr;
#pragma unroll
            for (int r = 0; r < RT; r++)
                if (r0 + 16 * r < g.rank_pad) *reinterpret_cast<f32x4 *>(p + 16 * r) = acc[r][t];
        }
    }
}

// u from its parts: eight lanes for the 64 ranks of a block of one token.
template <int T>
__global__ __launch_bounds__(256) void k_adapters_terms(AdapterArgs g)
{
    const uint32_t blocks = (g.rank_pad + 63) / 64;
    const uint64_t q = (uint64_t)blockIdx.x * 32 + threadIdx.x / 8, token = q / blocks;
    const uint32_t rb = (uint32_t)(q % blocks), k = 64 * rb + 8 * (threadIdx.x % 8);
    if (token >= g.m) return;
    const int64_t id = g.ids[token];
    if (id < 0 || id >= (int64_t)g.n) return;  // the same for a token's lanes
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] = 0.f;
    if (k < g.rank_pad) {
        const float *p = g.part + token * g.rank_pad + k;
        for (uint32_t s = 0; s < g.splits; s++, p += g.m * g.rank_pad) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(p), w = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                f[e] += v[e];
                f[4 + e] += w[e];
            }
        }
    }
    const float scale = g.scales ? g.scales[id] : 1.f;
    float most = 0.f, unscale;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        f[e] = k + e < g.rank ? scale * f[e] : 0.f;
        most = fmaxf(most, fabsf(f[e]));
    }
    if constexpr (T == WC_T_FP16)
        for (int o = 1; o < 8; o *= 2) most = fmaxf(most, __shfl_xor(most, o, 8));
    const float sc = term_scale<T>(most, unscale);
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] *= sc;
    if (k < g.rank_pad) put_terms<T>(g, token, k, f);
    if (threadIdx.x % 8 == 0) g.unscale[token * blocks + rb] = unscale;
}

// The same within a wave: u of one token (32 KS values, those of the lane; the
// lanes of a token are 16 apart) as terms.
template <int T, int KS, int C>
__device__ __forceinline__ float adapter_terms(float (&f)[KS][8], typename Type<T>::x8 (&u)[KS][C])
{
    float most = 0.f, unscale;
    if constexpr (T == WC_T_FP16) {
#pragma unroll
        for (int s = 0; s < KS; s++)
#pragma unroll
            for (int e = 0; e < 8; e++) most = fmaxf(most, fabsf(f[s][e]));
        most = fmaxf(most, __shfl_xor(most, 16, 64));
        most = fmaxf(most, __shfl_xor(most, 32, 64));
    }
    const float sc = term_scale<T>(most, unscale);
#pragma unroll
    for (int s = 0; s < KS; s++) {
        if constexpr (T == WC_T_FP16)
#pragma unroll
            for (int e = 0; e < 8; e++) f[s][e] *= sc;
        Terms<T>::split(f[s], u[s]);
    }
    return unscale;
}

// 64 rows of B from nb as four operand tiles whose rows are dealt out so that
// the four lanes of a token hold 64 bytes of its y side by side, 16 each: for
// a 32-bit y, row i of tile p is row 16 p + i of the 64; for a 16-bit y, row
// 32 (p / 2) + 8 (i / 4) + 4 (p % 2) + i % 4, and two tiles make 16 bytes.
template <int YT>
__device__ __forceinline__ uint32_t adapter_row(int p, uint32_t i)
{
    if constexpr (Type<YT>::kPer16 == 4) return 16 * p + i;
    else return 32 * (p >> 1) + 8 * (i >> 2) + 4 * (p & 1) + (i & 3);
}

// Eight elements of B from `at`, as far as B goes and at most `have`.
__device__ __noinline__ u32x4 b_end(const uint16_t *b, uint64_t at, uint64_t total, uint32_t have)
{
    u32x4 w{0u, 0u, 0u, 0u};
#pragma unroll
    for (uint32_t e = 0; e < 8; e++)
        if (e < have && at + e < total) w[e >> 1] |= (uint32_t)b[at + e] << (16 * (e & 1));
    return w;
}

// The rows of B of one adapter as operands.  A lane reads 16 bytes whatever
// the rank, so that all loads of a wave are on their way at once, and clears
// what is past the rank (it belongs to the rows behind); only where that
// would run past the end of B are elements read one by one.
template <int T, int YT, int KS>
struct BRows {
    const uint16_t *b;
    uint64_t left;      // elements from b to the end of B
    uint32_t keep[KS][4];
    uint32_t off[KS];   // the lane's first rank, 0 where it is past the rank

    __device__ __forceinline__ BRows(const AdapterArgs &g, uint32_t adapter, uint32_t k0)
    {
        b = g.b + (uint64_t)adapter * g.rows * g.rank;
        left = (uint64_t)(g.n - adapter) * g.rows * g.rank;
        const uint32_t gr = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int s = 0; s < KS; s++) {
            const uint32_t k = k0 + 32 * s + 8 * gr, have = k < g.rank ? g.rank - k : 0u;
            off[s] = have ? k : 0u;
#pragma unroll
            for (uint32_t e = 0; e < 4; e++) keep[s][e] = 2 * e + 1 < have ? ~0u : 2 * e < have ? 0xFFFFu : 0u;
        }
    }
    // tile p of the 64 rows from nb
    __device__ __forceinline__ void load(const AdapterArgs &g, uint32_t nb, int p, u32x4 (&v)[KS]) const
    {
        const bool end = left < (uint64_t)(min(nb + 64, g.rows) - 1) * g.rank + g.rank + 8;  // the same in all lanes
        const uint32_t row = min(nb + adapter_row<YT>(p, threadIdx.x & 15), g.rows - 1) * g.rank;  // below 2^31
#pragma unroll
        for (int s = 0; s < KS; s++) v[s] = end ? b_end(b, row + off[s], left, 8) : load16<2>(b + (row + off[s]));
    }
    __device__ __forceinline__ u32x4 kept(u32x4 v, int s) const
    {
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] &= keep[s][e];
        return v;
    }
    __device__ __forceinline__ void load(const AdapterArgs &g, uint32_t nb, typename Type<T>::x8 (&bv)[4][KS]) const
    {
        u32x4 v[4][KS];
#pragma unroll
        for (int p = 0; p < 4; p++) load(g, nb, p, v[p]);
#pragma unroll
        for (int p = 0; p < 4; p++)
#pragma unroll
            for (int s = 0; s < KS; s++) bv[p][s] = __builtin_bit_cast(typename Type<T>::x8, kept(v[p][s], s));
    }
};

// The lane's sixteen elements of 64 of a row of y from column n0: vectors of
// 16 bytes, 64 bytes apart.
template <int YT>
struct YRow {
    using Y = Type<YT>;
    using E = typename Y::elem;
    static constexpr int kPer = Y::kPer16, kVecs = 16 / kPer;
    u32x4 v[kVecs];
    __device__ __forceinline__ static uint32_t column(int q, uint32_t gr) { return (4 * q + gr) * kPer; }
    __device__ __forceinline__ void load(const E *p, uint32_t gr)
    {
#pragma unroll
        for (int q = 0; q < kVecs; q++) v[q] = load16<Y::kBytes>(p + column(q, gr));
    }
    __device__ __forceinline__ void add(E *p, uint32_t gr, const f32x4 (&acc)[4], float scale) const
    {
#pragma unroll
        for (int q = 0; q < kVecs; q++) {
            float f[kPer];
            Y::unpack(v[q], f);
#pragma unroll
            for (int e = 0; e < kPer; e++) f[e] += acc[q * kPer / 4 + e / 4][e & 3] * scale;
            store16<Y::kBytes>(p + column(q, gr), Y::pack(f));
        }
    }
};

// The same where the row ends within the 64, after `count`.
template <int YT>
__device__ __noinline__ void y_add_some(typename Type<YT>::elem *p, uint32_t gr, uint32_t count, f32x4 a0, f32x4 a1,
                                        f32x4 a2, f32x4 a3, float scale)
{
    using Y = Type<YT>;
    const f32x4 acc[4] = {a0, a1, a2, a3};
#pragma unroll
    for (int q = 0; q < YRow<YT>::kVecs; q++)
#pragma unroll
        for (int e = 0; e < Y::kPer16; e++) {
            const uint32_t n = YRow<YT>::column(q, gr) + e;
            if (n < count) p[n] = Y::from_f32(Y::to_f32(p[n]) + acc[q * Y::kPer16 / 4 + e / 4][e & 3] * scale);
        }
}

// y += B u.  Grid: x = tiles x row blocks, z = turns.  A wave takes 64 rows
// of B at a time; u, the sum of its parts, stays in its registers, or, with
// kBlocks blocks of 64 ranks (each with its own scaling), is read again for
// every 64 rows, as terms.  54 tokens of 32 adapters of rank 16, 14336 rows,
// FP32: 11.5 us (2.2 TB/s of B and y).  What bounds it is each wave's chain of
// waits (ids, then u, B and y at once, then the stores) over the waves that
// fit: 256 or 1024 rows a block took 15.5 and 12.3 us, and loading the next
// rows ahead costs registers, hence waves (16.3 us).
template <int T, int YT, int KS, bool kBlocks>
__global__ __launch_bounds__(256, KS == 1 ? 4 : 2) void k_adapters_up(AdapterArgs g)
{
    using Ty = Type<T>;
    using YE = typename Type<YT>::elem;
    using X8 = typename Ty::x8;
    constexpr int kTerms = Terms<T>::kCount;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t row_blocks = (g.rows + g.row_block - 1) / g.row_block, rank_blocks = kBlocks ? (g.rank_pad + 63) / 64 : 1;
    const uint64_t tile = (uint64_t)(blockIdx.x / row_blocks) * 16;
    const uint32_t n0 = (blockIdx.x % row_blocks) * g.row_block, n1 = min(g.rows, n0 + g.row_block);
    TileIds ids(g, tile, 16);
    uint32_t adapter, turn = 0;
    uint64_t mask;
    while (ids.next(adapter, mask)) {
        if (turn++ % gridDim.z != blockIdx.z) continue;
        const bool mine = (mask >> i) & 1;
        // lanes of other tokens repeat the first one's loads
        const uint64_t token = tile + (mine ? i : (uint32_t)__builtin_ctzll(mask));
        YE *const yr = static_cast<YE *>(g.y) + token * g.y_stride;
        const BRows<T, YT, KS> rows(g, adapter, 0);
        X8 bv[4][KS], u[KS][kTerms];
        YRow<YT> y;
        uint32_t nb = n0 + 64 * wave;
        auto fetch = [&]() {
            if (nb + 64 <= n1) y.load(yr + nb, gr);
            rows.load(g, nb, bv);
        };
        auto fetch_terms = [&](uint32_t rb) {
#pragma unroll
            for (int s = 0; s < KS; s++)
#pragma unroll
                for (int c = 0; c < kTerms; c++) {
                    const uint32_t k = min(64 * rb + 32 * s, g.rank_pad - 32) + 8 * gr;  // past it B is zero
                    u[s][c] = __builtin_bit_cast(X8, load16<16>(g.u + (c * g.m + token) * g.rank_pad + k));
                }
            return T == WC_T_FP16 ? g.unscale[token * rank_blocks + rb] : 1.f;
        };
        if (nb >= n1) continue;
        fetch();
        float unscale = 1.f;
        if constexpr (!kBlocks) {
            float f[KS][8];
            const float *p = g.part + token * g.rank_pad + 8 * gr;
            const float scale = g.scales ? g.scales[adapter] : 1.f;
#pragma unroll
            for (int s = 0; s < KS; s++)
#pragma unroll
                for (int e = 0; e < 8; e++) f[s][e] = 0.f;
            constexpr uint32_t kAtOnce = 4;  // parts on their way
            for (uint32_t z = 0; z < g.splits; z += kAtOnce) {
                f32x4 v[kAtOnce][KS][2];
#pragma unroll
                for (uint32_t q = 0; q < kAtOnce; q++)
#pragma unroll
                    for (int s = 0; s < 2 * KS; s++)
                        v[q][s / 2][s % 2] = *reinterpret_cast<const f32x4 *>(
                            p + min(z + q, g.splits - 1) * (g.m * g.rank_pad) + 32 * (s / 2) + 4 * (s % 2));
#pragma unroll
                for (uint32_t q = 0; q < kAtOnce; q++)
#pragma unroll
                    for (int s = 0; s < KS; s++)
#pragma unroll
                        for (int e = 0; e < 8; e++) f[s][e] += z + q < g.splits ? v[q][s][e / 4][e % 4] : 0.f;
            }
#pragma unroll
            for (int s = 0; s < KS; s++)
#pragma unroll
                for (int e = 0; e < 8; e++) f[s][e] = 32 * s + 8 * gr + e < g.rank ? scale * f[s][e] : 0.f;
            unscale = adapter_terms<T, KS>(f, u);
        }
        while (nb < n1) {
            f32x4 sum[4];
            for (uint32_t rb = 0; rb < rank_blocks; rb++) {
                float us = 1.f;
                if (kBlocks && rb) BRows<T, YT, KS>(g, adapter, 64 * rb).load(g, nb, bv);
                if (kBlocks) us = fetch_terms(rb);
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < KS; s++)
#pragma unroll
                        for (int c = kTerms - 1; c >= 0; c--) acc = Ty::mfma(bv[p][s], u[s][c], acc);
                    if (!kBlocks) sum[p] = acc;
                    else sum[p] = rb ? sum[p] + us * acc : us * acc;
                }
            }
            if (mine && nb + 64 <= n1) y.add(yr + nb, gr, sum, unscale);
            else if (mine) y_add_some<YT>(yr + nb, gr, n1 - nb, sum[0], sum[1], sum[2], sum[3], unscale);
            nb += 256;
            if (nb < n1) fetch();
        }
    }
}

// y += B u for many tokens and ranks up to 64.  Grid: x = tiles of 128 tokens
// x row blocks, z = turns.  The four waves of a block take 32 tokens each and the same
// 64 rows of B, which reach them through LDS in operand order: B would
// otherwise pass through the L1 cache once per 32 tokens, twice as many bytes
// as y, and how much can be on its way into that cache is what bounds a
// kernel that only streams.  y is read and written in whole lines, 64 elements
// of a token at a time, and past the caches where it is larger than they are
// (kStream); the products come to that order through LDS as well.  8192 tokens
// of 16 adapters of rank 64, 14336 rows, BF16: 119 us, 3.9 TB/s of y.
template <int T, int YT, int KS, bool kStream>
__global__ __launch_bounds__(256, KS == 2 && (T == WC_T_FP16 || YT == WC_T_FP32) ? 2 : 3) void k_adapters_up_many(AdapterArgs g)
{
    using Ty = Type<T>;
    using Y = Type<YT>;
    using YE = typename Y::elem;
    using X8 = typename Ty::x8;
    constexpr int kTerms = Terms<T>::kCount, TT = 2, kPer = Y::kPer16;
    constexpr uint32_t kLanes = 64 / kPer, kRows = 64 / kLanes, kVecs = 32 / kRows;  // of y: lanes a row, rows a load, loads
    constexpr uint32_t kPitch = 68;  // floats of a token's 64 products in LDS: rows in different banks
    __shared__ u32x4 sb[2][4][KS][64];
    __shared__ float products[4][32][kPitch];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t row_blocks = (g.rows + g.row_block - 1) / g.row_block;
    const uint32_t block = xcd_block();
    const uint64_t tile = (uint64_t)(block / row_blocks) * 128;
    const uint32_t n0 = (block % row_blocks) * g.row_block, n1 = min(g.rows, n0 + g.row_block);
    const uint32_t yrow = lane / kLanes, ycol = lane % kLanes * kPer;  // the lane's place in a load of y
    TileIds low(g, tile, 64), high(g, tile + 64, 64);
    uint64_t mlow, mhigh;
    uint32_t adapter, turn = 0;
    while (low.pending | high.pending) {
        if (low.next(adapter, mlow)) {
            high.take(adapter, mhigh);
        } else {
            mlow = 0;
            high.next(adapter, mhigh);
        }
        if (turn++ % gridDim.z != blockIdx.z) continue;
        const uint32_t mask = (uint32_t)((wave & 2 ? mhigh : mlow) >> (32 * (wave & 1)));  // the wave's tokens
        X8 u[TT][KS][kTerms];
        float unscale[TT];
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const uint64_t token = min(tile + 32 * wave + 16 * t + i, g.m - 1);
#pragma unroll
            for (int s = 0; s < KS; s++)
#pragma unroll
                for (int c = 0; c < kTerms; c++)
                    u[t][s][c] = __builtin_bit_cast(X8, load16<16>(g.u + (c * g.m + token) * g.rank_pad + 32 * s + 8 * gr));
            unscale[t] = T == WC_T_FP16 ? g.unscale[token] : 1.f;
        }
        const BRows<T, WC_T_FP32, KS> rows(g, adapter, 0);  // row i of tile p is row 16 p + i
        YE *const y0 = static_cast<YE *>(g.y) + (tile + 32 * wave) * g.y_stride + ycol;
        u32x4 nextb[KS];
        rows.load(g, n0, (int)wave, nextb);
        uint32_t buf = 0;
        for (uint32_t nb = n0; nb < n1; nb += 64, buf ^= 1) {
            const bool whole = nb + 64 <= n1;
            u32x4 y[kVecs];
            if (whole) {
#pragma unroll
                for (uint32_t q = 0; q < kVecs; q++) {
                    const uint32_t r = q * kRows + yrow;
                    if ((mask >> r) & 1) y[q] = read16<Y::kBytes, kStream>(y0 + r * g.y_stride + nb);
                }
            }
#pragma unroll
            for (int s = 0; s < KS; s++) sb[buf][wave][s][lane] = rows.kept(nextb[s], s);
            __syncthreads();  // the other buffer's last readers passed the barrier before this one
            if (nb + 64 < n1) rows.load(g, nb + 64, (int)wave, nextb);
            if (!mask) continue;
#pragma unroll
            for (int t = 0; t < TT; t++)
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    f32x4 sum{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < KS; s++) {
                        const X8 bv = __builtin_bit_cast(X8, sb[buf][p][s][lane]);
#pragma unroll
                        for (int c = kTerms - 1; c >= 0; c--) sum = Ty::mfma(bv, u[t][s][c], sum);
                    }
                    *reinterpret_cast<f32x4 *>(&products[wave][16 * t + i][16 * p + 4 * gr]) = unscale[t] * sum;
                }
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // a wave's own LDS: in order
#pragma unroll
            for (uint32_t q = 0; q < kVecs; q++) {
                const uint32_t r = q * kRows + yrow;
                if (!((mask >> r) & 1)) continue;
                YE *const yp = y0 + r * g.y_stride + nb;
                float f[kPer];
                if (whole) {
                    Y::unpack(y[q], f);
#pragma unroll
                    for (int e = 0; e < kPer; e++) f[e] += products[wave][r][ycol + e];
                    write16<Y::kBytes, kStream>(yp, Y::pack(f));
                } else {
                    for (uint32_t e = 0; e < (uint32_t)kPer && nb + ycol + e < n1; e++)
                        yp[e] = Y::from_f32(Y::to_f32(yp[e]) + products[wave][r][ycol + e]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        }
        __syncthreads();
    }
}

// Both products in one launch, for few tokens: every block of 1,024 rows (or
// a few times that) works out u for itself, its sixteen waves sharing the
// columns, while its first rows of B and y are on their way.  The row blocks
// of a tile's turn are on one XCD (blocks are dealt to the XCDs in the order
// of their number), where A comes from the L2 cache after the first of them.
// One token, rank 16, 4096 x 4096: 8.2 us, of which most is waiting for the
// ids, then A and x, then the other waves; two launches took 18.3 us a call.
// Grid: turns x tiles of 16 tokens, rounded up to 8, x row blocks.
template <int T, int YT, int RT>
__global__ __launch_bounds__(1024) void k_adapters_few(AdapterArgs g)
{
    using Ty = Type<T>;
    using YE = typename Type<YT>::elem;
    using X8 = typename Ty::x8;
    constexpr int kTerms = Terms<T>::kCount, KS = (RT + 1) / 2, Q = RT == 4 ? 1 : 4;
    constexpr int kPad = 32 * KS + 4;  // + 4: tokens in different banks
    __shared__ f32x4 part[16][RT][64];
    __shared__ float su[16][kPad];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t row_blocks = (g.rows + g.row_block - 1) / g.row_block;
    const uint32_t tiles = (uint32_t)((g.m + 15) / 16), slot = blockIdx.x / 8;
    const uint32_t pair = slot / row_blocks * 8 + blockIdx.x % 8;  // of a turn and a tile
    const uint64_t tile = (uint64_t)(pair % tiles) * 16;
    const uint32_t n0 = (slot % row_blocks) * g.row_block, n1 = min(g.rows, n0 + g.row_block);
    TileIds ids(g, tile, 16);
    uint32_t adapter;
    uint64_t mask;
    for (uint32_t turn = 0;; turn++) {
        if (!ids.next(adapter, mask)) return;
        if (turn == pair / tiles) break;
    }
    const bool mine = (mask >> i) & 1;
    // lanes of other tokens repeat the first one's loads
    const uint64_t token = tile + (mine ? i : (uint32_t)__builtin_ctzll(mask));
    YE *yr = static_cast<YE *>(g.y) + token * g.y_stride;
    uint32_t nb = n0 + 64 * wave;
    YRow<YT> y;
    X8 bv[4][KS];
    const BRows<T, YT, KS> rows(g, adapter, 0);
    auto fetch = [&]() {
        if (mine && nb + 64 <= n1) y.load(yr + nb, gr);
        rows.load(g, nb, bv);
    };
    if (nb < n1) fetch();
    const uint16_t *xr = g.x + token * g.x_stride;
    const uint16_t *ar[RT];
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) {
        ar[r] = g.a + ((uint64_t)adapter * g.rank + min(16 * r + i, g.rank - 1)) * g.cols;
        acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (uint32_t j = 0; 32 * wave_step<16>(wave, j) < g.cols; j += Q) {
        X8 av[Q][RT], xv[Q];
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const uint32_t k = 32 * wave_step<16>(wave, j + q) + 8 * gr;
            const bool in = k < g.cols;
            xv[q] = __builtin_bit_cast(X8, in ? load16<16>(xr + k) : u32x4{0u, 0u, 0u, 0u});
#pragma unroll
            for (int r = 0; r < RT; r++)
                av[q][r] = __builtin_bit_cast(X8, in ? load16<16>(ar[r] + k) : u32x4{0u, 0u, 0u, 0u});
        }
#pragma unroll
        for (int q = 0; q < Q; q++)
#pragma unroll
            for (int r = 0; r < RT; r++) acc[r] = Ty::mfma(av[q][r], xv[q], acc[r]);
    }
#pragma unroll
    for (int r = 0; r < RT; r++) part[wave][r][lane] = acc[r];
    __syncthreads();
    if (threadIdx.x < 256 * RT) {  // a thread per token and rank: element e of lane l of tile r
        const uint32_t r = threadIdx.x >> 8, l = (threadIdx.x >> 2) & 63, e = threadIdx.x & 3;
        const uint32_t rank = 16 * r + 4 * (l >> 4) + e;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 16; w++) v += part[w][r][l][e];
        su[l & 15][rank] = rank < g.rank ? v * (g.scales ? g.scales[adapter] : 1.f) : 0.f;
    }
    __syncthreads();
    float f[KS][8];
#pragma unroll
    for (int s = 0; s < KS; s++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t k = 32 * s + 8 * gr + e;
            f[s][e] = mine && k < 16 * RT ? su[i][k] : 0.f;
        }
    X8 u[KS][kTerms];
    const float unscale = adapter_terms<T, KS>(f, u);
    while (nb < n1) {
        f32x4 d[4];
#pragma unroll
        for (int p = 0; p < 4; p++) {
            d[p] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < KS; s++)
#pragma unroll
                for (int c = kTerms - 1; c >= 0; c--) d[p] = Ty::mfma(bv[p][s], u[s][c], d[p]);
        }
        if (mine && nb + 64 <= n1) y.add(yr + nb, gr, d, unscale);
        else if (mine) y_add_some<YT>(yr + nb, gr, n1 - nb, d[0], d[1], d[2], d[3], unscale);
        nb += 1024;
        if (nb < n1) fetch();
    }
}

}  // namespace ops
}  // namespace wc

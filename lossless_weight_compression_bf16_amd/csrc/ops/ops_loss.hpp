// ops_loss.hpp -- softmax cross entropy over a large vocabulary from hidden
// states, without the logits in memory, and its gradient:
//   z = H W^T,  lse_r = log sum_v exp z_rv,  loss_r = lse_r - z_r,t,
//   G_rv = (gl_r + gz_r) exp(z_rv - lse_r) - gl_r [v = t_r],  dH = G W,  dW = G^T H
// with gl and gz the gradients of loss and lse (gl = 0 where there is no token).
//
//   k_loss_few, k_loss        statistics (largest logit, sum of exponentials) of a tile of z
//   k_loss_join               lse and loss of a row from them
//   k_loss_rows               what the gradient needs of a row, and H without the rows that have no part in it
//   k_loss_grad_few, k_loss_grad  G of a piece of the vocabulary: z again, then the formula
//   k_product                 dH += G W and dW = G^T H of that piece
//
// G is fp32 and meets the matrix cores as a sum of two 16-bit terms, 16 of its bits in BF16 and 22
// in FP16, so that the gradients are as near to the exact ones as their own rounding leaves them (4096 rows, 128256 x 4096,
// BF16: 0.166% off in the root mean square, as fp32 products rounded once are; 100 rows, 50257 x 768, FP16: 0.0209%). Each term is a
// product of its own, one after the other in the same sums. A caller who asks for `rounded` has one
// term: 0.207% and 0.0239% for 9760 us in place of 16200, and 84 in place of 113.
//
// What bounds them, and what they take: up to 64 rows, reading W (61 rows, 128256 x 4096: 157 us, 6.7 TB/s); many rows, the
// matrix cores at the clock that their power leaves (4096 rows: 3230 us, 1.33 PFLOP/s; the gradients 16200 us, 21.5 TFLOP with both terms, 1.33);
// in between, stages of 0.9 us in which one wave on a SIMD reads, waits and multiplies in turn (100
// rows, 50257 x 768: 113 us in all).  G goes through memory once for each product: in the tile that made it, only one of the
// two could use it, and the other would make it again, a third product for each.
#pragma once

#include "ops_common.hpp"
#include "ops_grouped.hpp"
#include "ops_tiles.hpp"

namespace wc {
namespace ops {

struct LossArgs {
    const uint16_t *h, *w;
    uint64_t h_stride;
    uint32_t w_row;
    const int64_t *tokens;
    uint32_t m, vocab, k;
    uint32_t parts;      // tiles of the vocabulary
    float2 *part;        // m x parts: the largest logit of a tile, and the sum of exp(z - it)
    float *given;        // m: the logit of the row's token
    float *loss, *lse;
    uint32_t *err;
};

// Largest logit and sum of exponentials so far; -inf and 0 of nothing, and of
// nothing but -inf.  NaN and +inf make the sum NaN.
struct Stat {
    float most, sum;

    __device__ __forceinline__ static float base(float most) { return most == -kInf ? 0.f : most; }
    __device__ __forceinline__ void join(float most2, float sum2)
    {
        const float all = fmaxf(most, most2), b = base(all);
        sum = sum * exp2_fast((most - b) * kLog2e) + sum2 * exp2_fast((most2 - b) * kLog2e);
        most = all;
    }
};

// A tile of z: rows from m0 on against columns from n0 on.
template <class Ti>
struct LogitsJob {
    typename Ti::Place place;
    uint32_t m0, rows, n0, cols;

    // Tile (r, c) of m rows of h and v rows of w, of k values each.
    template <int BM, int BN>
    __device__ __forceinline__ void set(uint32_t r, uint32_t c, const uint16_t *h, uint64_t h_stride, uint32_t m, const uint16_t *w,
                                        uint64_t w_row, uint32_t v, uint32_t k)
    {
        m0 = BM * r;
        rows = min((uint32_t)BM, m - m0);
        n0 = BN * c;
        cols = min((uint32_t)BN, v - n0);
        place.q = Ti::Q::Where::at(h + m0 * h_stride, rows, k);
        place.p = Ti::P::Where::at(w + n0 * w_row, cols, k);
        place.k = k;
    }
};

// Statistics of a block's tiles.  Grid: 8 ceil(tiles / 8), or kCus (each_tile).
template <int T, int BM, int BN>
__global__ __launch_bounds__(256, tile_blocks(BM, BN)) void k_loss(LossArgs g)
{
    using Ti = Tile<T, BM, BN, true, true>;
    using Job = LogitsJob<Ti>;
    __shared__ __attribute__((aligned(1024))) char b0[Ti::kBytes];
    __shared__ __attribute__((aligned(1024))) char b1[Ti::kBytes];
    __shared__ float2 own[Ti::kNamed ? Ti::kWavesN : 1][Ti::kNamed ? BM : 1];
    // a wave's: where no other tile's operands are on their way, in their place
    float2(*stats)[BM] = reinterpret_cast<float2(*)[BM]>(Ti::kNamed ? (void *)own : (void *)b0);
    const uint32_t down = (g.m + BM - 1) / BM;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    Ti ti(g.h_stride, g.w_row);
    each_tile<Ti, Job>(
        ti, b0, b1,
        [&](uint32_t n, Job &j) {
            const uint32_t t = xcd_piece(block_of(n), down * g.parts);
            if (t >= down * g.parts) return false;
            uint32_t r, c;
            tile_of(t, down, g.parts, r, c);
            j.template set<BM, BN>(r, c, g.h, g.h_stride, g.m, g.w, g.w_row, g.vocab, g.k);
            return true;
        },
        [&](const Ti &ti, const Job &j) {
            if constexpr (!Ti::kNamed) Ti::all_done();
#pragma unroll
            for (int b = 0; b < Ti::kM; b++) {
                const uint32_t row = Ti::q_row(wave, b) + i;
                const int64_t token = row < j.rows ? g.tokens[j.m0 + row] - j.n0 : -1;
                Stat s{-kInf, 0.f};
#pragma unroll
                for (int a = 0; a < Ti::kN; a++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const uint32_t col = Ti::p_row(wave, a) + 4 * gr + e;
                        const float z = ti.acc[a][b][e];
                        if (col < j.cols) s.most = fmaxf(s.most, z);
                        if (token == (int64_t)col && col < j.cols) g.given[j.m0 + row] = z;
                    }
                const float base = Stat::base(s.most);
#pragma unroll
                for (int a = 0; a < Ti::kN; a++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (Ti::p_row(wave, a) + 4 * gr + e < j.cols) s.sum += exp2_fast((ti.acc[a][b][e] - base) * kLog2e);
                s.join(__shfl_xor(s.most, 16, 64), __shfl_xor(s.sum, 16, 64));
                s.join(__shfl_xor(s.most, 32, 64), __shfl_xor(s.sum, 32, 64));
                if (gr == 0) stats[wave % Ti::kWavesN][row] = float2{s.most, s.sum};
            }
            lds_barrier();
            if (threadIdx.x < j.rows) {
                Stat s{stats[0][threadIdx.x].x, stats[0][threadIdx.x].y};
#pragma unroll
                for (int w = 1; w < Ti::kWavesN; w++) s.join(stats[w][threadIdx.x].x, stats[w][threadIdx.x].y);
                g.part[(uint64_t)(j.m0 + threadIdx.x) * g.parts + j.n0 / BN] = float2{s.most, s.sum};
            }
        });
}

constexpr uint32_t kLossFew = 16;  // rows, at most, of k_loss_few and k_loss_grad_few

// The same for up to kLossFew rows: 32 columns of z for a block (128 without kSplit).
template <int T, bool kSplit>
__global__ __launch_bounds__(256, 2) void k_loss_few(LossArgs g)
{
    __shared__ Strip strips[4][2];
    __shared__ float2 stats[4][kLossFew];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t n0 = kSplit ? 32 * blockIdx.x : 128 * blockIdx.x + 32 * wave;
    constexpr uint32_t kShares = kSplit ? 1 : 4;  // waves with statistics of the same row
    if (g.m == 1) {
        const int64_t token = g.tokens[0];
        Stat s{-kInf, 0.f};
        for (uint32_t q = 0; q < (kSplit ? 1 : 4); q++) {
            const uint32_t n = n0 + 8 * (kSplit ? wave : q);
            if (n >= g.vocab) break;
            float mine = -kInf;
            one_product<T>(g.w, g.w_row, g.vocab, n, g.k, g.h, [&](uint32_t v, float z) {
                mine = z;
                if ((int64_t)v == token) g.given[0] = z;
            });
            const float most = wave_max(mine), base = Stat::base(most);
            s.join(most, wave_sum(lane < 8 && n + lane < g.vocab ? exp2_fast((mine - base) * kLog2e) : 0.f));
        }
        if (lane == 0) stats[wave][0] = float2{s.most, s.sum};
    } else if (kSplit || n0 < g.vocab) {
        few_product<T, kSplit, 1>(g.w, g.w_row, g.vocab, n0, g.k, g.h, g.h_stride, g.m, strips,
                               [&](uint32_t t, const uint32_t(&first)[2], f32x4 v0, f32x4 v1) {
                                   const uint32_t row = 16 * t + i;
                                   const int64_t token = row < g.m ? g.tokens[row] : -1;
                                   Stat s{-kInf, 0.f};
#pragma unroll
                                   for (int m = 0; m < 2; m++)
#pragma unroll
                                       for (uint32_t e = 0; e < 4; e++) {
                                           const uint32_t v = first[m] + 4 * gr + e;
                                           const float z = m ? v1[e] : v0[e];
                                           if (v < n0 + 16 * m || v >= g.vocab) continue;  // of the rows before
                                           s.most = fmaxf(s.most, z);
                                           if (token == (int64_t)v) g.given[row] = z;
                                       }
                                   const float base = Stat::base(s.most);
#pragma unroll
                                   for (int m = 0; m < 2; m++)
#pragma unroll
                                       for (uint32_t e = 0; e < 4; e++) {
                                           const uint32_t v = first[m] + 4 * gr + e;
                                           if (v < n0 + 16 * m || v >= g.vocab) continue;
                                           s.sum += exp2_fast(((m ? v1[e] : v0[e]) - base) * kLog2e);
                                       }
                                   s.join(__shfl_xor(s.most, 16, 64), __shfl_xor(s.sum, 16, 64));
                                   s.join(__shfl_xor(s.most, 32, 64), __shfl_xor(s.sum, 32, 64));
                                   if (gr == 0) stats[kSplit ? 0 : wave][row] = float2{s.most, s.sum};
                               });
    } else if (lane < kLossFew) {
        stats[wave][lane] = float2{-kInf, 0.f};
    }
    __syncthreads();
    if (threadIdx.x < g.m) {
        Stat s{-kInf, 0.f};
#pragma unroll
        for (uint32_t w = 0; w < 4; w++)
            if (w < kShares || g.m == 1) s.join(stats[w][threadIdx.x].x, stats[w][threadIdx.x].y);
        g.part[(uint64_t)threadIdx.x * g.parts + blockIdx.x] = float2{s.most, s.sum};
    }
}

// One block per row.
__global__ __launch_bounds__(256) void k_loss_join(LossArgs g)
{
    constexpr uint32_t kAtOnce = 8;  // parts of a thread whose loads are on their way together
    __shared__ float2 waves[4];
    const uint32_t r = blockIdx.x;
    const float2 *p = g.part + (uint64_t)r * g.parts;
    const int64_t t = g.tokens[r];
    const float given = g.given[r];  // not used, and not written, without a token
    Stat s{-kInf, 0.f};
    for (uint32_t q0 = threadIdx.x; q0 < g.parts; q0 += 256 * kAtOnce) {
        float2 v[kAtOnce];
        float most = -kInf, sum = 0.f;
#pragma unroll
        for (uint32_t q = 0; q < kAtOnce; q++) v[q] = p[min(q0 + 256 * q, g.parts - 1)];
#pragma unroll
        for (uint32_t q = 0; q < kAtOnce; q++) most = fmaxf(most, v[q].x);
#pragma unroll
        for (uint32_t q = 0; q < kAtOnce; q++)
            if (q0 + 256 * q < g.parts) sum += v[q].y * exp2_fast((v[q].x - Stat::base(most)) * kLog2e);
        s.join(most, sum);
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) s.join(__shfl_xor(s.most, o, 64), __shfl_xor(s.sum, o, 64));
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = float2{s.most, s.sum};
    __syncthreads();
    if (threadIdx.x) return;
#pragma unroll
    for (int w = 1; w < 4; w++) s.join(waves[w].x, waves[w].y);
    const float log_sum = __builtin_amdgcn_logf(s.sum) * kLn2;
    const bool nothing = s.most == -kInf && s.sum == 0.f;
    g.lse[r] = nothing ? -kInf : s.most + log_sum;
    float loss = 0.f;
    if (t >= 0 && t < (int64_t)g.vocab) {
        // the difference of logits first: the two are near each other where a loss is small
        loss = nothing ? kInf : (s.most - given) + log_sum;
    } else if (t != -1) {
        loss = nan32();
        report(g.err, WC_EF_BAD_INDEX);
    }
    g.loss[r] = loss;
}

struct LossGradArgs {
    const uint16_t *h, *w;
    uint64_t h_stride;
    uint32_t w_row;
    const int64_t *tokens;
    const float *lse, *grad_loss, *grad_lse;
    uint32_t m, vocab, k;
    // scratch
    uint16_t *live;      // m x k: H, rows without a part in the gradient as zeros; or NULL
    f32x4 *rows;         // m: lse, gl + gz, gl, token
    float *most;         // kLossRowBlocks: the largest |gl|, |gl + gz| of some rows
    uint16_t *grad;      // m x pitch: G of a piece
    uint64_t again;      // elements from there to what those numbers leave of G, or 0: nothing is kept of it
    uint32_t pitch, v0, width;
    uint32_t *err;
};

__global__ __launch_bounds__(256) void k_loss_rows(LossGradArgs g)
{
    float most = 0.f;
    for (uint32_t r = blockIdx.x; r < g.m; r += gridDim.x) {
        const int64_t t = g.tokens[r];
        const bool is = t >= 0 && t < (int64_t)g.vocab;
        const float lse = g.lse[r], none = lse == -kInf ? 0.f : 1.f;
        const float gl = is && g.grad_loss && none ? g.grad_loss[r] : 0.f;
        const float all = gl + (g.grad_lse && none ? g.grad_lse[r] : 0.f);
        const bool live = gl != 0.f || all != 0.f;
        most = fmaxf(most, fmaxf(fabsf(gl), fabsf(all)));
        if (threadIdx.x == 0) {
            g.rows[r] = f32x4{lse, all, gl, __builtin_bit_cast(float, is ? (int32_t)t : -1)};
            if (!is && t != -1) report(g.err, WC_EF_BAD_INDEX);
        }
        if (g.live)
            for (uint32_t c = 8 * threadIdx.x; c < g.k; c += 2048)
                *reinterpret_cast<u32x4 *>(g.live + (uint64_t)r * g.k + c) =
                    only(live, *reinterpret_cast<const u32x4 *>(g.h + r * g.h_stride + c));
    }
    if (threadIdx.x == 0) g.most[blockIdx.x] = most;
}

__device__ __forceinline__ float loss_gradient(f32x4 row, float z, uint32_t v, float scale)
{
    const float all = row[1], p = all == 0.f ? 0.f : all * exp2_fast((z - row[0]) * kLog2e);
    return scale * ((int32_t)v == __builtin_bit_cast(int32_t, (float)row[3]) ? p - row[2] : p);
}

// G of a block's tiles, in two terms with kWhole.  Grid: 8 ceil(tiles / 8), or kCus (each_tile).
template <int T, int BM, int BN, bool kWhole>
__global__ __launch_bounds__(256, tile_blocks(BM, BN)) void k_loss_grad(LossGradArgs g)
{
    using Ti = Tile<T, BM, BN, true, true>;
    using Job = LogitsJob<Ti>;
    __shared__ __attribute__((aligned(1024))) char b0[Ti::kBytes];
    __shared__ __attribute__((aligned(1024))) char b1[Ti::kBytes];
    const uint32_t down = (g.m + BM - 1) / BM, across = (g.width + BN - 1) / BN, wave = threadIdx.x >> 6;
    float unscale, early = 1.f;  // as in k_product
    if constexpr (Ti::kNamed) early = loss_scale<T>(g.most, unscale);
    Ti ti(g.h_stride, g.w_row);
    each_tile<Ti, Job>(
        ti, b0, b1,
        [&](uint32_t n, Job &j) {
            const uint32_t t = xcd_piece(block_of(n), down * across);
            if (t >= down * across) return false;
            uint32_t r, c;
            tile_of(t, down, across, r, c);
            j.template set<BM, BN>(r, c, g.h, g.h_stride, g.m, g.w + (uint64_t)g.v0 * g.w_row, g.w_row, g.width, g.k);
            return true;
        },
        [&](const Ti &ti, const Job &j) {
            float scale = early;
            if constexpr (!Ti::kNamed) scale = loss_scale<T>(g.most, unscale);
            f32x4 info[Ti::kM];
#pragma unroll
            for (int b = 0; b < Ti::kM; b++) info[b] = g.rows[j.m0 + min(Ti::q_row(wave, b) + (threadIdx.x & 15), j.rows - 1)];
            uint16_t *to = g.grad + (uint64_t)j.m0 * g.pitch + j.n0;
            const auto gradient = [&](uint32_t row, uint32_t col, f32x4 z) {
                const f32x4 of_row = info[(row / 16 - wave / Ti::kWavesN) / Ti::kWavesM];
#pragma unroll
                for (uint32_t e = 0; e < 4; e++)
                    z[e] = col + e < j.cols ? loss_gradient(of_row, z[e], g.v0 + j.n0 + col + e, scale) : 0.f;
                return z;
            };
            const auto put = [&](uint32_t row, uint32_t col, u32x4 v, auto... rest) {
                if (row >= j.rows || j.n0 + col >= g.pitch) return;
                uint16_t *at = to + (uint64_t)row * g.pitch + col;
                *reinterpret_cast<u32x4 *>(at) = v;
                ((*reinterpret_cast<u32x4 *>(at + g.again) = rest), ...);
            };
            if constexpr (kWhole) each_eight_whole<T>(ti, gradient, put);
            else each_eight<T>(ti, gradient, put);
        });
}

// The same for up to kLossFew rows.
template <int T, bool kSplit>
__global__ __launch_bounds__(256, 2) void k_loss_grad_few(LossGradArgs g)
{
    __shared__ Strip strips[4][2];
    const uint32_t wave = threadIdx.x >> 6, i = threadIdx.x & 15, gr = (threadIdx.x & 63) >> 4;
    const uint32_t n0 = 32 * (kSplit ? blockIdx.x : 4 * blockIdx.x + wave);
    if (!kSplit && n0 >= g.width) return;
    float unscale;
    const float scale = loss_scale<T>(g.most, unscale);
    few_product<T, kSplit, 1>(g.w + (uint64_t)g.v0 * g.w_row, g.w_row, g.width, n0, g.k, g.h, g.h_stride, g.m, strips,
                           [&](uint32_t t, const uint32_t(&first)[2], f32x4 v0, f32x4 v1) {
                               const uint32_t row = 16 * t + i;
                               if (row >= g.m) return;
                               const f32x4 info = g.rows[row];
                               uint16_t *to = g.grad + (uint64_t)row * g.pitch;
#pragma unroll
                               for (int m = 0; m < 2; m++)
#pragma unroll
                                   for (uint32_t e = 0; e < 4; e++) {
                                       const uint32_t v = first[m] + 4 * gr + e;
                                       if (v < n0 + 16 * m || v >= g.width) continue;
                                       const float z = m ? v1[e] : v0[e];
                                       const float all = loss_gradient(info, z, g.v0 + v, scale);
                                       const uint16_t first_term = Type<T>::from_f32(all);
                                       to[v] = first_term;
                                       if (!g.again) continue;
                                       const float had = Type<T>::to_f32(first_term);
                                       to[g.again + v] = Type<T>::from_f32(fabsf(had) < kInf ? all - had : 0.f);
                                   }
                               if (gr == 0 && n0 + 32 >= g.width)
                                   for (uint32_t v = g.width; v < g.pitch; v++) {
                                       to[v] = 0;
                                       if (g.again) to[g.again + v] = 0;
                                   }
                           });
}

struct ProductArgs {
    const uint16_t *q, *p;
    uint64_t again;           // elements between the two terms of Q, where it has as many
    uint64_t q_stride, p_stride;
    uint32_t m, n, k;         // of D
    uint32_t splits;          // of k, each with its own m x n of part
    float *part;              // or NULL: D goes to out
    uint32_t add;             // to what part holds
    uint16_t *out;
    uint64_t out_stride;
    const float *most;        // of G, by which it was scaled
};

// D = Q P^T of whole matrices, Q in kTerms terms.  kQAlong: k along the rows of Q's memory; P has
// it across.  Grid: 8 ceil(tiles / 8), or kCus (each_tile).
template <int T, int BM, int BN, bool kQAlong, int kTerms>
__global__ __launch_bounds__(256, tile_blocks(BM, BN)) void k_product(ProductArgs g)
{
    using Ti = Tile<T, BM, BN, kQAlong, false>;
    struct Job {
        typename Ti::Place place;
        uint32_t split, m0, rows, n0;
    };
    __shared__ __attribute__((aligned(1024))) char b0[Ti::kBytes];
    __shared__ __attribute__((aligned(1024))) char b1[Ti::kBytes];
    const uint32_t down = (g.m + BM - 1) / BM, across = (g.n + BN - 1) / BN, each = down * across;
    const uint32_t stages = (g.k + kTileK - 1) / kTileK;
    // asked for at the end where a block has one tile, and its loads would wait for this one
    float early = 1.f;
    if constexpr (Ti::kNamed) loss_scale<T>(g.most, early);
    Ti ti(g.q_stride, g.p_stride);
    each_tile<Ti, Job, kTerms>(
        ti, b0, b1,
        [&](uint32_t n, Job &j) {
            const uint32_t t = xcd_piece(block_of(n), each * g.splits);
            if (t >= each * g.splits) return false;
            uint32_t r, c;
            tile_of(t % each, down, across, r, c);
            j.split = t / each;
            j.m0 = BM * r;
            j.rows = min((uint32_t)BM, g.m - j.m0);
            j.n0 = BN * c;
            const uint32_t k0 = kTileK * (uint32_t)((uint64_t)stages * j.split / g.splits);
            const uint32_t k = min(g.k, kTileK * (uint32_t)((uint64_t)stages * (j.split + 1) / g.splits)) - k0;
            // G has whole 16 bytes of a row, zeros behind its width
            if constexpr (kQAlong) j.place.q = Ti::Q::Where::at(g.q + j.m0 * g.q_stride + k0, j.rows, (k + 7) / 8 * 8);
            else j.place.q = Ti::Q::Where::at(g.q + k0 * g.q_stride + j.m0, k, (g.m + 7) / 8 * 8 - j.m0);
            j.place.p = Ti::P::Where::at(g.p + k0 * g.p_stride + j.n0, k, g.n - j.n0);
            j.place.k = k;
            return true;
        },
        [&](const Ti &ti, const Job &j) {
            if (g.part) {
                float *part = g.part + ((uint64_t)j.split * g.m + j.m0) * g.n + j.n0;
                each_four(ti, [&](uint32_t row, uint32_t col, f32x4 v) {
                    if (row >= j.rows || j.n0 + col >= g.n) return;
                    f32x4 *to = reinterpret_cast<f32x4 *>(part + (uint64_t)row * g.n + col);
                    *to = g.add ? *to + v : v;
                });
            } else {
                uint16_t *out = g.out + j.m0 * g.out_stride + j.n0;
                float unscale = early;
                if constexpr (!Ti::kNamed) loss_scale<T>(g.most, unscale);
                each_eight<T>(ti, [&](uint32_t, uint32_t, f32x4 v) { return v * unscale; },
                              [&](uint32_t row, uint32_t col, u32x4 v) {
                                  if (row < j.rows && j.n0 + col < g.n)
                                      *reinterpret_cast<u32x4 *>(out + row * g.out_stride + col) = v;
                              });
            }
        },
        2 * g.again);
}

}  // namespace ops
}  // namespace wc

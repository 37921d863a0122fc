// ops_moe.hpp -- a whole mixture-of-experts layer for up to 64 tokens:
//   l = R x,  p = softmax(l),  the top_k experts of each token (weights p, or
//   p over the sum of the chosen),  y = sum_e p_e W2_e (silu(W1_e x) * W3_e x)
// with silu(v) = v / (1 + exp(-v)).
//
//   k_moe_route   router logits, split over blocks along the columns
//   k_moe_select  softmax and the top_k of each token: one wave per token
//   k_moe_route_one  both, where the router is small: one block per token
//   k_moe_up      h = silu(W1 x) * (W3 x), for every expert with tokens
//   k_moe_down    p W2 h of every expert
//   k_moe_join    their sums
//   k_moe_up_one, k_moe_down_one  instead of these three for a single token
// What bounds it: every expert that has tokens is read once, 6 bytes per
// row and column; with few tokens that is all the time there is.  So weights
// stay in their own row-major layout (no repacked copy), are read in whole
// lines and reach the matrix cores through LDS (Strip), 16 rows of weights
// against 16 tokens per MFMA, and experts with more than 16 tokens meet them
// all while their weights are there.  Products are exact and summed in fp32.
//
// h is fp32.  The matrix cores take it as a sum of 16-bit terms that the
// second product makes of it as it is read: of BF16 three, which are all of
// its 24 bits; of FP16 two of 11 bits, after a scaling by a power of two that
// brings the largest of a token's h in that expert to 2^14..2^15, so that
// they hold 22 bits of it and of whatever is down to 2^-17 of it, at any size.
//
// MFMA 16x16x32 (lane l = 16 g + i): A operand row i, k = 8 g .. 8 g + 7;
// B operand column i, the same k; D column i, rows 4 g .. 4 g + 3.  Here A is
// weights, a column a token.
#pragma once

#include "ops_common.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kMoeMaxTokens = 64, kMoeMaxTop = 16, kMoeMaxExperts = 1024;
constexpr uint32_t kMoeRouteSplits = 16;

struct MoeArgs {
    const uint16_t *x, *router, *w1, *w3, *w2;
    uint64_t x_stride, up_expert, up_row, down_expert, down_row;  // strides in elements
    uint16_t *out;
    uint64_t out_stride;
    uint32_t m, experts, top_k, cols, inner, renormalize;
    // scratch
    float *logits;        // route_splits x m x experts_pad
    int32_t *ids;         // m x top_k
    float *weights;       // m x top_k
    float *h;             // (m top_k) x inner
    uint32_t *most;       // m top_k: bits of the largest |h|
    float *part;          // (m top_k) x cols: each expert's part of y
    uint32_t experts_pad, route_splits, route_steps, slots;
};

// logits[split][t][e]: 16 experts per block, the columns of a split over its
// four waves.
template <int T, int TT>
__global__ __launch_bounds__(256) void k_moe_route(MoeArgs g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    __shared__ f32x4 part[4][TT][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t split = blockIdx.x % g.route_splits, e0 = 16 * (blockIdx.x / g.route_splits);
    const uint16_t *rr = g.router + (uint64_t)min(e0 + i, g.experts - 1) * g.cols;
    const uint16_t *xr[TT];
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; t++) {
        xr[t] = g.x + min(16 * t + i, g.m - 1) * g.x_stride;
        acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const uint32_t s0 = split * g.route_steps, s1 = min((g.cols + 31) / 32, s0 + g.route_steps);
    for (uint32_t j = 0; s0 + wave_step<4>(wave, j) < s1; j += 2) {
        X8 rv[2], xv[2][TT];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const uint32_t st = s0 + wave_step<4>(wave, j + u), c = 32 * st + 8 * gr, k = min(c, g.cols - 8);
            const bool in = st < s1 && c < g.cols;
            rv[u] = __builtin_bit_cast(X8, only(in, load16<16>(rr + k)));
#pragma unroll
            for (int t = 0; t < TT; t++) xv[u][t] = __builtin_bit_cast(X8, only(in, load16<16>(xr[t] + k)));
        }
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int t = 0; t < TT; t++) acc[t] = Ty::mfma(rv[u], xv[u][t], acc[t]);
    }
#pragma unroll
    for (int t = 0; t < TT; t++) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave < TT) {
        const uint32_t t = 16 * wave + i;
        const f32x4 v = (part[0][wave][lane] + part[1][wave][lane]) + (part[2][wave][lane] + part[3][wave][lane]);
        if (t < g.m) *reinterpret_cast<f32x4 *>(g.logits + ((uint64_t)split * g.m + t) * g.experts_pad + e0 + 4 * gr) = v;
    }
}

// The experts of one token by one wave, largest logit first, equal ones by
// their number, NaN last: always top_k different ones.  logit(e): expert e's.
template <int PER, class F>
__device__ __forceinline__ void moe_choose(const MoeArgs &g, uint32_t t, F logit)
{
    const uint32_t lane = threadIdx.x & 63;
    uint32_t key[PER];  // lane's expert 64 q + lane; 0: none, or taken
    float l[PER], most = -kInf, sum = 0.f;
#pragma unroll
    for (int q = 0; q < PER; q++) {
        const uint32_t e = 64 * q + lane;
        l[q] = e < g.experts ? logit(e) : -kInf;
        key[q] = e < g.experts ? key_of(l[q]) : 0u;
        most = fmaxf(most, l[q]);
    }
    most = wave_max(most);
#pragma unroll
    for (int q = 0; q < PER; q++)
        if (64 * q + lane < g.experts) sum += exp2_fast((l[q] - most) * kLog2e);  // NaN or +inf: NaN
    sum = wave_sum(sum);
    float chosen = 0.f, mine = 0.f;
    uint32_t id = 0;
    for (uint32_t s = 0; s < g.top_k; s++) {
        uint32_t best = 0;
#pragma unroll
        for (int q = 0; q < PER; q++) best = max(best, key[q]);
        best = ~wave_min(~best);
        uint32_t e = ~0u;
#pragma unroll
        for (int q = PER - 1; q >= 0; q--)
            if (key[q] == best) e = 64 * q + lane;
        e = wave_min(e);
#pragma unroll
        for (int q = 0; q < PER; q++)
            if (64 * q + lane == e) key[q] = 0;
        const float p = exp2_fast((key_value(best) - most) * kLog2e);
        chosen += p;
        if (lane == s) {
            mine = p;
            id = e;
        }
    }
    if (lane < g.top_k) {
        g.ids[t * g.top_k + lane] = (int32_t)id;
        g.most[t * g.top_k + lane] = 0;
        // p of a token with a NaN among its logits are NaN, the chosen ones' sum with them
        g.weights[t * g.top_k + lane] = mine / (g.renormalize && sum == sum ? chosen : sum);
    }
}

template <int PER>
__global__ __launch_bounds__(64) void k_moe_select(MoeArgs g)
{
    moe_choose<PER>(g, blockIdx.x, [&](uint32_t e) {
        const float *p = g.logits + (uint64_t)blockIdx.x * g.experts_pad + e;
        const uint64_t step = (uint64_t)g.m * g.experts_pad;
        float v[kMoeRouteSplits];  // all loads before the first sum
#pragma unroll
        for (uint32_t s = 0; s < kMoeRouteSplits; s++) v[s] = p[min(s, g.route_splits - 1) * step];
        float sum = v[0];
#pragma unroll
        for (uint32_t s = 1; s < kMoeRouteSplits; s++) sum += s < g.route_splits ? v[s] : 0.f;
        return sum;
    });
}

// Both for one token in one block, where the router is small: tiles of 16
// experts and, if they are fewer than the waves, pieces of the columns go
// round the waves; the token is the only column.
template <int T, int PER>
__global__ __launch_bounds__(1024) void k_moe_route_one(MoeArgs g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    constexpr uint32_t W = 16, U = 8;
    __shared__ float logits[W][64 * PER];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t tiles = g.experts_pad / 16, steps = (g.cols + 31) / 32;
    const uint32_t pieces = tiles < W ? W / tiles : 1u, piece = (steps + pieces - 1) / pieces;
    const uint16_t *xr = g.x + blockIdx.x * g.x_stride;
    for (uint32_t it = wave; it < tiles * pieces; it += W) {
        const uint32_t e0 = 16 * (it / pieces), pc = it % pieces, s1 = min(steps, (pc + 1) * piece);
        const uint16_t *rr = g.router + (uint64_t)min(e0 + i, g.experts - 1) * g.cols;
        f32x4 acc{0.f, 0.f, 0.f, 0.f};
        for (uint32_t st = pc * piece; st < s1; st += U) {
            X8 rv[U], xv[U];
#pragma unroll
            for (uint32_t u = 0; u < U; u++) {
                const uint32_t c = 32 * (st + u) + 8 * gr, k = min(c, g.cols - 8);
                const bool in = st + u < s1 && c < g.cols;
                rv[u] = __builtin_bit_cast(X8, only(in, load16<16>(rr + k)));
                xv[u] = __builtin_bit_cast(X8, only(in, load16<16>(xr + k)));
            }
#pragma unroll
            for (uint32_t u = 0; u < U; u++) acc = Ty::mfma(rv[u], xv[u], acc);
        }
        if (i == 0) *reinterpret_cast<f32x4 *>(&logits[pc][e0 + 4 * gr]) = acc;
    }
    __syncthreads();
    if (wave == 0)
        moe_choose<PER>(g, blockIdx.x, [&](uint32_t e) {
            float v = logits[0][e];
            for (uint32_t pc = 1; pc < pieces; pc++) v += logits[pc][e];
            return v;
        });
}

// The experts that have tokens, as a set in LDS.
struct MoeSet {
    uint32_t bits[kMoeMaxExperts / 32];
    int32_t ids[kMoeMaxTokens * kMoeMaxTop];

    __device__ void fill(const MoeArgs &g)
    {
        for (uint32_t q = threadIdx.x; q < kMoeMaxExperts / 32; q += blockDim.x) bits[q] = 0;
        __syncthreads();
        for (uint32_t q = threadIdx.x; q < g.m * g.top_k; q += blockDim.x) {
            const int32_t e = g.ids[q];
            ids[q] = e;
            atomicOr(&bits[e >> 5], 1u << (e & 31));
        }
        __syncthreads();
    }
    // how many experts, and the p-th of them (in every lane of a wave)
    __device__ uint32_t find(uint32_t p, uint32_t &expert) const
    {
        const uint32_t lane = threadIdx.x & 63;
        const uint32_t w = lane < kMoeMaxExperts / 32 ? bits[lane] : 0u;
        const uint32_t n = __popc(w);
        uint32_t upto = n;  // in words 0 .. lane
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up(upto, o, 64);
            if (lane >= (uint32_t)o) upto += v;
        }
        const uint32_t total = __shfl(upto, kMoeMaxExperts / 32 - 1, 64);
        const uint64_t has = __ballot(lane < kMoeMaxExperts / 32 && p < upto);
        const uint32_t word = has ? (uint32_t)__builtin_ctzll(has) : 0u;
        uint32_t rest = p - (__shfl(upto, word, 64) - __shfl(n, word, 64)), v = __shfl(w, word, 64);
        if (p < total)
            for (; rest; rest--) v &= v - 1;
        expert = 32 * word + (v ? __builtin_ctz(v) : 0u);
        return total;
    }
    // the tokens of an expert: lane l's choice of it, or -1
    __device__ int32_t choice(const MoeArgs &g, uint32_t expert) const
    {
        const uint32_t lane = threadIdx.x & 63;
        int32_t at = -1;
        if (lane < g.m)
            for (uint32_t s = 0; s < g.top_k; s++)
                if (ids[lane * g.top_k + s] == (int32_t)expert) at = (int32_t)(lane * g.top_k + s);
        return at;
    }
};

// acc[m][0][t] += W_m X_t over columns c0 .. c1 (multiples of 8) for M matrices
// of 16 rows and NT tiles of 16 tokens, whose numbers are 16-bit or, with
// kTerms, fp32 and taken as terms of scale[t] times them.  weights[m]: the
// first row; row(r): elements from there to row r; tokens(t): the lane's
// column.  acc[m][1][t] takes all terms but the first, so that these small
// products are not rounded to the large sum each time (of 64 tokens' results,
// 24 experts of 2048 x 7168, BF16, 0.05% are not the nearest number to the
// exact one, 0.07% with one sum; 13 tokens, 8 of 14336 x 4096, FP16, 0.39% and
// 0.46%; products and sums of fp32 numbers give 0.17% and 0.89%).  Loads past
// the end repeat the last 8 columns, and the operands are zero there.  The
// next columns are on their way while these are multiplied.
template <int T, int M, bool kTerms, int NT, class Row, class Tokens>
__device__ __forceinline__ void strip_product(const uint16_t *const (&weights)[M], Row row, Tokens tokens, uint32_t c0,
                                              uint32_t c1, Strip *strips, const float (&scale)[NT],
                                              f32x4 (&acc)[M][kTerms ? 2 : 1][NT])
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    constexpr int kSteps = kStripCols / 32, V = kTerms ? 2 : 1;  // vectors of 16 bytes for 8 numbers
    constexpr int S = 16 / (V * NT) < kSteps ? 16 / (V * NT) : kSteps, C = kTerms ? Terms<T>::kCount : 1;
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4, hi = lane >> 5, lo = lane & 31;
    uint32_t off[8];
#pragma unroll
    for (int u = 0; u < 8; u++) off[u] = row(2 * u + hi);
    const char *tk[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) tk[t] = reinterpret_cast<const char *>(tokens(t));
    u32x4 v[M][8], x[S][NT][V];
    auto fetch = [&](uint32_t c) {
        const uint32_t k = min(c + 8 * lo, c1 - 8);
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
            for (int u = 0; u < 8; u++) v[m][u] = read16<16, true>(weights[m] + (off[u] + k));
    };
    auto fetch_x = [&](uint32_t c, int s0) {
#pragma unroll
        for (int s = 0; s < S; s++) {
            const uint32_t k = min(c + 32 * (s0 + s) + 8 * gr, c1 - 8);
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int e = 0; e < V; e++) x[s][t][e] = load16<16>(tk[t] + (16 * V * (k / 8) + 16 * e));
        }
    };
    if (c0 < c1) {
        fetch(c0);
        fetch_x(c0, 0);
    }
    for (uint32_t c = c0; c < c1; c += kStripCols) {
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // a wave's own LDS: in order
        const bool there = c + 8 * lo < c1;
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
            for (int u = 0; u < 8; u++) strips[m].q[(2 * u + hi) * kStripPitch + lo] = only(there, v[m][u]);
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        if (c + kStripCols < c1) fetch(c + kStripCols);
#pragma unroll
        for (int s0 = 0; s0 < kSteps; s0 += S) {
            if (s0) fetch_x(c, s0);
#pragma unroll
            for (int s = 0; s < S; s++) {
                const bool in = c + 32 * (s0 + s) + 8 * gr < c1;
                X8 a[M];
#pragma unroll
                for (int m = 0; m < M; m++)
                    a[m] = __builtin_bit_cast(X8, strips[m].q[i * kStripPitch + 4 * (s0 + s) + gr]);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    X8 b[C];
                    if constexpr (kTerms) {
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const uint32_t w = x[s][t][e / 4][e % 4];
                            f[e] = in ? __builtin_bit_cast(float, w) * scale[t] : 0.f;
                        }
                        Terms<T>::split(f, b);
                    } else {
                        b[0] = __builtin_bit_cast(X8, only(in, x[s][t][0]));
                    }
#pragma unroll
                    for (int o = C - 1; o >= 0; o--)
#pragma unroll
                        for (int m = 0; m < M; m++) acc[m][o ? 1 : 0][t] = Ty::mfma(a[m], b[o], acc[m][o ? 1 : 0][t]);
                }
            }
        }
        if (c + kStripCols < c1) fetch_x(c + kStripCols, 0);
    }
}

// A wave's share of the columns for 16 rows of W1 and W3 of one expert against
// its tokens, up to 16 NT of them.
template <int T, int NT, int TT>
__device__ __forceinline__ void moe_up_rows(const MoeArgs &g, uint32_t expert, uint32_t n0, const int32_t *place,
                                            uint32_t count, uint32_t c0, uint32_t c1, Strip *strips,
                                            f32x4 (&gate)[TT], f32x4 (&up)[TT])
{
    const uint32_t i = threadIdx.x & 15;
    const uint64_t at = (uint64_t)expert * g.up_expert + (uint64_t)n0 * g.up_row;
    const uint16_t *const weights[2] = {g.w1 + at, g.w3 + at};
    const uint32_t rows = min(g.inner - n0, 16u), stride = (uint32_t)g.up_row;
    f32x4 acc[2][1][NT];
    const float scale[NT] = {};  // of no use here
#pragma unroll
    for (int t = 0; t < NT; t++) acc[0][0][t] = acc[1][0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    strip_product<T, 2, false, NT>(
        weights, [&](uint32_t r) { return min(r, rows - 1) * stride; },
        [&](int t) { return g.x + (uint64_t)((uint32_t)place[min(16 * t + i, count - 1)] / g.top_k) * g.x_stride; },
        c0, c1, strips, scale, acc);
#pragma unroll
    for (int t = 0; t < NT; t++) {
        gate[t] = acc[0][0][t];
        up[t] = acc[1][0][t];
    }
}

// A wave's share of the inner rows c0 .. c1 for twice 16 rows of W2 of one
// expert, from n[0] and n[1], against its tokens' h.
template <int T, int NT, int TT>
__device__ __forceinline__ void moe_down_rows(const MoeArgs &g, uint32_t expert, const uint32_t (&n)[2],
                                              const int32_t *place, uint32_t count, uint32_t c0, uint32_t c1,
                                              Strip *strips, f32x4 (&sum)[2][TT])
{
    const uint32_t i = threadIdx.x & 15, rows = min(g.cols, 16u), stride = (uint32_t)g.down_row;
    const uint16_t *const w = g.w2 + (uint64_t)expert * g.down_expert;
    const uint16_t *const weights[2] = {w + n[0] * g.down_row, w + n[1] * g.down_row};
    f32x4 acc[2][2][NT];
    float scale[NT], unscale[NT];
    uint32_t at[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        acc[0][0][t] = acc[0][1][t] = acc[1][0][t] = acc[1][1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        at[t] = (uint32_t)place[min(16 * t + i, count - 1)];
        scale[t] = term_scale<T>(T == WC_T_FP16 ? __builtin_bit_cast(float, g.most[at[t]]) : 0.f, unscale[t]);
    }
    strip_product<T, 2, true, NT>(
        weights, [&](uint32_t r) { return min(r, rows - 1) * stride; },
        [&](int t) { return g.h + (uint64_t)at[t] * g.inner; }, c0, c1, strips, scale, acc);
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int m = 0; m < 2; m++) sum[m][t] = unscale[t] * (acc[m][0][t] + acc[m][1][t]);
}

// The columns of one of four waves: a quarter, in multiples of `unit`.
__device__ __forceinline__ void wave_quarter(uint32_t cols, uint32_t unit, uint32_t wave, uint32_t &c0, uint32_t &c1)
{
    const uint32_t per = ((cols + 4 * unit - 1) / (4 * unit)) * unit;
    c0 = min(cols, wave * per);
    c1 = min(cols, c0 + per);
}

// A block's expert, the slot-th that has tokens, and its tokens: place[c] is
// token top_k + choice of column c.  Their number; 0 past the last expert.
__device__ __forceinline__ uint32_t moe_block(const MoeArgs &g, uint32_t slot, MoeSet &set, int32_t (&place)[64],
                                              uint32_t &expert)
{
    const uint32_t lane = threadIdx.x & 63, choices = g.m * g.top_k;
    const uint64_t below = (1ull << lane) - 1;
    if (choices <= 64) {
        // a choice per lane; experts in the order of their first choice.  No
        // barrier: every wave writes the same places and reads its own.
        const int32_t id = lane < choices ? g.ids[lane] : -1;
        uint64_t pending = __ballot(id >= 0), mask = 0;
        for (uint32_t p = 0; p <= slot; p++) {
            if (!pending) return 0;
            expert = (uint32_t)__builtin_amdgcn_readlane(id, __builtin_ctzll(pending));
            mask = __ballot(id == (int32_t)expert);
            pending &= ~mask;
        }
        if ((mask >> lane) & 1) place[__popcll(mask & below)] = (int32_t)lane;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        return (uint32_t)__popcll(mask);
    }
    set.fill(g);
    if (slot >= set.find(slot, expert)) return 0;
    const int32_t mine = set.choice(g, expert);
    const uint64_t mask = __ballot(mine >= 0);
    if (mine >= 0) place[__popcll(mask & below)] = mine;  // the same from every wave
    __syncthreads();
    return (uint32_t)__popcll(mask);
}

// h of 16 inner rows of one expert.  Grid: slots x inner / 16.  Columns over
// the four waves.  Reading W1 and W3 is the bound: 64 tokens, 256 experts of
// 2048 x 7168, 1.90 ms, 6.9 TB/s; 13 tokens, 8 of 14336 x 4096, FP16, 282 us,
// 6.7 TB/s.  Operands straight from memory, 64 bytes of each of 16 rows at a time,
// took 4.5 ms for the former's whole layer where this takes 2.9.
template <int T, int TT>
__global__ __launch_bounds__(256, 2) void k_moe_up(MoeArgs g)
{
    __shared__ MoeSet set;
    __shared__ int32_t place[64];
    __shared__ Strip strips[4][2];
    f32x4(*part)[2 * TT][64] = reinterpret_cast<f32x4(*)[2 * TT][64]>(&strips[0][0]);  // [4], when the strips are done
    static_assert(sizeof(strips) >= 4 * 2 * TT * 64 * 16, "the waves' sums fit into the strips");
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t slot = blockIdx.x % g.slots, n0 = 16 * (blockIdx.x / g.slots);
    uint32_t expert, c0, c1;
    const uint32_t count = moe_block(g, slot, set, place, expert);
    if (count == 0) return;
    wave_quarter(g.cols, kStripCols, wave, c0, c1);
    const uint32_t c = 16 * wave + i;
    uint32_t seen = 0;  // the largest |h| so far, or less; looked at here, where nothing waits for it
    if (T == WC_T_FP16 && wave < TT && c < count)
        seen = __hip_atomic_load(g.most + place[c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    f32x4 gate[TT], up[TT];
    if (TT == 1 || count <= 16) moe_up_rows<T, 1, TT>(g, expert, n0, place, count, c0, c1, strips[wave], gate, up);
    else if (TT == 2 || count <= 32) moe_up_rows<T, 2, TT>(g, expert, n0, place, count, c0, c1, strips[wave], gate, up);
    else moe_up_rows<T, 4, TT>(g, expert, n0, place, count, c0, c1, strips[wave], gate, up);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TT; t++) {
        if (16 * t < (int)count) {
            part[wave][t][lane] = gate[t];
            part[wave][TT + t][lane] = up[t];
        }
    }
    __syncthreads();
    const uint32_t n = n0 + 4 * gr;
    if (wave >= TT) return;
    float most = 0.f;
    if (c < count && n < g.inner) {
        const uint32_t q = TT + wave;
        const f32x4 gv = (part[0][wave][lane] + part[1][wave][lane]) + (part[2][wave][lane] + part[3][wave][lane]);
        const f32x4 uv = (part[0][q][lane] + part[1][q][lane]) + (part[2][q][lane] + part[3][q][lane]);
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float v = gv[e], w = v / (1.f + exp2_fast(-v * kLog2e)) * uv[e];
            h[e] = w;
            most = fmaxf(most, fabsf(w));
        }
        *reinterpret_cast<f32x4 *>(g.h + (uint64_t)place[c] * g.inner + n) = h;
    }
    if constexpr (T == WC_T_FP16) {
        // A maximum does not depend on the order.  Few blocks raise it, and
        // all of them raising the same few words would take longer than their
        // weights (13 tokens on 8 wide experts: 580 us for the layer).
        most = fmaxf(most, __shfl_xor(most, 16, 64));
        most = fmaxf(most, __shfl_xor(most, 32, 64));
        const uint32_t bits = __builtin_bit_cast(uint32_t, most);
        if (gr == 0 && c < count && seen < bits) atomicMax(g.most + place[c], bits);
    }
}

// p W2 h of one expert into part[token top_k + choice].  Grid: slots x
// columns / 128 (kSplit: / 32).  A wave has twice 16 rows of W2 of its own, or
// with kSplit, where blocks would be too few, a quarter of their inner rows.
// Where the last 16 rows would run past the end they begin earlier: those that
// two waves have come out the same.  Reading W2 is the bound, and making the
// terms of h beside it (5% of the first): the same two layers, 991 us (6.6
// TB/s) and 164 us (5.7).  Where an expert has more than 32 tokens the terms
// cost more: 64 tokens on 2 experts of 14336 x 4096, BF16, 385 us for the
// layer, 338 with h rounded to two BF16 terms by the first product.  With 16
// rows a wave h is as many lines on their way into the L1 cache as the rows,
// and more for 13 tokens: with those two terms 1075 us, against 940 with 32
// rows, and 181 against 149.
template <int T, int TT, bool kSplit>
__global__ __launch_bounds__(256, 2) void k_moe_down(MoeArgs g)
{
    __shared__ MoeSet set;
    __shared__ int32_t place[64];
    __shared__ Strip strips[4][2];
    f32x4(*sums)[2 * TT][64] = reinterpret_cast<f32x4(*)[2 * TT][64]>(&strips[0][0]);  // [4], when the strips are done
    static_assert(sizeof(strips) >= 4 * 2 * TT * 64 * 16, "the waves' sums fit into the strips");
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t slot = blockIdx.x % g.slots;
    const uint32_t n0 = kSplit ? 32 * (blockIdx.x / g.slots) : 128 * (blockIdx.x / g.slots) + 32 * wave;
    const uint32_t last = g.cols > 16 ? g.cols - 16 : 0u, rows[2] = {min(n0, last), min(n0 + 16, last)};
    uint32_t expert, c0 = 0, c1 = g.inner;
    const uint32_t count = moe_block(g, slot, set, place, expert);
    if (count == 0) return;
    if (kSplit) wave_quarter(g.inner, kStripCols, wave, c0, c1);
    f32x4 sum[2][TT];
    if (n0 < g.cols) {
        Strip *const st = strips[wave];
        if (TT == 1 || count <= 16) moe_down_rows<T, 1, TT>(g, expert, rows, place, count, c0, c1, st, sum);
        else if (TT == 2 || count <= 32) moe_down_rows<T, 2, TT>(g, expert, rows, place, count, c0, c1, st, sum);
        else moe_down_rows<T, 4, TT>(g, expert, rows, place, count, c0, c1, st, sum);
    }
    if constexpr (kSplit) {
        __syncthreads();
#pragma unroll
        for (int m = 0; m < 2; m++)
#pragma unroll
            for (int t = 0; t < TT; t++)
                if (16 * t < (int)count) sums[wave][m * TT + t][lane] = sum[m][t];
        __syncthreads();
    }
    if (n0 >= g.cols) return;
#pragma unroll
    for (int m = 0; m < 2; m++) {
        const uint32_t n = rows[m] + 4 * gr;
#pragma unroll
        for (int t = 0; t < TT; t++) {
            const int q = m * TT + t;
            if ((kSplit && q % 4 != (int)wave) || 16 * t + i >= count || n >= g.cols) continue;
            f32x4 v = sum[m][t];
            if constexpr (kSplit) v = (sums[0][q][lane] + sums[1][q][lane]) + (sums[2][q][lane] + sums[3][q][lane]);
            const uint32_t at = (uint32_t)place[16 * t + i];
            *reinterpret_cast<f32x4 *>(g.part + (uint64_t)at * g.cols + n) = g.weights[at] * v;
        }
    }
}

// y from the experts' parts, in the order of each token's choices.
template <int T>
__global__ __launch_bounds__(64) void k_moe_join(MoeArgs g)
{
    const uint32_t q = blockIdx.x * 64 + threadIdx.x, per = g.cols / 4;
    if (q >= g.m * per) return;
    const uint32_t t = q / per, n = 4 * (q % per);
    const float *p = g.part + (uint64_t)t * g.top_k * g.cols + n;
    f32x4 v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (uint32_t s = 0; s < g.top_k; s++) v += *reinterpret_cast<const f32x4 *>(p + (uint64_t)s * g.cols);
    uint16_t *o = g.out + t * g.out_stride + n;
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = Type<T>::from_f32(v[e]);
}

// One token.  Its rows of weights meet one column, so that the matrix cores
// would be a sixteenth used and the way through LDS only cost time: a wave
// reads whole rows, 512 columns at a time, eight of a lane, and multiplies them
// in fp32 with a vector that stays in registers; h stays in fp32.  A block of
// the second product has all of the token's experts, so that no launch joins
// them.  8 of 64 experts of 1024 x 2048: 14.4 + 8.0 us (4.7 and 4.2 TB/s)
// where the three kernels above take 15.1 + 11.4 + 3.9; 2 of 8 experts of
// 14336 x 4096, where reading is all there is, 130 us for the layer and 126.

// acc[r] += scale * row r of `rows` (`step` elements apart), columns c0 .. c1,
// times v, per lane.  vec(c, f): eight values of v from column c.
template <int T, int R, class Vec>
__device__ __forceinline__ void rows_product(const uint16_t *const (&rows)[R], uint32_t c0, uint32_t c1, Vec vec,
                                             float (&acc)[R])
{
    const uint32_t lane = threadIdx.x & 63;
    auto some = [&](uint32_t c, bool in) {
        u32x4 w[R];
        float f[8];
        const uint32_t k = in ? c : c1 - 8;
#pragma unroll
        for (int r = 0; r < R; r++) w[r] = read16<16, true>(rows[r] + k);
        vec(k, f);
#pragma unroll
        for (int r = 0; r < R; r++) {
            float a[8];
            Type<T>::unpack(w[r], a);
            float sum = acc[r];
#pragma unroll
            for (int e = 0; e < 8; e++) sum = __builtin_fmaf(a[e], f[e], sum);
            acc[r] = in ? sum : acc[r];
        }
    };
    uint32_t c = c0 + 8 * lane;
    const uint32_t whole = c0 + (c1 - c0) / 512 * 512;
#pragma unroll 2
    for (; c < whole; c += 512) some(c, true);
    if (whole < c1) some(c, c < c1);
}

// h of four inner rows of one of the token's experts per wave.
// Grid: choices x inner / 16, rounded up.
template <int T>
__global__ __launch_bounds__(256) void k_moe_up_one(MoeArgs g)
{
    constexpr int R = 4;
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, s = blockIdx.x % g.top_k;
    const uint32_t n0 = 16 * (blockIdx.x / g.top_k) + R * wave;
    if (n0 >= g.inner) return;  // a multiple of 8: all four rows are there
    const uint64_t at = (uint64_t)(uint32_t)g.ids[s] * g.up_expert + (uint64_t)n0 * g.up_row;
    const uint16_t *rows[2 * R];
    float acc[2 * R];
#pragma unroll
    for (int r = 0; r < R; r++) {
        rows[r] = g.w1 + at + r * g.up_row;
        rows[R + r] = g.w3 + at + r * g.up_row;
    }
#pragma unroll
    for (int r = 0; r < 2 * R; r++) acc[r] = 0.f;
    rows_product<T, 2 * R>(rows, 0, g.cols, [&](uint32_t c, float *f) { Type<T>::unpack(load16<16>(g.x + c), f); }, acc);
#pragma unroll
    for (int r = 0; r < 2 * R; r++) acc[r] = wave_sum(acc[r]);
    float *h = g.h + (uint64_t)s * g.inner + n0;
#pragma unroll
    for (int r = 0; r < R; r++)
        if (lane == (uint32_t)r) h[r] = acc[r] / (1.f + exp2_fast(-acc[r] * kLog2e)) * acc[R + r];
}

// y of eight columns per block: its waves share the experts and, where those
// are fewer, their inner rows.  Grid: columns / 8.
template <int T>
__global__ __launch_bounds__(1024) void k_moe_down_one(MoeArgs g)
{
    constexpr int R = 8;
    constexpr uint32_t W = 16;
    __shared__ float sums[W][R];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, n0 = R * blockIdx.x;
    const uint32_t chunks = (g.inner + 511) / 512, most = (W + g.top_k - 1) / g.top_k;
    const uint32_t per = (chunks + most - 1) / most, pieces = (chunks + per - 1) / per;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; r++) acc[r] = 0.f;
    for (uint32_t q = wave; q < g.top_k * pieces; q += W) {
        const uint32_t s = q / pieces, c0 = q % pieces * per * 512, c1 = min(g.inner, c0 + per * 512);
        const uint16_t *w = g.w2 + (uint64_t)(uint32_t)g.ids[s] * g.down_expert + (uint64_t)n0 * g.down_row;
        const float *h = g.h + (uint64_t)s * g.inner, p = g.weights[s];
        const uint16_t *rows[R];
        float part[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            rows[r] = w + r * g.down_row;
            part[r] = 0.f;
        }
        rows_product<T, R>(
            rows, c0, c1,
            [&](uint32_t c, float *f) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(h + c), b = *reinterpret_cast<const f32x4 *>(h + c + 4);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    f[e] = a[e];
                    f[4 + e] = b[e];
                }
            },
            part);
#pragma unroll
        for (int r = 0; r < R; r++) acc[r] = __builtin_fmaf(p, part[r], acc[r]);
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        acc[r] = wave_sum(acc[r]);
        if (lane == (uint32_t)r) sums[wave][r] = acc[r];
    }
    __syncthreads();
    if (threadIdx.x < R) {
        float v = sums[0][threadIdx.x];
#pragma unroll
        for (uint32_t w = 1; w < W; w++) v += sums[w][threadIdx.x];
        g.out[n0 + threadIdx.x] = Type<T>::from_f32(v);
    }
}

}  // namespace ops
}  // namespace wc

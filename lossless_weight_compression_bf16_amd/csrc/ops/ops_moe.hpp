// ops_moe.hpp -- a whole mixture-of-experts layer for up to 64 tokens:
//   l = R x,  p = softmax(l),  the top_k experts of each token (weights p, or
//   p over the sum of the chosen),  y = sum_e p_e W2_e (silu(W1_e x) * W3_e x)
// with silu(v) = v / (1 + exp(-v)).
//
//   k_moe_route   router logits, split over blocks along the columns
//   k_moe_select  softmax and the top_k of each token: one wave per token
//   k_moe_route_one  both, where the router is small: one block per token
//   k_moe_up      h = silu(W1 x) * (W3 x), for every expert with tokens
//   k_moe_down    y = sum p W2 h, in the order of the experts
//   k_moe_join    where few rows of y make k_moe_down split the experts
// What bounds it: every expert that has tokens is read once, 6 bytes per
// row and column; with few tokens that is all the time there is.  So weights
// go from memory into the matrix cores' registers in their own row-major
// layout (no repacked copy), 16 rows of weights against 16 tokens per MFMA,
// and experts with more than 16 tokens meet them all while their weights are
// in registers.  Products are exact and summed in fp32.
//
// h leaves k_moe_up as two 16-bit terms, BF16 h = a + b (16 bits), FP16
// h / 256 = a + b / 4096 with a and b accumulated apart (22 bits, |h| up to
// 2^24 and down to 2^-20), so that y is rounded once, at the end: one term
// alone would add as much error as that rounding.
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
    uint16_t *h;          // 2 terms x (m top_k) x inner
    float *part;          // parts x m x cols
    uint32_t experts_pad, route_splits, route_steps, slots, parts;
};

template <int T>
struct MoeTerms;  // h as two 16-bit terms, and what their sums are multiplied by
template <>
struct MoeTerms<WC_T_BF16> {
    static constexpr float kScale[2] = {1.f, 1.f};
    __device__ static void split(float h, uint16_t &a, uint16_t &b)
    {
        a = Type<WC_T_BF16>::from_f32(h);
        const float t = Type<WC_T_BF16>::to_f32(a);
        b = Type<WC_T_BF16>::from_f32(fabsf(t) < kInf ? h - t : 0.f);
    }
};
template <>
struct MoeTerms<WC_T_FP16> {
    static constexpr float kScale[2] = {256.f, 1.f / 16.f};
    __device__ static void split(float h, uint16_t &a, uint16_t &b)
    {
        const float v = h * (1.f / 256.f);
        a = Type<WC_T_FP16>::from_f32(v);
        const float t = Type<WC_T_FP16>::to_f32(a);
        b = Type<WC_T_FP16>::from_f32(fabsf(t) < kInf ? (v - t) * 4096.f : 0.f);
    }
};

__device__ __forceinline__ u32x4 zero4() { return u32x4{0u, 0u, 0u, 0u}; }
__device__ __forceinline__ u32x4 only(bool in, u32x4 v)  // all lanes load, some drop what they got
{
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = in ? v[e] : 0u;
    return v;
}

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
        g.weights[t * g.top_k + lane] = mine / (g.renormalize ? chosen : sum);
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

// A wave's share of the columns for 16 rows (the lane's at `row`) of W1 and W3
// of one expert against its tokens, up to 16 NT of them, into part.
template <int T, int NT, int TT>
__device__ __forceinline__ void moe_up_rows(const MoeArgs &g, uint64_t row, const int32_t *place, uint32_t count,
                                            f32x4 (&part)[4][2 * TT][64])
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    constexpr int U = NT == 4 ? 2 : 4;  // steps on their way at once
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint16_t *w1 = g.w1 + row, *w3 = g.w3 + row, *xr[NT];
    f32x4 acc[2][NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        xr[t] = g.x + (uint64_t)((uint32_t)place[min(16 * t + i, count - 1)] / g.top_k) * g.x_stride;
        acc[0][t] = acc[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (uint32_t j = 0; 32 * wave_step<4>(wave, j) < g.cols; j += U) {
        X8 a[U], b[U], xv[U][NT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            // past the rows' end the loads repeat their last numbers, and the operands are zero
            const uint32_t c = 32 * wave_step<4>(wave, j + u) + 8 * gr, k = min(c, g.cols - 8);
            const bool in = c < g.cols;
            a[u] = __builtin_bit_cast(X8, only(in, load16<16>(w1 + k)));
            b[u] = __builtin_bit_cast(X8, only(in, load16<16>(w3 + k)));
#pragma unroll
            for (int t = 0; t < NT; t++) xv[u][t] = __builtin_bit_cast(X8, only(in, load16<16>(xr[t] + k)));
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
                acc[0][t] = Ty::mfma(a[u], xv[u][t], acc[0][t]);
                acc[1][t] = Ty::mfma(b[u], xv[u][t], acc[1][t]);
            }
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
        part[wave][t][lane] = acc[0][t];
        part[wave][TT + t][lane] = acc[1][t];
    }
}

// h of 16 inner rows of one expert.  Grid: slots x inner / 16; a slot is the
// p-th expert that has tokens.  Columns over the four waves.
template <int T, int TT>
__global__ __launch_bounds__(256) void k_moe_up(MoeArgs g)
{
    __shared__ MoeSet set;
    __shared__ f32x4 part[4][2 * TT][64];
    __shared__ int32_t place[64];  // token top_k + choice of column c
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t slot = blockIdx.x % g.slots, n0 = 16 * (blockIdx.x / g.slots);
    set.fill(g);
    uint32_t expert;
    if (slot >= set.find(slot, expert)) return;
    const int32_t mine = set.choice(g, expert);
    const uint64_t mask = __ballot(mine >= 0);
    const uint32_t count = (uint32_t)__popcll(mask);
    if (mine >= 0) place[__popcll(mask & ((1ull << lane) - 1))] = mine;  // the same from every wave
    __syncthreads();
    const uint64_t row = (uint64_t)expert * g.up_expert + (uint64_t)min(n0 + i, g.inner - 1) * g.up_row;
    if (TT == 1 || count <= 16) moe_up_rows<T, 1, TT>(g, row, place, count, part);
    else if (TT == 2 || count <= 32) moe_up_rows<T, 2, TT>(g, row, place, count, part);
    else moe_up_rows<T, 4, TT>(g, row, place, count, part);
    __syncthreads();
    const uint32_t n = n0 + 4 * gr, c = 16 * wave + i;
    if (wave < TT && c < count && n < g.inner) {
        const f32x4 gate = (part[0][wave][lane] + part[1][wave][lane]) + (part[2][wave][lane] + part[3][wave][lane]);
        const uint32_t q = TT + wave;
        const f32x4 up = (part[0][q][lane] + part[1][q][lane]) + (part[2][q][lane] + part[3][q][lane]);
        uint16_t a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const float v = gate[e];
            MoeTerms<T>::split(v / (1.f + exp2_fast(-v * kLog2e)) * up[e], a[e], b[e]);
        }
        uint16_t *h = g.h + (uint64_t)place[c] * g.inner + n;
        const u32x2 va{(uint32_t)a[0] | ((uint32_t)a[1] << 16), (uint32_t)a[2] | ((uint32_t)a[3] << 16)};
        const u32x2 vb{(uint32_t)b[0] | ((uint32_t)b[1] << 16), (uint32_t)b[2] | ((uint32_t)b[3] << 16)};
        *reinterpret_cast<u32x2 *>(h) = va;
        *reinterpret_cast<u32x2 *>(h + (uint64_t)g.m * g.top_k * g.inner) = vb;
    }
}

// One piece of one expert in k_moe_down: steps s0 .. s1 of W2's 16 rows (the
// lane's at w2) against the expert's tokens, up to 16 NT of them, added into
// sums.  With kHalf, for up to 8 tokens, there are only 8 rows, and the
// operands' other halves are the same rows and tokens at the second half of
// the steps: of the product, the two quarters count where both are alike.
template <int T, int NT, bool kHalf>
__device__ __forceinline__ void moe_down_piece(const MoeArgs &g, const uint16_t *w2, const int32_t *place, uint32_t count,
                                               uint32_t s0, uint32_t s1, f32x4 (*sums)[4])
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    constexpr int U = NT == 1 ? 4 : NT == 2 ? 2 : 1;  // steps on their way at once: NT U x 2 KiB of h
    const uint32_t lane = threadIdx.x & 63, gr = lane >> 4, i = kHalf ? lane & 7 : lane & 15;
    const uint32_t half = kHalf ? (s1 - s0 + 1) / 2 : 0, second = kHalf && (lane & 8) ? half : 0;
    const uint32_t e1 = kHalf ? min(s1, s0 + second + half) : s1;  // the end of the lane's steps
    const uint64_t plane = (uint64_t)g.m * g.top_k * g.inner;
    const uint16_t *hr[NT];
    int32_t at[NT];
    f32x4 acc[2][NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
        at[t] = place[min(16 * t + i, count - 1)];
        hr[t] = g.h + (uint64_t)at[t] * g.inner;
        acc[0][t] = acc[1][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (uint32_t st = s0; st < (kHalf ? s0 + half : s1); st += U) {
        X8 a[U], h0[U][NT], h1[U][NT];
#pragma unroll
        for (int u = 0; u < U; u++) {
            // past the piece, or the rows' end, the operands are zero
            const uint32_t c = 32 * (st + u + second) + 8 * gr, k = min(c, g.inner - 8);
            const bool in = st + u + second < e1 && c < g.inner;
            a[u] = __builtin_bit_cast(X8, only(in, load16<16>(w2 + k)));
#pragma unroll
            for (int t = 0; t < NT; t++) {
                h0[u][t] = __builtin_bit_cast(X8, only(in, load16<16>(hr[t] + k)));
                h1[u][t] = __builtin_bit_cast(X8, only(in, load16<16>(hr[t] + plane + k)));
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
                acc[0][t] = Ty::mfma(a[u], h0[u][t], acc[0][t]);
                acc[1][t] = Ty::mfma(a[u], h1[u][t], acc[1][t]);
            }
    }
#pragma unroll
    for (int t = 0; t < NT; t++) {
        if (16 * t + i < count) {
            const float p = g.weights[at[t]];
            const f32x4 v = p * (MoeTerms<T>::kScale[0] * acc[0][t] + MoeTerms<T>::kScale[1] * acc[1][t]);
            if constexpr (!kHalf) {
                sums[(uint32_t)at[t] / g.top_k][gr] += v;
            } else {
                f32x4 &s = sums[(uint32_t)at[t] / g.top_k][gr & 1];
                if (lane < 32 && !(lane & 8)) s += v;
                __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // a wave's own LDS: in order
                if (lane >= 32 && (lane & 8)) s += v;
            }
        }
    }
}

// 16 columns of y (rows of W2), with kHalf 8.  Grid: columns / 16 (8) x parts.  The experts
// with tokens, each cut into pieces along the inner rows where they are few,
// go round the W waves of all parts; a wave adds its tokens' products, times
// their weights, into a slice of LDS of its own, and at the end the slices
// are added in the order of the waves.
template <int T, int TT, int W, bool kHalf>
__global__ __launch_bounds__(64 * W, 4) void k_moe_down(MoeArgs g)
{
    using Ty = Type<T>;
    constexpr uint32_t kRows = kHalf ? 8 : 16;
    __shared__ MoeSet set;
    __shared__ f32x4 sums[W][16 * TT][4];   // [wave][token][column / 4]
    __shared__ int32_t place[W][64];
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & (kRows - 1);
    const uint32_t part = blockIdx.x % g.parts, n0 = kRows * (blockIdx.x / g.parts);
    for (uint32_t q = lane; q < 64 * TT; q += 64) sums[wave][q >> 2][q & 3] = f32x4{0.f, 0.f, 0.f, 0.f};
    set.fill(g);
    uint32_t expert;
    const uint32_t active = set.find(0, expert);
    // pieces of an expert: enough for every wave, as evenly as may be
    const uint32_t waves = W * g.parts, steps = (g.inner + 31) / 32;
    uint32_t pieces = active >= 8 * waves ? 1u : min((4 * waves + active - 1) / active, max(steps / 8, 1u));
    const uint32_t piece = (steps + pieces - 1) / pieces;
    pieces = (steps + piece - 1) / piece;
    const uint64_t row = (uint64_t)min(n0 + i, g.cols - 1) * g.down_row;
    for (uint32_t it = wave + W * part; it < active * pieces; it += waves) {
        set.find(it / pieces, expert);
        const int32_t mine = set.choice(g, expert);
        const uint64_t mask = __ballot(mine >= 0);
        const uint32_t count = (uint32_t)__popcll(mask);
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // a wave's own LDS: in order
        if (mine >= 0) place[wave][__popcll(mask & ((1ull << lane) - 1))] = mine;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        const uint16_t *w2 = g.w2 + (uint64_t)expert * g.down_expert + row;
        const uint32_t s0 = (it % pieces) * piece, s1 = min(steps, s0 + piece);
        if (TT == 1 || count <= 16) moe_down_piece<T, 1, kHalf>(g, w2, place[wave], count, s0, s1, sums[wave]);
        else if (TT == 2 || count <= 32) moe_down_piece<T, 2, false>(g, w2, place[wave], count, s0, s1, sums[wave]);
        else moe_down_piece<T, 4, false>(g, w2, place[wave], count, s0, s1, sums[wave]);
    }
    __syncthreads();
    for (uint32_t q = threadIdx.x; q < 4 * g.m; q += 64 * W) {
        const uint32_t t = q >> 2, n = n0 + 4 * (q & 3);
        if (4 * (q & 3) >= kRows || n >= g.cols) continue;
        f32x4 v = sums[0][t][q & 3];
#pragma unroll
        for (int w = 1; w < W; w++) v += sums[w][t][q & 3];
        if (g.parts == 1) {
            uint16_t *o = g.out + t * g.out_stride + n;
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = Ty::from_f32(v[e]);
        } else {
            *reinterpret_cast<f32x4 *>(g.part + ((uint64_t)part * g.m + t) * g.cols + n) = v;
        }
    }
}

template <int T>
__global__ __launch_bounds__(256) void k_moe_join(MoeArgs g)
{
    const uint32_t q = blockIdx.x * 256 + threadIdx.x, per = g.cols / 4;
    if (q >= g.m * per) return;
    const uint32_t t = q / per, n = 4 * (q % per);
    f32x4 v{0.f, 0.f, 0.f, 0.f};
    for (uint32_t p = 0; p < g.parts; p++) v += *reinterpret_cast<const f32x4 *>(g.part + ((uint64_t)p * g.m + t) * g.cols + n);
    uint16_t *o = g.out + t * g.out_stride + n;
#pragma unroll
    for (int e = 0; e < 4; e++) o[e] = Type<T>::from_f32(v[e]);
}

}  // namespace ops
}  // namespace wc

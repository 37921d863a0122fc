// wc_ops.hip -- C ABI of the operators beside the compressed weights (see
// include/wc.h): argument checks, launch shapes and scratch layout.  Like
// the codec's calls these only enqueue on the caller's stream; no
// allocation, no synchronisation, no global state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wc.h"
#include "ops_adapters.hpp"
#include "ops_common.hpp"
#include "ops_host.hpp"
#include "ops_logprobs.hpp"
#include "ops_moe.hpp"

using namespace wc::ops;

namespace {

// Blocks of a row of the log probabilities: one, up to the batches that its
// LDS has room for; more only for larger vocabularies, and then a second
// launch joins them.  (Four blocks a row for 64 rows of 128,256 logits took
// 12 us and 6 us for the join, against 16 us in one block and one launch.)
void logprob_slices(uint32_t vocab, uint32_t *slices, uint32_t *slice)
{
    const uint64_t s = ceil_div(vocab, kMaxSlice);
    *slice = (uint32_t)((ceil_div(vocab, s) + 7) / 8 * 8);
    *slices = (uint32_t)ceil_div(vocab, *slice);
}

uint64_t logprob_scratch(uint64_t m, uint32_t vocab, uint32_t top)
{
    uint32_t slices, slice;
    logprob_slices(vocab, &slices, &slice);
    return slices == 1 ? 0 : m * slices * (16 + 8ull * top);
}

// The same from row r on.
LogprobArgs from_row(LogprobArgs g, uint64_t r, uintptr_t bytes)
{
    g.logits = static_cast<const char *>(g.logits) + r * g.stride * bytes;
    g.tokens += r;
    g.logprob += r;
    g.entropy += r;
    g.lse += r;
    if (g.top) {
        g.top_logprobs += r * g.top;
        g.top_ids += r * g.top;
    }
    return g;
}

template <int T, bool kTop, int NT>
void launch_rows(const LogprobArgs &all, uint64_t m, hipStream_t stream)
{
    static_assert(NT >= kJoinThreads, "the join's grid is the smaller one");
    const uint64_t most = max_blocks(NT) / all.slices;
    for (uint64_t r = 0; r < m; r += most) {  // every launch's parts in the same scratch
        const LogprobArgs g = from_row(all, r, type_bytes(T));
        const uint64_t rows = m - r < most ? m - r : most;
        hipLaunchKernelGGL((k_logprobs<T, kTop, NT>), dim3((uint32_t)(rows * g.slices)), dim3(NT), 0, stream, g);
        if (g.slices > 1)
            hipLaunchKernelGGL((k_logprobs_join<T, kTop>), dim3((uint32_t)rows), dim3(kJoinThreads), 0, stream, g);
    }
}

template <int T>
wc_status launch_logprobs(const LogprobArgs &g, uint64_t m, hipStream_t stream)
{
    // 1,024 threads a row while every row has a compute unit of its own, else
    // 256; us with 1,024 and with 256, BF16, 5 best: 64 rows of 128256 17 and
    // 22, 256 rows 21 and 26, 300 rows 35 and 29, 512 rows 42 and 32, 2048 rows
    // 146 and 93; 256 rows of 50257 14.7 and 16.0, 300 rows 25 and 19
    const bool few = m * g.slices <= kCus;
    if (g.top) few ? launch_rows<T, true, 1024>(g, m, stream) : launch_rows<T, true, 256>(g, m, stream);
    else few ? launch_rows<T, false, 1024>(g, m, stream) : launch_rows<T, false, 256>(g, m, stream);
    return launched();
}

template <int T>
void launch_grad(LogprobGradArgs g, uint64_t m, hipStream_t stream)
{
    const uintptr_t es = type_bytes(T);
    // past the caches where logits and gradient do not fit into the last of them
    // (256 MiB); us through them and past them, MiB of logits: 19 11.6 and 12.4,
    // 48 21.7 and 22.3, 125 49.3 both, 171 73 and 65, 502 192 and 180
    const bool large = m * g.vocab * es > (128ull << 20);
    const uint64_t most = max_blocks(kGradThreads) / g.blocks;
    while (m) {
        const uint64_t rows = m < most ? m : most;
        const dim3 grid((uint32_t)(rows * g.blocks));
        if (large) hipLaunchKernelGGL((k_logprobs_grad<T, true>), grid, dim3(kGradThreads), 0, stream, g);
        else hipLaunchKernelGGL((k_logprobs_grad<T, false>), grid, dim3(kGradThreads), 0, stream, g);
        m -= rows;
        g.logits = static_cast<const char *>(g.logits) + rows * g.stride * es;
        g.out = static_cast<char *>(g.out) + rows * g.out_stride * es;
        g.tokens += rows;
        g.lse += rows;
        if (g.entropy) g.entropy += rows;
        if (g.grad_logprob) g.grad_logprob += rows;
        if (g.grad_entropy) g.grad_entropy += rows;
    }
}

// Launch shapes of the adapters: tiles of 16 tokens, each turn of a tile (an
// adapter) its own block, so that as many blocks as possible share the
// reading; or, with `many`, tiles of 128 tokens, where prompts repeat their
// adapter over many tokens, so that it is read once per tile.
struct AdapterPlan {
    bool few;                                                    // k_adapters_few
    bool terms;                                                  // k_adapters_terms
    uint32_t rank_pad, rank_blocks, tile, turns, splits, split_cols;  // k_adapters_down, k_adapters_down_many
    uint32_t up_tile, row_blocks, row_block;                     // k_adapters_up, k_adapters_up_many
    uint64_t tiles, up_tiles, u, unscale, scratch;               // u, unscale: their places in the scratch
};

AdapterPlan adapter_plan(uint64_t m, uint32_t n, uint32_t rank, uint32_t cols, uint32_t rows, bool many)
{
    AdapterPlan p{};
    p.rank_pad = (rank + 31) / 32 * 32;
    // one launch where reading A again costs less than the second launch: at
    // most 256 KiB of A for a block, which waits for them, and 16 MiB for all,
    // a block per 1,024 to 4,096 rows.  us in one launch and in two, FP32 y,
    // 4096 x 4096, one token of rank 16 (128 KiB) 10.7 and 15.4, of 32 13.0 and
    // 15.1, of 48 18.0 and 14.7, of 64 23 and 14.7; 64 tokens of rank 16 (8 MiB)
    // 14.3 and 17.5; 512 x 4096, one of rank 64 (64 KiB) 10.7 and 14.8; 4096 x
    // 14336, 32 tokens of rank 16 in 16 MiB 14.5, in 56 MiB 21.1, and 21.4.
    // Ranks over 64 would not leave k_adapters_few registers.
    const uint64_t reading = m * rank * cols * 2, pairs = ceil_div(ceil_div(m, 16) * (m < 16 ? m : 16), 8) * 8;
    for (uint32_t r = 1024; r <= 4096 && rank <= 64 && m <= 64 && 2ull * rank * cols <= (256u << 10) && !p.few; r *= 2) {
        p.row_block = r;
        p.row_blocks = (uint32_t)ceil_div(rows, r);
        p.few = reading * p.row_blocks <= (16ull << 20) && pairs * p.row_blocks <= max_blocks(1024);
    }
    // a tile of 128 tokens has few adapters, and the blocks of turns that it
    // does not have cost little: us for one turn and three, BF16, rank 64, 8192
    // tokens, 14336 rows: of 1 adapter 138 both, of 16 164 and 155, of 128 353
    // and 239
    p.turns = many ? (n < 1 ? 1 : n < 3 ? n : 3) : (uint32_t)(m < 16 ? m : 16);
    if (p.few) {
        p.tile = p.up_tile = 16;
        p.tiles = p.up_tiles = ceil_div(m, 16);
        return p;
    }
    p.rank_blocks = (uint32_t)ceil_div(rank, 64);
    p.tile = many ? 128 : 16;
    p.tiles = ceil_div(m, p.tile);
    // columns of a block: as many of its loads as are on their way at once, or
    // more where the tiles alone fill the compute units
    const uint32_t step = many ? kStripCols : 32 * 4 * kDownWaves;
    const uint64_t most = ceil_div(cols, step);
    // with tiles of 128, a second turn for every adapter's first tile
    const uint64_t blocks = many ? p.tiles + (n < p.tiles ? n : p.tiles) : p.tiles * p.turns;
    uint64_t splits = ceil_div(kCus, blocks * p.rank_blocks);
    if (splits > most) splits = most;
    if (splits > 8) splits = 8;
    p.split_cols = (uint32_t)(ceil_div(most, splits) * step);
    p.splits = (uint32_t)ceil_div(cols, p.split_cols);
    // k_adapters_up_many takes 128 tokens and 64 rows at a time, k_adapters_up
    // 16 and 256; the former has registers for the terms of 64 ranks, no more
    const bool wide = many && rank <= 64;
    p.up_tile = wide ? 128 : 16;
    p.up_tiles = ceil_div(m, p.up_tile);
    const uint32_t least = wide ? 64 : 256;
    uint64_t rb = ceil_div((wide ? 4 : 8) * kCus, p.up_tiles * (many ? 1 : p.turns));
    const uint64_t rmost = ceil_div(rows, least);
    if (rb > rmost) rb = rmost;
    p.row_block = (uint32_t)(ceil_div(ceil_div(rows, rb), least) * least);
    p.row_blocks = (uint32_t)ceil_div(rows, p.row_block);
    p.terms = many || rank > 64;
    p.u = 4ull * p.splits * m * p.rank_pad;
    p.unscale = p.u + (p.terms ? 2ull * Terms<WC_T_BF16>::kCount * m * p.rank_pad : 0);  // the most terms of all types
    p.scratch = p.unscale + (p.terms ? 4 * m * p.rank_blocks : 0);
    return p;
}

// Tiles of 128 tokens: where the tokens are many and an adapter has 64 of them
// or more (their number is the host's only word on how long its runs are: a
// tile of 128 takes its adapters three at a time).  us a call, tiles of 16 and
// of 128, BF16, 4096 x 4096: rank 64, 256 tokens of 2 adapters 35 and 22, 2048
// of 8 55 and 41, of 32 79 and 59, of 64 82 and 86; rank 16, 1024 tokens of 16
// 26 and 29, of 32 26 and 30, of 64 24 and 42.
bool many_tokens(uint64_t m, uint32_t n) { return m >= 256 && m >= 64ull * n; }

// Tokens of one set of launches: no grid of theirs comes near max_blocks
// (2^20 tiles of 16 tokens, and then one block of rows, or fewer tiles with
// up to 2,048 blocks more), and the scratch stays small.  Columns are in
// parts for less than 2^15 tokens only, up to 8 of them.
constexpr uint64_t kMaxTokens = 1ull << 24;

bool valid_adapters(uint64_t m, uint32_t rank, uint32_t cols, uint32_t rows)
{
    return m <= (1ull << 31) && rank >= 1 && rank <= kAdapterMaxRank && cols >= 8 && cols % 8 == 0 && rows >= 1 &&
           cols <= (1u << 30) && (uint64_t)rows * rank < (1ull << 31);
}

template <int T>
void launch_down(const AdapterArgs &g, const AdapterPlan &p, hipStream_t stream)
{
    const dim3 grid((uint32_t)(p.tiles * p.splits), p.rank_blocks, p.turns), block(64 * kDownWaves);
    if (g.rank <= 16) hipLaunchKernelGGL((k_adapters_down<T, 1>), grid, block, 0, stream, g);
    else if (g.rank <= 32) hipLaunchKernelGGL((k_adapters_down<T, 2>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_adapters_down<T, 4>), grid, block, 0, stream, g);
}

template <int T>
void launch_down_many(const AdapterArgs &g, const AdapterPlan &p, hipStream_t stream)
{
    const dim3 grid((uint32_t)(p.tiles * p.splits), p.rank_blocks, p.turns), block(256);
    if (g.rank <= 16) hipLaunchKernelGGL((k_adapters_down_many<T, 1>), grid, block, 0, stream, g);
    else if (g.rank <= 32) hipLaunchKernelGGL((k_adapters_down_many<T, 2>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_adapters_down_many<T, 4>), grid, block, 0, stream, g);
}

template <int T, int YT>
void launch_up(const AdapterArgs &g, const AdapterPlan &p, hipStream_t stream)
{
    const dim3 grid((uint32_t)(p.up_tiles * p.row_blocks), 1, p.turns), block(256);
    // past the caches where y does not stay in them; us through them and past
    // them, MiB of y: 64 60 and 65, 112 71 both, 128 83.6 and 82.9, 224 142 and 137
    const bool large = g.m * g.rows * type_bytes(YT) > (128ull << 20);
    if (p.up_tile == 128 && g.rank <= 32) {
        if (large) hipLaunchKernelGGL((k_adapters_up_many<T, YT, 1, true>), grid, block, 0, stream, g);
        else hipLaunchKernelGGL((k_adapters_up_many<T, YT, 1, false>), grid, block, 0, stream, g);
    } else if (p.up_tile == 128) {
        if (large) hipLaunchKernelGGL((k_adapters_up_many<T, YT, 2, true>), grid, block, 0, stream, g);
        else hipLaunchKernelGGL((k_adapters_up_many<T, YT, 2, false>), grid, block, 0, stream, g);
    }
    else if (g.rank <= 32) hipLaunchKernelGGL((k_adapters_up<T, YT, 1, false>), grid, block, 0, stream, g);
    else if (g.rank <= 64) hipLaunchKernelGGL((k_adapters_up<T, YT, 2, false>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_adapters_up<T, YT, 2, true>), grid, block, 0, stream, g);
}

template <int T, int YT>
void launch_few(const AdapterArgs &g, const AdapterPlan &p, hipStream_t stream)
{
    const dim3 grid((uint32_t)(ceil_div(p.tiles * p.turns, 8) * 8 * p.row_blocks)), block(1024);
    if (g.rank <= 16) hipLaunchKernelGGL((k_adapters_few<T, YT, 1>), grid, block, 0, stream, g);
    else if (g.rank <= 32) hipLaunchKernelGGL((k_adapters_few<T, YT, 2>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_adapters_few<T, YT, 4>), grid, block, 0, stream, g);
}

template <int T, int YT>
wc_status launch_adapters(const AdapterArgs &g, const AdapterPlan &p, hipStream_t stream)
{
    if (p.few) {
        launch_few<T, YT>(g, p, stream);
    } else {
        if (p.tile == 128) launch_down_many<T>(g, p, stream);
        else launch_down<T>(g, p, stream);
        if (p.terms)
            hipLaunchKernelGGL(k_adapters_terms<T>, dim3((uint32_t)ceil_div(g.m * p.rank_blocks, 32)), dim3(256),
                               0, stream, g);
        launch_up<T, YT>(g, p, stream);
    }
    return launched();
}

template <int T>
wc_status launch_adapters(const AdapterArgs &g, const AdapterPlan &p, uint32_t y_type, hipStream_t stream)
{
    return y_type == WC_T_FP32 ? launch_adapters<T, WC_T_FP32>(g, p, stream) : launch_adapters<T, T>(g, p, stream);
}

// Launch shapes and scratch of the mixture-of-experts layer.
struct MoePlan {
    bool one;       // k_moe_route_one
    bool split;     // k_moe_down with four waves for 16 columns
    uint32_t route_tiles, route_splits, route_steps, experts_pad, slots, up_tiles, down_tiles;
    uint64_t logits, ids, weights, most, h, part, bytes;  // offsets in the scratch
};

MoePlan moe_plan(uint32_t m, uint32_t experts, uint32_t top_k, uint32_t cols, uint32_t inner)
{
    MoePlan p{};
    p.route_tiles = (experts + 15) / 16;
    p.experts_pad = 16 * p.route_tiles;
    // one launch for the router where one compute unit reads it in the time of
    // a second launch: 64 KiB take 6 us, 256 KiB 13 us against 3 + 3 us in two
    p.one = (uint64_t)experts * cols * 2 <= (64u << 10) && experts <= 256;
    const uint32_t steps = (cols + 31) / 32;
    uint32_t splits = 128 / p.route_tiles;
    const uint32_t most = (steps + 7) / 8;  // two steps for each of a block's waves
    if (splits > most) splits = most;
    if (splits > kMoeRouteSplits) splits = kMoeRouteSplits;
    if (splits < 1) splits = 1;
    p.route_steps = (uint32_t)(ceil_div(ceil_div(steps, splits), 8) * 8);
    p.route_splits = (uint32_t)ceil_div(steps, p.route_steps);
    p.slots = m * top_k < experts ? m * top_k : experts;
    p.up_tiles = (inner + 15) / 16;
    // a wave for twice 16 rows of W2, or four where that gives too few blocks.
    // us of a layer with one and with four, BF16, blocks of one: 256 (13 tokens
    // on 8 experts of 4096 x 14336) 469 and 426; 512 (16 tokens, 32 of 2048 x
    // 2048) 160 and 147, but (64 tokens, 32 of 2048 x 1024) 95 and 103; 1024 (64
    // of 2048 x 1024) 162 and 183; 2048 (64 of 4096 x 1536) 400 and 447
    p.split = (uint64_t)p.slots * ceil_div(cols, 128) < 4 * kCus;
    p.down_tiles = (uint32_t)ceil_div(cols, p.split ? 32 : 128);
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at = ceil_div(at + bytes, 256) * 256;
        return here;
    };
    p.logits = take(p.one ? 0 : 4ull * p.route_splits * m * p.experts_pad);
    p.ids = take(4ull * m * top_k);
    p.weights = take(4ull * m * top_k);
    p.most = take(4ull * m * top_k);
    p.h = take(4ull * m * top_k * inner);
    p.part = take(4ull * m * top_k * cols);
    p.bytes = at;
    return p;
}

bool valid_moe(uint64_t m, uint32_t experts, uint32_t top_k, uint32_t cols, uint32_t inner)
{
    return m <= kMoeMaxTokens && experts >= 1 && experts <= kMoeMaxExperts && top_k >= 1 && top_k <= kMoeMaxTop &&
           top_k <= experts && cols >= 8 && cols % 8 == 0 && cols <= (1u << 20) && inner >= 8 && inner % 8 == 0 &&
           inner <= (1u << 20) && (m * top_k < experts ? m * top_k : experts) * ((inner + 15) / 16) <= max_blocks(256);
}

template <int T, int TT>
wc_status launch_moe(const MoeArgs &g, const MoePlan &p, hipStream_t stream)
{
    const dim3 tokens(g.m);
    if (p.one) {
        if (g.experts <= 64) hipLaunchKernelGGL((k_moe_route_one<T, 1>), tokens, dim3(1024), 0, stream, g);
        else hipLaunchKernelGGL((k_moe_route_one<T, 4>), tokens, dim3(1024), 0, stream, g);
    } else {
        hipLaunchKernelGGL((k_moe_route<T, TT>), dim3(p.route_tiles * p.route_splits), dim3(256), 0, stream, g);
        if (g.experts <= 64) hipLaunchKernelGGL(k_moe_select<1>, tokens, dim3(64), 0, stream, g);
        else if (g.experts <= 256) hipLaunchKernelGGL(k_moe_select<4>, tokens, dim3(64), 0, stream, g);
        else hipLaunchKernelGGL(k_moe_select<16>, tokens, dim3(64), 0, stream, g);
    }
    if (g.m == 1) {
        hipLaunchKernelGGL(k_moe_up_one<T>, dim3((uint32_t)(g.top_k * p.up_tiles)), dim3(256), 0, stream, g);
        hipLaunchKernelGGL(k_moe_down_one<T>, dim3(g.cols / 8), dim3(1024), 0, stream, g);
        return launched();
    }
    hipLaunchKernelGGL((k_moe_up<T, TT>), dim3(p.slots * p.up_tiles), dim3(256), 0, stream, g);
    const dim3 down(p.slots * p.down_tiles);
    if (p.split) hipLaunchKernelGGL((k_moe_down<T, TT, true>), down, dim3(256), 0, stream, g);
    else hipLaunchKernelGGL((k_moe_down<T, TT, false>), down, dim3(256), 0, stream, g);
    hipLaunchKernelGGL(k_moe_join<T>, dim3((g.m * (g.cols / 4) + 63) / 64), dim3(64), 0, stream, g);
    return launched();
}

template <int T>
wc_status launch_moe_tiles(const MoeArgs &g, const MoePlan &p, hipStream_t stream)
{
    if (g.m <= 16) return launch_moe<T, 1>(g, p, stream);
    if (g.m <= 32) return launch_moe<T, 2>(g, p, stream);
    return launch_moe<T, 4>(g, p, stream);
}

}  // namespace

extern "C" {

uint64_t wc_token_logprobs_scratch(uint64_t m, uint32_t vocab, uint32_t top)
{
    if (m == 0 || m > kMaxRows || vocab == 0 || vocab > kMaxVocab || top > kMaxTop) return 0;
    return logprob_scratch(m, vocab, top);
}

wc_status wc_token_logprobs(const wc_logprobs *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err,
                            hipStream_t stream)
{
    if (!a || !valid_type(a->type) || a->vocab == 0 || a->vocab > kMaxVocab || a->top > kMaxTop || a->top > a->vocab)
        return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (a->m > kMaxRows || (a->m > 1 && a->stride < a->vocab)) return WC_ERR_ARG;
    if (!a->logits || !aligned(a->logits, type_bytes(a->type)) || !a->tokens || !aligned(a->tokens, 8))
        return WC_ERR_ARG;
    if (!a->logprob || !a->entropy || !a->lse || !aligned(a->logprob, 4) || !aligned(a->entropy, 4) ||
        !aligned(a->lse, 4))
        return WC_ERR_ARG;
    if (a->top && (!a->top_logprobs || !a->top_ids || !aligned(a->top_logprobs, 4) || !aligned(a->top_ids, 8)))
        return WC_ERR_ARG;
    LogprobArgs g{};
    logprob_slices(a->vocab, &g.slices, &g.slice);
    const uint64_t need = logprob_scratch(a->m, a->vocab, a->top);
    if (scratch_bytes < need) return WC_ERR_CAPACITY;
    if (need && (!d_scratch || !aligned(d_scratch, 16))) return WC_ERR_ARG;
    g.logits = a->logits;
    g.stride = a->stride;
    g.tokens = a->tokens;
    g.vocab = a->vocab;
    g.top = a->top;
    g.logprob = a->logprob;
    g.entropy = a->entropy;
    g.lse = a->lse;
    g.top_logprobs = a->top_logprobs;
    g.top_ids = a->top_ids;
    g.part = static_cast<float *>(d_scratch);
    g.part_top = need ? reinterpret_cast<uint64_t *>(static_cast<char *>(d_scratch) + 16 * a->m * g.slices) : nullptr;
    g.err = d_err;
    switch (a->type) {
    case WC_T_BF16: return launch_logprobs<WC_T_BF16>(g, a->m, stream);
    case WC_T_FP16: return launch_logprobs<WC_T_FP16>(g, a->m, stream);
    default: return launch_logprobs<WC_T_FP32>(g, a->m, stream);
    }
}

wc_status wc_token_logprobs_backward(const wc_logprobs_grad *a, uint32_t *d_err, hipStream_t stream)
{
    if (!a || !valid_type(a->type) || a->vocab == 0 || a->vocab > kMaxVocab) return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (a->m > kMaxRows || (a->m > 1 && (a->stride < a->vocab || a->out_stride < a->vocab))) return WC_ERR_ARG;
    const uintptr_t es = type_bytes(a->type);
    if (!a->logits || !a->out || !aligned(a->logits, es) || !aligned(a->out, es)) return WC_ERR_ARG;
    if (!a->tokens || !aligned(a->tokens, 8) || !a->lse || !aligned(a->lse, 4)) return WC_ERR_ARG;
    if (!aligned(a->grad_logprob, 4) || !aligned(a->grad_entropy, 4)) return WC_ERR_ARG;
    if (a->grad_entropy && (!a->entropy || !aligned(a->entropy, 4))) return WC_ERR_ARG;
    if ((a->out != a->logits || (a->m > 1 && a->out_stride != a->stride)) &&
        !rows_apart(a->logits, es * a->stride, es * a->vocab, a->out, es * a->out_stride, es * a->vocab, a->m))
        return WC_ERR_ARG;
    LogprobGradArgs g{};
    g.logits = a->logits;
    g.out = a->out;
    g.stride = a->stride;
    g.out_stride = a->out_stride;
    g.tokens = a->tokens;
    g.lse = a->lse;
    g.entropy = a->entropy;
    g.grad_logprob = a->grad_logprob;
    g.grad_entropy = a->grad_entropy;
    g.vocab = a->vocab;
    g.blocks = a->out == a->logits ? 1 : (uint32_t)ceil_div(a->vocab, kGradThreads * kBatch);
    g.err = d_err;
    switch (a->type) {
    case WC_T_BF16: launch_grad<WC_T_BF16>(g, a->m, stream); break;
    case WC_T_FP16: launch_grad<WC_T_FP16>(g, a->m, stream); break;
    default: launch_grad<WC_T_FP32>(g, a->m, stream); break;
    }
    return launched();
}

uint64_t wc_add_adapters_scratch(uint64_t m, uint32_t rank, uint32_t cols, uint32_t rows)
{
    if (m == 0 || !valid_adapters(m, rank, cols, rows)) return 0;
    // enough for either plan: the adapters' number is not known here
    if (m > kMaxTokens) m = kMaxTokens;
    const uint64_t small = adapter_plan(m, 0, rank, cols, rows, false).scratch;
    const uint64_t large = many_tokens(m, 1) ? adapter_plan(m, 0, rank, cols, rows, true).scratch : 0;
    return small > large ? small : large;
}

wc_status wc_add_adapters(const wc_adapters *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err,
                          hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16) || (a->y_type != a->type && a->y_type != WC_T_FP32))
        return WC_ERR_ARG;
    if (!valid_adapters(a->m, a->rank, a->cols, a->rows) || a->n > 0x7FFFFFFFu) return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (a->n && (!a->a || !aligned(a->a, 16) || !a->b || !aligned(a->b, 2))) return WC_ERR_ARG;
    if (!a->x || !aligned(a->x, 16) || (a->m > 1 && (a->x_stride < a->cols || a->x_stride % 8))) return WC_ERR_ARG;
    if (!a->y || !aligned(a->y, type_bytes(a->y_type)) || (a->m > 1 && a->y_stride < a->rows)) return WC_ERR_ARG;
    if (!a->ids || !aligned(a->ids, 8) || !aligned(a->scales, 4)) return WC_ERR_ARG;
    auto plan = [&](uint64_t m) { return adapter_plan(m, a->n, a->rank, a->cols, a->rows, many_tokens(m, a->n)); };
    AdapterPlan p = plan(a->m < kMaxTokens ? a->m : kMaxTokens);
    if (scratch_bytes < p.scratch) return WC_ERR_CAPACITY;
    if (p.scratch && (!d_scratch || !aligned(d_scratch, 16))) return WC_ERR_ARG;
    const uint64_t yb = type_bytes(a->y_type);
    // a block may read x where another has written y
    if (!rows_apart(a->x, 2 * a->x_stride, 2ull * a->cols, a->y, yb * a->y_stride, yb * a->rows, a->m)) return WC_ERR_ARG;
    wc_status status = WC_OK;
    for (uint64_t t = 0; t < a->m && status == WC_OK; t += kMaxTokens) {
        const uint64_t m = a->m - t < kMaxTokens ? a->m - t : kMaxTokens;
        if (t && m < kMaxTokens) p = plan(m);  // the last: its scratch is smaller, also with columns in 8 parts
        AdapterArgs g{};
        g.x = static_cast<const uint16_t *>(a->x) + t * a->x_stride;
        g.x_stride = a->x_stride;
        g.y = static_cast<char *>(a->y) + t * a->y_stride * yb;
        g.y_stride = a->y_stride;
        g.a = static_cast<const uint16_t *>(a->a);
        g.b = static_cast<const uint16_t *>(a->b);
        g.ids = a->ids + t;
        g.scales = a->scales;
        g.m = m;
        g.n = a->n;
        g.rank = a->rank;
        g.cols = a->cols;
        g.rows = a->rows;
        g.part = static_cast<float *>(d_scratch);
        g.u = reinterpret_cast<uint16_t *>(static_cast<char *>(d_scratch) + p.u);
        g.unscale = reinterpret_cast<float *>(static_cast<char *>(d_scratch) + p.unscale);
        g.rank_pad = p.rank_pad;
        g.splits = p.splits;
        g.split_cols = p.split_cols;
        g.row_block = p.row_block;
        g.err = d_err;
        status = a->type == WC_T_BF16 ? launch_adapters<WC_T_BF16>(g, p, a->y_type, stream)
                                      : launch_adapters<WC_T_FP16>(g, p, a->y_type, stream);
    }
    return status;
}

uint64_t wc_moe_layer_scratch(uint64_t m, uint32_t experts, uint32_t top_k, uint32_t cols, uint32_t inner)
{
    if (m == 0 || !valid_moe(m, experts, top_k, cols, inner)) return 0;
    return moe_plan((uint32_t)m, experts, top_k, cols, inner).bytes;
}

wc_status wc_moe_layer(const wc_moe *a, void *d_scratch, uint64_t scratch_bytes, hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16)) return WC_ERR_ARG;
    if (!valid_moe(a->m, a->experts, a->top_k, a->cols, a->inner)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (!a->x || !aligned(a->x, 16) || (a->m > 1 && (a->x_stride < a->cols || a->x_stride % 8))) return WC_ERR_ARG;
    if (!a->router || !aligned(a->router, 16)) return WC_ERR_ARG;
    if (!a->w1 || !a->w3 || !a->w2 || !aligned(a->w1, 16) || !aligned(a->w3, 16) || !aligned(a->w2, 16))
        return WC_ERR_ARG;
    if (a->up_row < a->cols || a->up_row % 8 || a->up_expert % 8 || a->down_row < a->inner || a->down_row % 8 ||
        a->down_expert % 8 || a->up_row > (1u << 26) || a->down_row > (1u << 26))
        return WC_ERR_ARG;
    if (!a->out || !aligned(a->out, 2) || (a->m > 1 && a->out_stride < a->cols)) return WC_ERR_ARG;
    const MoePlan p = moe_plan((uint32_t)a->m, a->experts, a->top_k, a->cols, a->inner);
    if (scratch_bytes < p.bytes) return WC_ERR_CAPACITY;
    if (!d_scratch || !aligned(d_scratch, 256)) return WC_ERR_ARG;
    char *s = static_cast<char *>(d_scratch);
    MoeArgs g{};
    g.x = static_cast<const uint16_t *>(a->x);
    g.router = static_cast<const uint16_t *>(a->router);
    g.w1 = static_cast<const uint16_t *>(a->w1);
    g.w3 = static_cast<const uint16_t *>(a->w3);
    g.w2 = static_cast<const uint16_t *>(a->w2);
    g.x_stride = a->x_stride;
    g.up_expert = a->up_expert;
    g.up_row = a->up_row;
    g.down_expert = a->down_expert;
    g.down_row = a->down_row;
    g.out = static_cast<uint16_t *>(a->out);
    g.out_stride = a->out_stride;
    g.m = (uint32_t)a->m;
    g.experts = a->experts;
    g.top_k = a->top_k;
    g.cols = a->cols;
    g.inner = a->inner;
    g.renormalize = a->renormalize;
    g.logits = reinterpret_cast<float *>(s + p.logits);
    g.ids = reinterpret_cast<int32_t *>(s + p.ids);
    g.weights = reinterpret_cast<float *>(s + p.weights);
    g.most = reinterpret_cast<uint32_t *>(s + p.most);
    g.h = reinterpret_cast<float *>(s + p.h);
    g.part = reinterpret_cast<float *>(s + p.part);
    g.experts_pad = p.experts_pad;
    g.route_splits = p.route_splits;
    g.route_steps = p.route_steps;
    g.slots = p.slots;
    return a->type == WC_T_BF16 ? launch_moe_tiles<WC_T_BF16>(g, p, stream)
                                : launch_moe_tiles<WC_T_FP16>(g, p, stream);
}

}  // extern "C"

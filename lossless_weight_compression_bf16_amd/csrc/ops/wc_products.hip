// wc_products.hip -- C ABI of the products of a training step beside the
// compressed weights (see include/wc.h): products grouped by expert, cross
// entropy from hidden states, and their gradients.  Argument checks, launch
// shapes and scratch layout; like the other calls these only enqueue on the
// caller's stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "wc.h"
#include "ops_common.hpp"
#include "ops_grouped.hpp"
#include "ops_host.hpp"
#include "ops_loss.hpp"

using namespace wc::ops;

namespace {

// Rows that a tile's window can hold: 256 of them below 2^31 bytes.
constexpr uint64_t kMaxPitch = (1ull << 22) - 8;
constexpr uint32_t kMaxCols = 1u << 20;

// Tiles of a product, and the parts of k that it is split into.
enum TileSize { kFlat, kSmall, kLarge };  // 64 rows (by 256 columns, or 128 with P across), 128 x 128, 256 x 256
struct TilePlan {
    TileSize size;
    uint32_t splits;
};

// The tile and the parts of k with the least time, of `tiles` (of 256, of 128)
// with `stages` of k each.  What a compute unit takes for a stage, and for the
// beginning and the end of a tile: one large tile 1.5 and 10 us, two small ones
// 1.1 and 5, a single small one 0.75 and 3.5.  Parts are summed in fp32 by
// another launch.  (Small and large tiles: 32768 rows of 256 experts of 2048 x 7168, of which
// a large tile is half empty, 2040 and 1870 us; both gradients of 16384 rows of 8 experts of
// 14336 x 4096, 3700 and 3065.  128 x 256 for the former: 2090.)
TilePlan tile_plan(uint64_t large, uint64_t small, uint64_t stages, uint64_t results, bool joined, uint32_t most = 64)
{
    TilePlan best{kSmall, 1};
    double least = 1e30;
    for (int size = 0; size < 2; size++) {
        for (uint32_t s = 1; s <= most && (s == 1 || stages >= 4 * s); s *= 2) {
            const double tiles = (double)(size ? large : small) * s, each = (double)ceil_div(stages, s);
            const bool single = !size && tiles <= kCus;
            const double rounds = size ? ceil(tiles / kCus) : single ? 1.0 : ceil(tiles / (2 * kCus));
            double t = rounds * (size ? 1.5 * each + 10 : single ? 0.75 * each + 3.5 : 1.1 * each + 5);
            if (s > 1) t += (joined ? 0.0 : 5.0) + (double)results * s * 8 / 4e6;
            if (t < least) {
                least = t;
                best = {size ? kLarge : kSmall, s};
            }
        }
    }
    return best;
}

// ------------------------------------------------------------- grouped by expert

uint64_t tiles_of(uint64_t m, uint32_t experts, uint64_t tile)  // the most there can be
{
    return m / tile + (m < experts ? m : experts);
}
uint64_t tiles_expected(uint64_t m, uint32_t experts, uint64_t tile)  // with the rows dealt evenly
{
    const uint64_t hit = m < experts ? m : experts;
    return hit * ceil_div(ceil_div(m, hit), tile);
}

// Tiles of 64 rows read the weights as fast as memory gives them, where there are enough of them; below that smaller ones
// use more of the compute units.  us by tiles of 64 and of 128, 17 to 64 rows of a vocabulary of 128256 x 4096 160 and 180, of
// 100000 x 768 34 to 37 and 43 to 45, of 32768 x 2048 45 and 35, of 50257 x 768 25 and 22; 9 to 64 rows of each of 8 experts of
// 14336 x 4096 145 to 157 and 165 to 180 (dx 149 to 168 and 166 to 181), of 64 of 1024 x 2048 51 to 63 and 69 to 74 (dx 53 to 61 and
// 64 to 70), of 8 of 2048 x 4096 32 to 41 and 28 to 35; 65 to 128 rows of each of 8 of 14336 x 4096 340 to 250 and 180 to 203.
bool flat(uint64_t rows, uint64_t weights) { return rows <= 64 && weights > 1ull << 26; }

// The tiles of y of m rows with n columns each, from k, or of dx (across), whose tiles of 64 rows have 128 columns and are more
// where k is over 1024.  us by them and by tiles of 128, 64 rows of each expert, dx of 2048 columns from k = 768, 1032, 1536 and 4096:
// one expert 12.4, 13.5, 13.4 and 15.9, and 11.0, 13.0, 13.7 and 19.9; 4 experts 12.9, 15.3, 16.7 and 28.6, and 12.8, 17.9, 18.9 and
// 28.2; 16 experts 14.9, 27.5, 30.5 and 63, and 16.7, 28.8, 33.5 and 63.  Over 1 to 16 experts, 9 to 64 rows and 768 or 2048
// columns they take 4% less on average from k over 1024 (6% more to 20% less), up to there
// 1% less (15% more to 23% less).
TileSize grouped_size(uint64_t m, uint32_t experts, uint32_t n, uint32_t k, bool across)
{
    const uint64_t hit = m < experts ? m : experts, rows = ceil_div(m, hit);
    if (flat(rows, hit * n * k) || (across && rows <= 64 && k > 1024)) return kFlat;
    return tile_plan(tiles_expected(m, experts, 256) * ceil_div(n, 256), tiles_expected(m, experts, 128) * ceil_div(n, 128),
                     ceil_div(k, kTileK), m * n, true, 1)
        .size;
}
// Room for the tiles of the last round in parts, one for every slot, where that
// round is more than a sixth of the time.
uint64_t grouped_part(TileSize size, uint64_t m, uint32_t experts, uint32_t n, uint32_t k, uint32_t flat_n)
{
    const uint64_t bm = size == kLarge ? 256 : size == kSmall ? 128 : 64, bn = size == kFlat ? flat_n : bm;
    const uint64_t slots = kCus * (size == kLarge ? 1 : 2);
    const bool few = tiles_expected(m, experts, bm) * ceil_div(n, bn) < 6 * slots;
    return few && k >= 16 * kTileK ? 4 * bm * bn * slots : 0;
}

// Few rows of each expert, whose weights are few: no tile, but more and smaller blocks.  us by
// k_grouped_few and by tiles.  k over 1024: one row of 1024 x 2048 11 and 15, of each of 8 and 16 such experts 11.8 and 15.7,
// 23 and 17.6; one row of 14336 x 4096 41 and 25, of each of 2 and 8 of 2048 x 7168 18 and 20.5, 55 and 45.  k up to 1024, 8 rows
// (one row) of each of 32 experts of 2048 x 512 14.7 and 15.9 (14.3 and 15.8), of 2048 x 1024 24 and 29.5 (26 and 29), of 4096 x 1024
// 53 and 45 (56 and 45); of 64 of 4096 x 256 28 and 37 (35 and 36), of 8192 x 256 55 and 50 (68 and 47); of 256 of 768 x 256 25 and 30
// (30 and 29), of 2048 x 256 63 and 54 (77 and 52), of 2048 x 768 149 and 135 (139 and 129).  From 2^26 weights on the
// tiles are of 64 rows past the caches; up to there few rows gain by 14 to 21% on average, one by 2%.
bool grouped_few(uint64_t m, uint32_t experts, uint32_t n, uint32_t k)
{
    const uint64_t hit = m < experts ? m : experts;
    return m <= 8 * hit && hit * n * k <= (k <= 1024 ? 1ull << 26 : (1ull << 25) - 1);
}

TilePlan grouped_dw_plan(uint64_t m, uint32_t experts, uint32_t n, uint32_t k)
{
    const uint64_t hit = m < experts ? (m ? m : 1) : experts;
    return tile_plan(experts * ceil_div(n, 256) * ceil_div(k, 256), experts * ceil_div(n, 128) * ceil_div(k, 128),
                     ceil_div(ceil_div(m, hit), kTileK), (uint64_t)experts * n * k, false);
}

uint64_t part_bytes(uint64_t results, uint32_t splits) { return splits > 1 ? 4 * results * splits : 0; }

bool valid_grouped(uint64_t m, uint32_t experts, uint32_t rows, uint32_t cols)
{
    if (m > kMaxRows || experts < 1 || experts > kGroupedMaxExperts || rows < 8 || rows % 8 || rows > kMaxCols || cols < 8 ||
        cols % 8 || cols > kMaxCols)
        return false;
    const uint64_t most = max_blocks(256) / 16 - 8, wide = rows > cols ? rows : cols;
    return (m / 128 + experts) * ceil_div(wide, 32) <= most && experts * ceil_div(rows, 128) * ceil_div(cols, 128) <= most;
}

void launch_join(int type, const JoinArgs &g, hipStream_t stream)
{
    const uint64_t fours = ceil_div(g.rows * (g.cols / 4), 256), blocks = fours < max_blocks(256) ? fours : max_blocks(256);
    if (!blocks) return;
    if (type == WC_T_BF16) hipLaunchKernelGGL(k_join<WC_T_BF16>, dim3((uint32_t)blocks), dim3(256), 0, stream, g);
    else hipLaunchKernelGGL(k_join<WC_T_FP16>, dim3((uint32_t)blocks), dim3(256), 0, stream, g);
}

uint32_t xcd_grid(uint64_t pieces) { return (uint32_t)(8 * ceil_div(pieces, 8)); }
// Blocks of a kernel that takes one large tile after the other.
uint32_t large_grid(uint64_t pieces) { return xcd_grid(pieces < kCus ? pieces : kCus); }

// A block's four waves on the same rows of weights, or each on its own.  us of 2 to 16 rows, a vocabulary of 128256 x 4096: 157 to 160
// and 166 to 174; of 50257 x 768 22 to 23 and 19 to 20; one row of each of 8 experts of 1024 x 2048 11.8 and 19.6.
bool few_split(uint32_t k) { return k > 1024; }

constexpr int kFlatAlong = 256, kFlatAcross = 128;  // columns of the flat tiles

// y, or dx (kPAlong false), by tiles of BM x BN
template <int T, int BM, int BN, bool kPAlong>
void launch_tiles(const GroupedArgs &g, hipStream_t stream)
{
    constexpr uint32_t slots = GroupedPieces<BM, BN>::kSlots;
    // rows behind the last expert's fill a tile more, and may take one that the experts' would have
    const uint64_t tiles = (tiles_of(g.m, g.experts, BM) + 1) * ceil_div(g.n, BN);
    // a last round in parts has no more blocks than slots; the XCDs' ranges of parts and zeros are rounded up
    const uint64_t pieces = tiles + (g.part ? slots : 0) + 16;
    const uint32_t blocks = BM == 256 ? large_grid(pieces) : xcd_grid(pieces);
    hipLaunchKernelGGL((k_grouped<T, BM, BN, kPAlong>), dim3(blocks), dim3(256), 0, stream, g);
    if (g.part) hipLaunchKernelGGL((k_grouped_join<T, BM, BN>), dim3(slots / 2 * 8), dim3(256), 0, stream, g);
}
template <int T, bool kPAlong>
void launch_grouped(GroupedArgs g, TileSize size, hipStream_t stream)
{
    if (size == kLarge) launch_tiles<T, 256, 256, kPAlong>(g, stream);
    else if (size == kSmall) launch_tiles<T, 128, 128, kPAlong>(g, stream);
    else launch_tiles<T, 64, kPAlong ? kFlatAlong : kFlatAcross, kPAlong>(g, stream);
}

template <int T>
wc_status launch_grouped_linear(GroupedArgs g, hipStream_t stream)
{
    if (grouped_few(g.m, g.experts, g.n, g.k)) {
        const bool split = few_split(g.k);
        g.slots = (g.m < g.experts ? g.m : g.experts) + (g.zero_rest ? 1 : 0);
        const dim3 grid((uint32_t)(g.slots * ceil_div(g.n, split ? 32 : 128)));
        if (split) hipLaunchKernelGGL((k_grouped_few<T, true>), grid, dim3(256), 0, stream, g);
        else hipLaunchKernelGGL((k_grouped_few<T, false>), grid, dim3(256), 0, stream, g);
    } else {
        launch_grouped<T, true>(g, grouped_size(g.m, g.experts, g.n, g.k, false), stream);
    }
    return launched();
}

// No rows: all there is to do is to look at the ends, if they are to be looked at.
wc_status launch_ends(const int64_t *ends, uint32_t experts, uint32_t *err, hipStream_t stream)
{
    if (!err) return WC_OK;
    if (!ends || !aligned(ends, 8)) return WC_ERR_ARG;
    hipLaunchKernelGGL(k_grouped_ends, dim3(1), dim3(256), 0, stream, ends, experts, err);
    return launched();
}

template <int T>
void launch_grouped_dw(GroupedDwArgs g, const TilePlan &p, hipStream_t stream)
{
    g.splits = p.splits;
    const uint64_t tile = p.size == kLarge ? 256 : 128;
    const uint64_t pieces = g.experts * xcd_grid(ceil_div(g.n, tile) * ceil_div(g.k, tile) * g.splits);
    const dim3 grid(p.size == kLarge ? large_grid(pieces) : (uint32_t)pieces), block(256);
    if (p.size == kLarge) hipLaunchKernelGGL((k_grouped_dw<T, 256, 256>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_grouped_dw<T, 128, 128>), grid, block, 0, stream, g);
    if (g.splits > 1)
        launch_join(T, JoinArgs{g.part, g.dw, g.k, (uint64_t)g.experts * g.n, g.k, g.splits, nullptr}, stream);
}

// ------------------------------------------------------------- cross entropy

constexpr uint64_t kLossMaxRows = 1ull << 19;
constexpr uint32_t kLossSlice = 1u << 15;  // rows of one set of launches of the forward pass
// G of a piece of the vocabulary, all terms of it: at most 2^27 numbers, 256 MiB, what the last cache holds, or 256 columns.  ms with pieces of 2^25,
// 2^26, 2^27, 2^28 and 2^30: 4096 rows, 128256 x 4096, 16.4, 16.2, 16.3, 16.5 and 16.6 (rounded 10.3, 9.7, 9.8, 9.9 and 9.9); 16384
// rows, 32000 x 2048, 12.4, 10.1, 9.3, 9.0 and 8.9; 65536 rows, 16384 x 1024, whose pieces are of 256 to 8192 columns
// and whose sums of dH are read and written for each, 24.4, 16.1, 12.6, 11.1 and 10.3: what more scratch would give, and many rows pay.
constexpr uint64_t kLossPiece = 1ull << 27;

bool valid_loss(uint64_t m, uint32_t vocab, uint32_t cols)
{
    return m <= kLossMaxRows && vocab >= 1 && vocab <= (1u << 22) && cols >= 8 && cols % 8 == 0 && cols <= kMaxCols;
}

// us by k_loss_few and by tiles: 12 and 16 rows of a vocabulary of 50257 x 768 20 and 25 (32 rows 26 and 25), of 128256 x
// 4096 156 to 160 and 160 (32 rows 212 and 160)
bool loss_few(uint64_t m) { return m <= kLossFew; }
TileSize loss_tile(uint64_t m, uint32_t vocab, uint32_t k)
{
    if (flat(m, (uint64_t)vocab * k)) return kFlat;
    return tile_plan(ceil_div(m, 256) * ceil_div(vocab, 256), ceil_div(m, 128) * ceil_div(vocab, 128), ceil_div(k, kTileK), 0, true, 1).size;
}
uint32_t loss_parts(uint64_t m, uint32_t vocab, uint32_t k)
{
    return (uint32_t)ceil_div(vocab, loss_few(m) ? (few_split(k) ? 32 : 128) : loss_tile(m, vocab, k) == kSmall ? 128 : 256);
}
uint64_t up256(uint64_t n) { return ceil_div(n, 256) * 256; }

template <int T>
void launch_loss(const LossArgs &g, hipStream_t stream)
{
    if (loss_few(g.m)) {
        const bool split = few_split(g.k);
        const dim3 grid((uint32_t)ceil_div(g.vocab, split ? 32 : 128));
        if (split) hipLaunchKernelGGL((k_loss_few<T, true>), grid, dim3(256), 0, stream, g);
        else hipLaunchKernelGGL((k_loss_few<T, false>), grid, dim3(256), 0, stream, g);
    } else {
        const TileSize size = loss_tile(g.m, g.vocab, g.k);
        const uint64_t tiles = ceil_div(g.m, size == kLarge ? 256 : size == kSmall ? 128 : 64) * g.parts;
        const dim3 grid(size == kLarge ? large_grid(tiles) : xcd_grid(tiles)), block(256);
        if (size == kLarge) hipLaunchKernelGGL((k_loss<T, 256, 256>), grid, block, 0, stream, g);
        else if (size == kSmall) hipLaunchKernelGGL((k_loss<T, 128, 128>), grid, block, 0, stream, g);
        else hipLaunchKernelGGL((k_loss<T, 64, 256>), grid, block, 0, stream, g);
    }
    hipLaunchKernelGGL(k_loss_join, dim3(g.m), dim3(256), 0, stream, g);
}

struct LossGradPlan {
    uint32_t piece;          // columns of the vocabulary
    TilePlan dh, dw;
    uint64_t live, rows, most, grad, dh_part, dw_part, bytes;  // offsets in the scratch
    bool dh_sums;            // dH goes through fp32 sums
};

// terms: of G, each 16 bits
LossGradPlan loss_grad_plan(uint64_t m, uint32_t vocab, uint32_t k, uint32_t terms)
{
    LossGradPlan p{};
    uint64_t piece = kLossPiece / terms / m / 256 * 256;
    if (piece < 256) piece = 256;
    const uint64_t pieces = ceil_div(vocab, piece);
    p.piece = (uint32_t)(pieces == 1 ? vocab : ceil_div(ceil_div(vocab, pieces), 256) * 256);
    p.dh = tile_plan(ceil_div(m, 256) * ceil_div(k, 256), ceil_div(m, 128) * ceil_div(k, 128), terms * ceil_div(p.piece, kTileK),
                     m * k, pieces > 1);
    p.dw = tile_plan(ceil_div(p.piece, 256) * ceil_div(k, 256), ceil_div(p.piece, 128) * ceil_div(k, 128),
                     terms * ceil_div(m, kTileK), (uint64_t)p.piece * k, false);
    p.dh_sums = pieces > 1 || p.dh.splits > 1;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at = up256(at + bytes);
        return here;
    };
    p.rows = take(16 * m);
    p.most = take(4 * kLossRowBlocks);
    p.live = take(2 * m * k);
    p.grad = take(2 * terms * m * ((p.piece + 7) / 8 * 8));
    p.dh_part = take(p.dh_sums ? 4 * m * k * p.dh.splits : 0);
    p.dw_part = take(part_bytes((uint64_t)p.piece * k, p.dw.splits));
    p.bytes = at;
    return p;
}

template <int T, bool kQAlong, int kTerms>
void launch_product(const ProductArgs &g, bool large, hipStream_t stream)
{
    const uint64_t tile = large ? 256 : 128, tiles = ceil_div(g.m, tile) * ceil_div(g.n, tile) * g.splits;
    if (large) hipLaunchKernelGGL((k_product<T, 256, 256, kQAlong, kTerms>), dim3(large_grid(tiles)), dim3(256), 0, stream, g);
    else hipLaunchKernelGGL((k_product<T, 128, 128, kQAlong, kTerms>), dim3(xcd_grid(tiles)), dim3(256), 0, stream, g);
}
template <int T, int BM, int BN>
void launch_loss_grad_tiles(const LossGradArgs &g, hipStream_t stream)
{
    const uint64_t tiles = ceil_div(g.m, BM) * ceil_div(g.width, BN);
    const dim3 grid(BM == 256 ? large_grid(tiles) : xcd_grid(tiles)), block(256);
    if (g.again) hipLaunchKernelGGL((k_loss_grad<T, BM, BN, true>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_loss_grad<T, BM, BN, false>), grid, block, 0, stream, g);
}

template <int T>
void launch_loss_grad(const wc_linear_loss_grad &a, LossGradArgs g, const LossGradPlan &p, uint32_t terms, char *s,
                      hipStream_t stream)
{
    hipLaunchKernelGGL(k_loss_rows, dim3(kLossRowBlocks), dim3(256), 0, stream, g);
    float *dh_part = reinterpret_cast<float *>(s + p.dh_part), *dw_part = reinterpret_cast<float *>(s + p.dw_part);
    for (uint64_t v0 = 0; v0 < g.vocab; v0 += p.piece) {
        g.v0 = (uint32_t)v0;
        g.width = (uint32_t)(g.vocab - v0 < p.piece ? g.vocab - v0 : p.piece);
        g.pitch = (g.width + 7) / 8 * 8;
        g.again = terms > 1 ? (uint64_t)g.m * g.pitch : 0;
        if (loss_few(g.m)) {
            const bool split = few_split(g.k);
            const dim3 grid((uint32_t)ceil_div(g.width, split ? 32 : 128));
            if (split) hipLaunchKernelGGL((k_loss_grad_few<T, true>), grid, dim3(256), 0, stream, g);
            else hipLaunchKernelGGL((k_loss_grad_few<T, false>), grid, dim3(256), 0, stream, g);
        } else {
            const TileSize size = loss_tile(g.m, p.piece, g.k);
            if (size == kLarge) launch_loss_grad_tiles<T, 256, 256>(g, stream);
            else if (size == kSmall) launch_loss_grad_tiles<T, 128, 128>(g, stream);
            else launch_loss_grad_tiles<T, 64, 256>(g, stream);
        }
        if (a.grad_hidden) {
            ProductArgs d{g.grad, g.w + v0 * g.w_row, g.again, g.pitch, g.w_row, g.m, g.k, g.width, p.dh.splits,
                          p.dh_sums ? dh_part : nullptr, v0 ? 1u : 0u, static_cast<uint16_t *>(a.grad_hidden),
                          a.grad_hidden_stride, g.most};
            if (g.again) launch_product<T, true, 2>(d, p.dh.size == kLarge, stream);
            else launch_product<T, true, 1>(d, p.dh.size == kLarge, stream);
        }
        if (a.grad_weight) {
            uint16_t *out = static_cast<uint16_t *>(a.grad_weight) + v0 * g.k;
            ProductArgs d{g.grad, g.live, g.again, g.pitch, g.k, g.width, g.k, g.m, p.dw.splits,
                          p.dw.splits > 1 ? dw_part : nullptr, 0, out, g.k, g.most};
            if (g.again) launch_product<T, false, 2>(d, p.dw.size == kLarge, stream);
            else launch_product<T, false, 1>(d, p.dw.size == kLarge, stream);
            if (p.dw.splits > 1) launch_join(T, JoinArgs{dw_part, out, g.k, g.width, g.k, p.dw.splits, g.most}, stream);
        }
    }
    if (a.grad_hidden && p.dh_sums)
        launch_join(T, JoinArgs{dh_part, static_cast<uint16_t *>(a.grad_hidden), a.grad_hidden_stride, g.m, g.k, p.dh.splits,
                                g.most},
                    stream);
}

bool rows16(const void *p, uint64_t stride, uint64_t width) { return p && aligned(p, 16) && stride >= width && stride % 8 == 0 && stride <= kMaxPitch; }

}  // namespace

extern "C" {

uint64_t wc_grouped_linear_scratch(uint64_t m, uint32_t experts, uint32_t rows, uint32_t cols)
{
    if (m == 0 || !valid_grouped(m, experts, rows, cols) || grouped_few(m, experts, rows, cols)) return 0;
    return grouped_part(grouped_size(m, experts, rows, cols, false), m, experts, rows, cols, kFlatAlong);
}

wc_status wc_grouped_linear(const wc_grouped *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err, hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16) || !valid_grouped(a->m, a->experts, a->rows, a->cols))
        return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return launch_ends(a->ends, a->experts, d_err, stream);
    if (!rows16(a->x, a->x_stride, a->cols) || !rows16(a->w, a->w_row, a->cols) || a->w_expert % 8 ||
        !rows16(a->y, a->y_stride, a->rows) || !a->ends || !aligned(a->ends, 8))
        return WC_ERR_ARG;
    if (!rows_apart(a->x, 2 * a->x_stride, 2ull * a->cols, a->y, 2 * a->y_stride, 2ull * a->rows, a->m)) return WC_ERR_ARG;
    const uint64_t need = wc_grouped_linear_scratch(a->m, a->experts, a->rows, a->cols);
    if (scratch_bytes < need) return WC_ERR_CAPACITY;
    if (need && (!d_scratch || !aligned(d_scratch, 16))) return WC_ERR_ARG;
    if (!apart(rows_of(a->y, a->y_stride, a->rows, a->m), experts_of(a->w, a->w_expert, a->w_row, a->cols, a->rows, a->experts),
               line(a->ends, 8 * a->experts)))
        return WC_ERR_ARG;
    GroupedArgs g{};
    g.x = static_cast<const uint16_t *>(a->x);
    g.w = static_cast<const uint16_t *>(a->w);
    g.ends = a->ends;
    g.y = static_cast<uint16_t *>(a->y);
    g.x_stride = a->x_stride;
    g.w_expert = a->w_expert;
    g.y_stride = a->y_stride;
    g.w_row = (uint32_t)a->w_row;
    g.m = (uint32_t)a->m;
    g.experts = a->experts;
    g.n = a->rows;
    g.k = a->cols;
    g.zero_rest = a->zero_rest;
    g.part = need ? static_cast<float *>(d_scratch) : nullptr;
    g.err = d_err;
    return a->type == WC_T_BF16 ? launch_grouped_linear<WC_T_BF16>(g, stream) : launch_grouped_linear<WC_T_FP16>(g, stream);
}

uint64_t wc_grouped_linear_backward_scratch(uint64_t m, uint32_t experts, uint32_t rows, uint32_t cols)
{
    if (m == 0 || !valid_grouped(m, experts, rows, cols)) return 0;
    // one after the other
    const uint64_t dx = grouped_part(grouped_size(m, experts, cols, rows, true), m, experts, cols, rows, kFlatAcross);
    const uint64_t dw = part_bytes((uint64_t)experts * rows * cols, grouped_dw_plan(m, experts, rows, cols).splits);
    return dx > dw ? dx : dw;
}

wc_status wc_grouped_linear_backward(const wc_grouped_grad *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err,
                                     hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16) || !valid_grouped(a->m, a->experts, a->rows, a->cols))
        return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (!a->ends || !aligned(a->ends, 8) || (a->m && !rows16(a->grad, a->grad_stride, a->rows))) return WC_ERR_ARG;
    if (a->m && a->grad_x && (!rows16(a->w, a->w_row, a->cols) || a->w_expert % 8 || !rows16(a->grad_x, a->grad_x_stride, a->cols) ||
                              !rows_apart(a->grad, 2 * a->grad_stride, 2ull * a->rows, a->grad_x, 2 * a->grad_x_stride,
                                          2ull * a->cols, a->m)))
        return WC_ERR_ARG;
    if (a->grad_w && (!aligned(a->grad_w, 16) || (a->m && !rows16(a->x, a->x_stride, a->cols)))) return WC_ERR_ARG;
    const uint64_t need = wc_grouped_linear_backward_scratch(a->m, a->experts, a->rows, a->cols);
    if (scratch_bytes < need) return WC_ERR_CAPACITY;
    if (need && (!d_scratch || !aligned(d_scratch, 16))) return WC_ERR_ARG;
    // the gradient of x is written while w and the other results' inputs are still to be read, that of w after w
    const Rows ends = line(a->ends, 8 * a->experts), dw = line(a->grad_w, 2ull * a->experts * a->rows * a->cols);
    if (a->m && a->grad_x &&
        !apart(rows_of(a->grad_x, a->grad_x_stride, a->cols, a->m), ends, dw,
               experts_of(a->w, a->w_expert, a->w_row, a->cols, a->rows, a->experts),
               rows_of(a->grad_w ? a->x : nullptr, a->x_stride, a->cols, a->m)))
        return WC_ERR_ARG;
    if (!apart(dw, ends, rows_of(a->grad, a->grad_stride, a->rows, a->m), rows_of(a->x, a->x_stride, a->cols, a->m)))
        return WC_ERR_ARG;
    if (!a->m && !a->grad_w) return launch_ends(a->ends, a->experts, d_err, stream);
    if (!a->grad_x && !a->grad_w) return WC_OK;
    if (a->grad_x && a->m) {
        GroupedArgs g{};
        g.x = static_cast<const uint16_t *>(a->grad);
        g.w = static_cast<const uint16_t *>(a->w);
        g.ends = a->ends;
        g.y = static_cast<uint16_t *>(a->grad_x);
        g.x_stride = a->grad_stride;
        g.w_expert = a->w_expert;
        g.y_stride = a->grad_x_stride;
        g.w_row = (uint32_t)a->w_row;
        g.m = (uint32_t)a->m;
        g.experts = a->experts;
        g.n = a->cols;
        g.k = a->rows;
        g.zero_rest = a->zero_rest;
        g.err = d_err;
        const TileSize p = grouped_size(a->m, a->experts, a->cols, a->rows, true);
        if (grouped_part(p, a->m, a->experts, a->cols, a->rows, kFlatAcross)) g.part = static_cast<float *>(d_scratch);
        if (a->type == WC_T_BF16) launch_grouped<WC_T_BF16, false>(g, p, stream);
        else launch_grouped<WC_T_FP16, false>(g, p, stream);
    }
    if (a->grad_w) {
        GroupedDwArgs g{};
        g.x = static_cast<const uint16_t *>(a->x);
        g.dy = static_cast<const uint16_t *>(a->grad);
        g.ends = a->ends;
        g.dw = static_cast<uint16_t *>(a->grad_w);
        g.x_stride = a->x_stride;
        g.dy_stride = a->grad_stride;
        g.m = (uint32_t)a->m;
        g.experts = a->experts;
        g.n = a->rows;
        g.k = a->cols;
        g.part = static_cast<float *>(d_scratch);
        g.err = d_err;
        const TilePlan p = grouped_dw_plan(a->m, a->experts, a->rows, a->cols);
        if (a->type == WC_T_BF16) launch_grouped_dw<WC_T_BF16>(g, p, stream);
        else launch_grouped_dw<WC_T_FP16>(g, p, stream);
    }
    return launched();
}

uint64_t wc_linear_cross_entropy_scratch(uint64_t m, uint32_t vocab, uint32_t cols)
{
    if (m == 0 || !valid_loss(m, vocab, cols)) return 0;
    const uint64_t most = m < kLossSlice ? m : kLossSlice;
    // of all the sets of launches: the last one's tiles may be smaller
    uint64_t bytes = up256(8 * most * loss_parts(most, vocab, cols));
    if (m > most && m % most) {
        const uint64_t last = up256(8 * (m % most) * loss_parts(m % most, vocab, cols));
        bytes = bytes > last ? bytes : last;
    }
    return bytes + up256(4 * most);
}

wc_status wc_linear_cross_entropy(const wc_linear_loss *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err,
                                  hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16) || !valid_loss(a->m, a->vocab, a->cols)) return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (!rows16(a->hidden, a->hidden_stride, a->cols) || !rows16(a->weight, a->weight_stride, a->cols) || !a->tokens ||
        !aligned(a->tokens, 8) || !a->loss || !aligned(a->loss, 4) || !a->lse || !aligned(a->lse, 4))
        return WC_ERR_ARG;
    const uint64_t need = wc_linear_cross_entropy_scratch(a->m, a->vocab, a->cols);
    if (scratch_bytes < need) return WC_ERR_CAPACITY;
    if (!d_scratch || !aligned(d_scratch, 256)) return WC_ERR_ARG;
    const Rows hidden = rows_of(a->hidden, a->hidden_stride, a->cols, a->m), tokens = line(a->tokens, 8 * a->m);
    const Rows weight = rows_of(a->weight, a->weight_stride, a->cols, a->vocab), lse = line(a->lse, 4 * a->m);
    if (!apart(line(a->loss, 4 * a->m), lse, hidden, weight, tokens) || !apart(lse, hidden, weight, tokens)) return WC_ERR_ARG;
    const uint64_t most = a->m < kLossSlice ? a->m : kLossSlice;
    for (uint64_t r = 0; r < a->m; r += most) {
        LossArgs g{};
        g.h = static_cast<const uint16_t *>(a->hidden) + r * a->hidden_stride;
        g.w = static_cast<const uint16_t *>(a->weight);
        g.h_stride = a->hidden_stride;
        g.w_row = (uint32_t)a->weight_stride;
        g.tokens = a->tokens + r;
        g.m = (uint32_t)(a->m - r < most ? a->m - r : most);
        g.vocab = a->vocab;
        g.k = a->cols;
        g.parts = loss_parts(g.m, a->vocab, a->cols);
        g.given = static_cast<float *>(d_scratch);
        g.part = reinterpret_cast<float2 *>(static_cast<char *>(d_scratch) + up256(4 * most));
        g.loss = a->loss + r;
        g.lse = a->lse + r;
        g.err = d_err;
        if (a->type == WC_T_BF16) launch_loss<WC_T_BF16>(g, stream);
        else launch_loss<WC_T_FP16>(g, stream);
    }
    return launched();
}

uint64_t wc_linear_cross_entropy_backward_scratch(uint64_t m, uint32_t vocab, uint32_t cols)
{
    if (m == 0 || !valid_loss(m, vocab, cols)) return 0;
    const uint64_t whole = loss_grad_plan(m, vocab, cols, 2).bytes, rounded = loss_grad_plan(m, vocab, cols, 1).bytes;
    return whole > rounded ? whole : rounded;
}

wc_status wc_linear_cross_entropy_backward(const wc_linear_loss_grad *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err,
                                           hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16) || a->m == 0 || !valid_loss(a->m, a->vocab, a->cols))
        return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (!rows16(a->hidden, a->hidden_stride, a->cols) || !rows16(a->weight, a->weight_stride, a->cols) || !a->tokens ||
        !aligned(a->tokens, 8) || !a->lse || !aligned(a->lse, 4) || !aligned(a->grad_loss, 4) || !aligned(a->grad_lse, 4))
        return WC_ERR_ARG;
    if (a->grad_hidden && !rows16(a->grad_hidden, a->grad_hidden_stride, a->cols)) return WC_ERR_ARG;
    if (a->grad_weight && !aligned(a->grad_weight, 16)) return WC_ERR_ARG;
    const uint32_t terms = a->rounded ? 1 : 2;
    const LossGradPlan p = loss_grad_plan(a->m, a->vocab, a->cols, terms);
    if (scratch_bytes < wc_linear_cross_entropy_backward_scratch(a->m, a->vocab, a->cols)) return WC_ERR_CAPACITY;
    if (!d_scratch || !aligned(d_scratch, 256)) return WC_ERR_ARG;
    const Rows hidden = rows_of(a->hidden, a->hidden_stride, a->cols, a->m), tokens = line(a->tokens, 8 * a->m);
    const Rows weight = rows_of(a->weight, a->weight_stride, a->cols, a->vocab), lse = line(a->lse, 4 * a->m);
    const Rows gl = line(a->grad_loss, 4 * a->m), gz = line(a->grad_lse, 4 * a->m);
    const Rows dw = line(a->grad_weight, 2ull * a->vocab * a->cols);
    if (!apart(rows_of(a->grad_hidden, a->grad_hidden_stride, a->cols, a->m), dw, hidden, weight, tokens, lse, gl, gz) ||
        !apart(dw, hidden, weight, tokens, lse, gl, gz))
        return WC_ERR_ARG;
    if (!a->grad_hidden && !a->grad_weight) return WC_OK;
    char *s = static_cast<char *>(d_scratch);
    LossGradArgs g{};
    g.h = static_cast<const uint16_t *>(a->hidden);
    g.w = static_cast<const uint16_t *>(a->weight);
    g.h_stride = a->hidden_stride;
    g.w_row = (uint32_t)a->weight_stride;
    g.tokens = a->tokens;
    g.lse = a->lse;
    g.grad_loss = a->grad_loss;
    g.grad_lse = a->grad_lse;
    g.m = (uint32_t)a->m;
    g.vocab = a->vocab;
    g.k = a->cols;
    g.live = a->grad_weight ? reinterpret_cast<uint16_t *>(s + p.live) : nullptr;
    g.rows = reinterpret_cast<f32x4 *>(s + p.rows);
    g.most = reinterpret_cast<float *>(s + p.most);
    g.grad = reinterpret_cast<uint16_t *>(s + p.grad);
    g.err = d_err;
    if (a->type == WC_T_BF16) launch_loss_grad<WC_T_BF16>(*a, g, p, terms, s, stream);
    else launch_loss_grad<WC_T_FP16>(*a, g, p, terms, s, stream);
    return launched();
}

}  // extern "C"

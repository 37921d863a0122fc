// ops_grouped.hpp -- matrix products grouped by expert over ragged rows.  Rows
// lo_e .. hi_e of x belong to expert e (lo_e = ends[e - 1], hi_e = ends[e]):
//   y_r = W_e x_r,   dx_r = W_e^T dy_r,   dW_e = sum_r dy_r x_r^T.
//
//   k_grouped_few  y, for few rows of each expert
//   k_grouped      y, or dx, by tiles of an expert's rows
//   k_grouped_dw   dW, by tiles of an expert's weights
//   k_grouped_join, k_join  sums of products that were split along k
// The ends stay on the device: a block finds its expert and rows from them by
// itself (every wave adds up the experts' tiles by lane moves).
//
// What bounds them, and what they take: few rows, reading the weights once (122 rows of 8 experts of 14336 x 4096, by
// tiles of 64: 147 us, 6.4 TB/s); one row of each, waits that follow each other (8 of 1024 x 2048, by k_grouped_few: 11.8 us, of
// which 4.7 at the rate of reading: two trips to memory for the ends, then four for 512 columns of a wave's eight rows, at most two of them
// on their way at once, by one wave on a SIMD); many, the matrix cores at the clock that their power leaves (16384 rows of 8 of 14336 x 4096:
// dx 1520 us, dW 1550 us, 1.25 PFLOP/s); in between, tiles that are not full (32768 rows of 256 of 2048 x 7168: 1890 us, 4.3 TB/s).
#pragma once

#include "ops_common.hpp"
#include "ops_deal.hpp"
#include "ops_moe.hpp"
#include "ops_tiles.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kGroupedMaxExperts = 1024;

struct GroupedArgs {
    const uint16_t *x, *w;
    const int64_t *ends;
    uint16_t *y;
    uint64_t x_stride, w_expert, y_stride;  // strides in elements
    uint32_t w_row;
    uint32_t m, experts;
    uint32_t n, k;      // columns of y and of x
    uint32_t zero_rest; // rows behind the last expert's: zeros, else left as they are
    uint32_t slots;     // k_grouped_few
    float *part;        // tiles in parts along k; or NULL: none
    uint32_t *err;
};

// Rows of an expert, whatever the ends are (from 0 on, and not past m).
__device__ __forceinline__ uint32_t group_end(const int64_t *ends, uint32_t e, uint32_t m)
{
    // nothing writes the ends while the kernel runs: one number for all lanes is a scalar load, which does not wait for the
    // vector memory's queue
    const int64_t v = ((__attribute__((address_space(4))) const int64_t *)ends)[e];
    return v < 0 ? 0u : v < (int64_t)m ? (uint32_t)v : m;
}
__device__ __forceinline__ void group_rows(const int64_t *ends, uint32_t e, uint32_t m, uint32_t &lo, uint32_t &hi)
{
    lo = e ? group_end(ends, e - 1, m) : 0u;
    hi = max(lo, group_end(ends, e, m));
}

// Ends that go back, or past the rows.
__device__ __forceinline__ void check_ends(const int64_t *ends, uint32_t experts, uint32_t m, uint32_t *err)
{
    if (!err || blockIdx.x) return;
    for (uint32_t e = threadIdx.x; e < experts; e += blockDim.x)
        if (ends[e] > (int64_t)m || ends[e] < (e ? ends[e - 1] : 0)) report(err, WC_EF_BAD_INDEX);
}

// That look alone, where there are no rows.
__global__ __launch_bounds__(256) void k_grouped_ends(const int64_t *ends, uint32_t experts, uint32_t *err)
{
    check_ends(ends, experts, 0, err);
}

__device__ __forceinline__ uint32_t wave_upto(uint32_t v)  // the sum of lanes 0 .. this one
{
    v += lanes_moved<0x111, 0xF>(v, 0u);
    v += lanes_moved<0x112, 0xF>(v, 0u);
    v += lanes_moved<0x114, 0xF>(v, 0u);
    v += lanes_moved<0x118, 0xF>(v, 0u);
    v += lanes_moved<0x142, 0xA>(v, 0u);
    v += lanes_moved<0x143, 0xC>(v, 0u);
    return v;
}

// The experts' rows in units, of which each expert has units(count).  A wave's
// view: lane l has the experts from per l on.
struct Groups {
    uint32_t per, mine, upto, total, lo, hi;  // lo, hi: of the lane's last expert

    template <class F>
    __device__ __forceinline__ void count(const GroupedArgs &g, F units)
    {
        const uint32_t lane = threadIdx.x & 63;
        per = (g.experts + 63) / 64;
        mine = lo = hi = 0;
        for (uint32_t q = 0; q < per; q++) {
            const uint32_t e = per * lane + q;
            if (e >= g.experts) break;
            group_rows(g.ends, e, g.m, lo, hi);
            mine += units(hi - lo);
        }
        upto = wave_upto(mine);
        total = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    }
    // The expert of unit u < total, its rows, and the unit's place among its own.
    template <class F>
    __device__ __forceinline__ void find(const GroupedArgs &g, uint32_t u, F units, uint32_t &expert, uint32_t &lo, uint32_t &hi,
                                         uint32_t &place) const
    {
        const uint32_t owner = (uint32_t)__builtin_ctzll(__ballot(upto > u));
        place = u - (uint32_t)__builtin_amdgcn_readlane((int)(upto - mine), owner);
        expert = per * owner;
        if (per == 1) {
            lo = (uint32_t)__builtin_amdgcn_readlane((int)this->lo, owner);
            hi = (uint32_t)__builtin_amdgcn_readlane((int)this->hi, owner);
            return;
        }
        for (uint32_t q = 0; q < per; q++) {
            expert = min(per * owner + q, g.experts - 1);
            group_rows(g.ends, expert, g.m, lo, hi);
            const uint32_t n = units(hi - lo);
            if (place < n) break;
            place -= n;
        }
    }
};

// The tiles of y or dx, and how they are dealt to the blocks (Dealing); the sums of the
// last ones' parts are added up by k_grouped_join.
template <int BM, int BN>
struct GroupedPieces {
    static constexpr uint32_t kSlots = kCus * tile_blocks(BM, BN);
    static_assert(kSlots % 8 == 0, "the XCDs have as many each");
    Groups groups;
    Dealing deal;
    uint32_t last, down, across, stages;

    __device__ __forceinline__ static uint32_t tiles(uint32_t rows) { return (rows + BM - 1) / BM; }

    __device__ __forceinline__ void init(const GroupedArgs &g)
    {
        groups.count(g, tiles);
        last = group_end(g.ends, g.experts - 1, g.m);
        down = groups.total;
        across = (g.n + BN - 1) / BN;
        stages = (g.k + kTileK - 1) / kTileK;
        deal = Dealing::of(down * across, stages, kSlots, g.part != nullptr, g.zero_rest ? tiles(g.m - last) * across : 0u);
    }
    // The expert, rows and first column of tile t.
    __device__ __forceinline__ bool tile(const GroupedArgs &g, uint32_t t, uint32_t &expert, uint32_t &m0, uint32_t &rows,
                                         uint32_t &n0) const
    {
        uint32_t r, c, lo, hi, place;
        tile_of(t, down, across, r, c);
        groups.find(g, r, tiles, expert, lo, hi, place);
        m0 = lo + BM * place;
        n0 = BN * c;
        if ((uint64_t)place * BM >= hi - lo) return false;  // bad ends
        rows = min((uint32_t)BM, hi - m0);
        return true;
    }
};

// y (kPAlong) or dx by tiles: an expert's rows in tiles of BM against tiles of
// BN columns.  Grid: 8 ceil(tiles / 8) for the most pieces there can be, or kCus (each_tile).
template <int T, int BM, int BN, bool kPAlong>
__global__ __launch_bounds__(256, tile_blocks(BM, BN)) void k_grouped(GroupedArgs g)
{
    using Ti = Tile<T, BM, BN, true, kPAlong>;
    struct Job {
        typename Ti::Place place;
        uint32_t m0, rows, n0, part;  // part: of the tiles in parts, or none
    };
    __shared__ __attribute__((aligned(1024))) char b0[Ti::kBytes];
    __shared__ __attribute__((aligned(1024))) char b1[Ti::kBytes];
    check_ends(g.ends, g.experts, g.m, g.err);
    GroupedPieces<BM, BN> p;
    p.init(g);
    Ti ti(g.x_stride, g.w_row);
    uint32_t turn = 0;
    each_tile<Ti, Job>(
        ti, b0, b1,
        [&](uint32_t, Job &j) {
            for (;;) {
                uint32_t t, expert;
                const PieceKind kind = p.deal.next(blockIdx.x, gridDim.x, turn, t);
                if (kind == kNoMore) return false;
                if (kind == kZeros) {
                    const uint32_t m0 = p.last + BM * (t / p.across), n0 = BN * (t % p.across), cols = min((uint32_t)BN, g.n - n0) / 8;
                    for (uint32_t q = threadIdx.x; q < min((uint32_t)BM, g.m - m0) * cols; q += 256)
                        *reinterpret_cast<u32x4 *>(g.y + (m0 + q / cols) * g.y_stride + n0 + 8 * (q % cols)) = u32x4{0, 0, 0, 0};
                    continue;
                }
                const bool part = kind == kPart;
                const uint32_t split = part ? t / p.deal.left : 0, splits = part ? p.deal.splits : 1;
                if (!p.tile(g, part ? p.deal.whole + t % p.deal.left : t, expert, j.m0, j.rows, j.n0)) continue;
                j.part = splits > 1 ? t : ~0u;
                const uint32_t k0 = kTileK * (p.stages * split / splits), k = min(g.k, kTileK * (p.stages * (split + 1) / splits)) - k0;
                const uint16_t *w = g.w + expert * g.w_expert;
                j.place.q = Ti::Q::Where::at(g.x + j.m0 * g.x_stride + k0, j.rows, k);
                if constexpr (kPAlong) j.place.p = Ti::P::Where::at(w + (uint64_t)j.n0 * g.w_row + k0, min((uint32_t)BN, g.n - j.n0), k);
                else j.place.p = Ti::P::Where::at(w + (uint64_t)k0 * g.w_row + j.n0, k, g.n - j.n0);
                j.place.k = k;
                return true;
            }
        },
        [&](const Ti &ti, const Job &j) {
            if (j.part != ~0u) {
                float *part = g.part + (uint64_t)j.part * (BM * BN);
                each_four(ti, [&](uint32_t row, uint32_t col, f32x4 v) {
                    if (row < j.rows && j.n0 + col < g.n) *reinterpret_cast<f32x4 *>(part + row * BN + col) = v;
                });
            } else {
                uint16_t *y = g.y + j.m0 * g.y_stride + j.n0;
                each_eight<T>(ti, AsIs{}, [&](uint32_t row, uint32_t col, u32x4 v) {
                    if (row < j.rows && j.n0 + col < g.n) *reinterpret_cast<u32x4 *>(y + row * g.y_stride + col) = v;
                });
            }
        });
}

// The sum of n parts, `step` numbers apart, in their order; eight are on their way at once.
__device__ __forceinline__ f32x4 sum_parts(const float *p, uint64_t step, uint32_t n)
{
    f32x4 sum = *reinterpret_cast<const f32x4 *>(p);
    uint32_t s = 1;
    for (; s + 8 <= n; s += 8) {
        f32x4 v[8];
#pragma unroll
        for (uint32_t q = 0; q < 8; q++) v[q] = *reinterpret_cast<const f32x4 *>(p + (s + q) * step);
#pragma unroll
        for (uint32_t q = 0; q < 8; q++) sum += v[q];
    }
    for (; s < n; s++) sum += *reinterpret_cast<const f32x4 *>(p + s * step);
    return sum;
}

// The sums of the tiles in parts, in the order of k.  Grid: kSlots / 2 tiles, and 8 blocks for each.
template <int T, int BM, int BN>
__global__ __launch_bounds__(256) void k_grouped_join(GroupedArgs g)
{
    GroupedPieces<BM, BN> p;
    p.init(g);
    const uint32_t q = blockIdx.x / 8;
    uint32_t expert, m0, rows, n0;
    if (p.deal.splits == 1 || q >= p.deal.left || !p.tile(g, p.deal.whole + q, expert, m0, rows, n0)) return;
    const uint32_t from = BM / 8 * (blockIdx.x % 8);
    for (uint32_t e = threadIdx.x; e < BM / 8 * BN / 4; e += 256) {
        const uint32_t row = from + e / (BN / 4), col = 4 * (e % (BN / 4));
        if (row >= rows || n0 + col >= g.n) continue;
        const float *part = g.part + (uint64_t)q * (BM * BN) + row * BN + col;
        store_four<T>(g.y + (m0 + row) * g.y_stride + n0 + col, sum_parts(part, (uint64_t)p.deal.left * (BM * BN), p.deal.splits));
    }
}

struct GroupedDwArgs {
    const uint16_t *x, *dy;
    const int64_t *ends;
    uint16_t *dw;                 // experts x n x k, contiguous
    uint64_t x_stride, dy_stride;
    uint32_t m, experts, n, k;    // columns of dy and of x
    uint32_t splits;              // of an expert's rows, each with its own dW in part
    float *part;
    uint32_t *err;
};

// dW by tiles of BM rows and BN columns of it.  Grid: experts x 8 ceil(tiles of one / 8), or kCus (each_tile).
template <int T, int BM, int BN>
__global__ __launch_bounds__(256, tile_blocks(BM, BN)) void k_grouped_dw(GroupedDwArgs g)
{
    using Ti = Tile<T, BM, BN, false, false>;
    struct Job {
        typename Ti::Place place;
        uint32_t expert, split, m0, rows, n0;
    };
    __shared__ __attribute__((aligned(1024))) char b0[Ti::kBytes];
    __shared__ __attribute__((aligned(1024))) char b1[Ti::kBytes];
    check_ends(g.ends, g.experts, g.m, g.err);
    const uint32_t down = (g.n + BM - 1) / BM, across = (g.k + BN - 1) / BN, each = down * across;
    // every XCD has an eighth of each expert: the experts have different numbers of rows
    const uint32_t pieces = each * g.splits, per = (pieces + 7) / 8;
    Ti ti(g.dy_stride, g.x_stride);
    uint32_t turn = 0;
    each_tile<Ti, Job>(
        ti, b0, b1,
        [&](uint32_t, Job &j) {
            for (;; turn++) {
                const uint32_t b = block_of(turn), t = b % 8 * per + b / 8 % per;
                j.expert = b / 8 / per;
                if (j.expert >= g.experts) return false;
                if (t >= pieces) continue;
                j.split = t / each;
                uint32_t r, c, lo, hi;
                tile_of(t % each, down, across, r, c);
                group_rows(g.ends, j.expert, g.m, lo, hi);
                const uint32_t stages = (hi - lo + kTileK - 1) / kTileK;
                const uint32_t from = min(hi, lo + kTileK * (uint32_t)((uint64_t)stages * j.split / g.splits));
                const uint32_t to = min(hi, lo + kTileK * (uint32_t)((uint64_t)stages * (j.split + 1) / g.splits));
                j.m0 = BM * r;
                j.n0 = BN * c;
                j.rows = BM;
                j.place.q = Ti::Q::Where::at(g.dy + from * g.dy_stride + j.m0, to - from, g.n - j.m0);
                j.place.p = Ti::P::Where::at(g.x + from * g.x_stride + j.n0, to - from, g.k - j.n0);
                j.place.k = to - from;
                turn++;
                return true;
            }
        },
        [&](const Ti &ti, const Job &j) {
            const uint64_t at = ((uint64_t)j.expert * g.n + j.m0) * g.k + j.n0;
            if (g.splits > 1) {
                float *part = g.part + j.split * ((uint64_t)g.experts * g.n * g.k) + at;
                each_four(ti, [&](uint32_t row, uint32_t col, f32x4 v) {
                    if (j.m0 + row < g.n && j.n0 + col < g.k) *reinterpret_cast<f32x4 *>(part + (uint64_t)row * g.k + col) = v;
                });
            } else {
                uint16_t *dw = g.dw + at;
                each_eight<T>(ti, AsIs{}, [&](uint32_t row, uint32_t col, u32x4 v) {
                    if (j.m0 + row < g.n && j.n0 + col < g.k) *reinterpret_cast<u32x4 *>(dw + (uint64_t)row * g.k + col) = v;
                });
            }
        });
}

constexpr uint32_t kLossRowBlocks = 256;

// What G is multiplied by before it is rounded: 1 (BF16) or 2^14 (FP16) over the
// largest gradient of a row, from the largest of each of kLossRowBlocks parts.  So
// where all rows have the same one, as under a mean, what it is has no rounding
// of its own where G is rounded to one of them (the gradients of a mean over 4096 rows, BF16, were 0.26% off so, most of it
// one common factor, and are 0.21%), and FP16 numbers stay in range.
template <int T>
__device__ __forceinline__ float loss_scale(const float *most, float &unscale)
{
    constexpr float kTop = T == WC_T_FP16 ? 16384.f : 1.f;
    float v = 0.f;
#pragma unroll
    for (uint32_t q = 0; q < kLossRowBlocks / 64; q++) v = fmaxf(v, most[64 * q + (threadIdx.x & 63)]);
    v = wave_max(v);
    if (!(v > 0x1p-100f && v < 0x1p100f)) return term_scale<T>(v, unscale);
    unscale = v * (1.f / kTop);
    return kTop / v;
}

// out = the sum of `splits` parts of rows x cols each, in their order.
struct JoinArgs {
    const float *part;
    uint16_t *out;
    uint64_t out_stride;
    uint64_t rows;
    uint32_t cols, splits;
    const float *most;     // or NULL: what the numbers were scaled by (loss_scale)
};

// Four numbers a thread, or where a launch cannot hold so many threads, every gridDim.x * 256th four.
template <int T>
__global__ __launch_bounds__(256) void k_join(JoinArgs g)
{
    float unscale = 1.f;
    if (g.most) loss_scale<T>(g.most, unscale);
    const uint32_t per = g.cols / 4;
    for (uint64_t q = (uint64_t)blockIdx.x * 256 + threadIdx.x; q < g.rows * per; q += (uint64_t)gridDim.x * 256) {
        const uint64_t row = q / per;
        const uint32_t col = 4 * (uint32_t)(q % per);
        const f32x4 v = sum_parts(g.part + row * g.cols + col, g.rows * g.cols, g.splits) * unscale;
        store_four<T>(g.out + row * g.out_stride + col, v);
    }
}

// Sixteen rows of weights from n and the sixteen after them (fewer than 32:
// the second ones overlap the first) against up to 16 NT rows of x.
template <int T, int NT>
__device__ __forceinline__ void few_rows(const uint16_t *w, uint32_t pitch, uint32_t n, const uint32_t (&first)[2],
                                         const uint16_t *x, uint64_t x_stride, uint32_t count, uint32_t c0, uint32_t c1,
                                         Strip *strips, f32x4 (&sum)[2][2])
{
    const uint32_t i = threadIdx.x & 15, rows = min(16u, n);
    const uint16_t *const weights[2] = {w + (uint64_t)first[0] * pitch, w + (uint64_t)first[1] * pitch};
    f32x4 acc[2][1][NT];
    const float scale[NT] = {};  // of no use here
#pragma unroll
    for (int t = 0; t < NT; t++) acc[0][0][t] = acc[1][0][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    strip_product<T, 2, false, NT>(
        weights, [&](uint32_t r) { return min(r, rows - 1) * pitch; },
        [&](int t) { return x + min(16 * t + i, count - 1) * x_stride; }, c0, c1, strips, scale, acc);
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int m = 0; m < 2; m++) sum[m][t] = acc[m][0][t];
}

// 32 rows of weights (n of them in all) from n0 on against `count` <= 16 kTiles rows of
// x, columns of all k.  kSplit: the block's four waves share the columns, and
// f(t, sums) is called by the wave t with the sums of 16 rows of x; otherwise the rows
// are the wave's own, and it calls f for every t.  sums[m]: the lane's four
// of weights' rows first[m] + 4 gr on, against row 16 t + i of x.
template <int T, bool kSplit, int kTiles, class F>
__device__ __forceinline__ void few_product(const uint16_t *w, uint32_t pitch, uint32_t n, uint32_t n0, uint32_t k,
                                            const uint16_t *x, uint64_t x_stride, uint32_t count, Strip (*strips)[2], F f)
{
    static_assert(kTiles == 1 || kTiles == 2, "one sixteen of rows of x or two");
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const uint32_t most = n < 16 ? 0 : n - 16, first[2] = {min(n0, most), min(n0 + 16, most)};
    uint32_t c0 = 0, c1 = k;
    if (kSplit) wave_quarter(k, kStripCols, wave, c0, c1);
    f32x4 sum[2][2];
    const uint32_t tiles = kTiles == 1 ? 1 : (count + 15) / 16;
    if (tiles == 1) few_rows<T, 1>(w, pitch, n, first, x, x_stride, count, c0, c1, strips[wave], sum);
    else few_rows<T, kTiles>(w, pitch, n, first, x, x_stride, count, c0, c1, strips[wave], sum);
    if constexpr (!kSplit) {
#pragma unroll
        for (uint32_t t = 0; t < kTiles; t++)
            if (t < tiles) f(t, first, sum[0][t], sum[1][t]);
    } else {
        f32x4(*part)[4][64] = reinterpret_cast<f32x4(*)[4][64]>(&strips[0][0]);  // [4], when the strips are done
        static_assert(sizeof(Strip) * 8 >= 4 * 4 * 64 * 16, "the waves' sums fit into the strips");
        __syncthreads();
#pragma unroll
        for (uint32_t t = 0; t < kTiles; t++)
            if (t < tiles) {
                part[wave][2 * t][lane] = sum[0][t];
                part[wave][2 * t + 1][lane] = sum[1][t];
            }
        __syncthreads();
        if (wave < tiles) {
            f32x4 v[2];
#pragma unroll
            for (int m = 0; m < 2; m++) {
                const uint32_t q = 2 * wave + m;
                v[m] = (part[0][q][lane] + part[1][q][lane]) + (part[2][q][lane] + part[3][q][lane]);
            }
            f(wave, first, v[0], v[1]);
        }
        __syncthreads();  // before the strips are written again
    }
}

// Eight rows of weights (n of them in all) from n0 on against one row of x, by
// a wave.  f(row, sum) by one lane for each row that exists.
template <int T, class F>
__device__ __forceinline__ void one_product(const uint16_t *w, uint32_t pitch, uint32_t n, uint32_t n0, uint32_t k,
                                            const uint16_t *x, F f)
{
    constexpr int R = 8;
    const uint32_t lane = threadIdx.x & 63;
    const uint16_t *rows[R];
    float acc[R], mine = 0.f;
#pragma unroll
    for (int r = 0; r < R; r++) {
        rows[r] = w + (uint64_t)min(n0 + r, n - 1) * pitch;
        acc[r] = 0.f;
    }
    rows_product<T, R>(rows, 0, k, [&](uint32_t c, float *v) { Type<T>::unpack(load16<16>(x + c), v); }, acc);
#pragma unroll
    for (int r = 0; r < R; r++) {
        acc[r] = wave_sum(acc[r]);
        if (lane == (uint32_t)r) mine = acc[r];
    }
    if (lane < R && n0 + lane < n) f(n0 + lane, mine);
}

// y for experts with few rows: a block has 32 rows of weights (128 without
// kSplit) of the slot-th expert that has rows.  Reading the weights is the
// bound, so they go in whole lines past the caches, and 32 rows of x meet them
// at a time; a single one meets them without the matrix cores.  Grid: slots x ceil(n / 32
// or 128); one slot more where the rows behind the last expert's are to be zeros.
template <int T, bool kSplit>
__global__ __launch_bounds__(256, 2) void k_grouped_few(GroupedArgs g)
{
    __shared__ Strip strips[4][2];
    check_ends(g.ends, g.experts, g.m, g.err);
    const uint32_t wave = threadIdx.x >> 6, i = threadIdx.x & 15, gr = (threadIdx.x & 63) >> 4;
    const uint32_t slot = blockIdx.x % g.slots, n0 = blockIdx.x / g.slots * (kSplit ? 32 : 128) + (kSplit ? 0 : 32 * wave);
    auto any = [](uint32_t rows) { return rows ? 1u : 0u; };
    Groups groups;
    groups.count(g, any);
    uint32_t expert, lo, hi, place;
    if (slot >= groups.total) {
        const uint32_t last = group_end(g.ends, g.experts - 1, g.m);
        if (slot > groups.total || !g.zero_rest) return;
        const uint32_t from = kSplit ? 32 * (blockIdx.x / g.slots) : 128 * (blockIdx.x / g.slots), per = kSplit ? 4 : 16;
        for (uint32_t q = threadIdx.x; q < (g.m - last) * per; q += 256) {
            const uint32_t c = from + 8 * (q % per);
            if (c < g.n) *reinterpret_cast<u32x4 *>(g.y + (last + q / per) * g.y_stride + c) = u32x4{0, 0, 0, 0};
        }
        return;
    }
    groups.find(g, slot, any, expert, lo, hi, place);
    const uint16_t *w = g.w + expert * g.w_expert;
    for (uint32_t r0 = lo; r0 < hi; r0 += 32) {
        const uint32_t count = min(32u, hi - r0);
        const uint16_t *x = g.x + r0 * g.x_stride;
        if (count == 1) {
            uint16_t *y = g.y + r0 * g.y_stride;
            for (uint32_t q = 0; q < (kSplit ? 1 : 4); q++) {
                const uint32_t n = kSplit ? n0 + 8 * wave : n0 + 8 * q;
                if (n < g.n) one_product<T>(w, g.w_row, g.n, n, g.k, x, [&](uint32_t r, float v) { y[r] = Type<T>::from_f32(v); });
            }
        } else if (kSplit || n0 < g.n) {
            few_product<T, kSplit, 2>(w, g.w_row, g.n, n0, g.k, x, g.x_stride, count, strips,
                                   [&](uint32_t t, const uint32_t(&first)[2], f32x4 v0, f32x4 v1) {
                                       const uint32_t r = 16 * t + i;
                                       if (r >= count) return;
                                       uint16_t *y = g.y + (r0 + r) * g.y_stride + 4 * gr;
                                       const uint32_t a = first[0] + 4 * gr, b = first[1] + 4 * gr;
                                       if (a >= n0 && a < g.n) store_four<T>(y + first[0], v0);
                                       if (b >= n0 + 16 && b < g.n) store_four<T>(y + first[1], v1);
                                   });
        }
    }
}

}  // namespace ops
}  // namespace wc

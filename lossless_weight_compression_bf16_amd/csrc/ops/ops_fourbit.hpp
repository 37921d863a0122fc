// ops_fourbit.hpp -- products of few rows with weights of 4 bits and group
// scales, and their making:
//   w_rk = s_rg (q_rk - z_rg),  g = k / group,   y = x w^T
// with q in 0..15, two of them in a byte (the even column in the low half), and z 8 where none is given.
//
//   k_linear4    y
//   k_quantize4  q, s and z of 16-bit weights
// What bounds it: reading the weights, half a byte for a column, so that
// little may be done for each.  A wave keeps its 256 columns of x in registers, in
// operand order, and reads those of one sixteen of rows of weights after the
// other, two sixteens ahead.  Eight weights are a
// word; two shifts and masks with a constant make a pair of them the 16-bit
// numbers 16 + q, exactly, and the matrix cores sum (16 + q) x over a group in
// fp32.  The group's result is s (that - (16 + z) sum x), the sum of x having been made
// once by a product with ones, and being where the group's sum begins.  So a weight takes 1 to 1.5 vector
// instructions, and s and z meet it in fp32.  With an infinity in x the result is
// NaN, also where every weight is finite, and so it may be where a group's sum of 31 |x| passes fp32's range.
// Measured: 1 row and 4096 x 4096, groups of 64: 7.4 us in the kernel, of which the weights' 8.9 MB take
// 1.4 at the rate of a copy and the rest is one launch and one way through memory, LDS and a
// barrier; 1 row and 128256 x 4096, 63 us, 4.5 TB/s: a barrier of 16 waves and a joining of their sums for every sixteen of rows, while
// the next two are on their way; 61 rows and 14336 x 4096, groups of 128, 29 us, of which vector instructions take 11 and
// LDS 6: the rest is the same barrier, twice for each sixteen (4096 columns are two passes of eight waves) and all of it twice, as
// 61 rows are two times 32.  More rows are more such turns: 2048 rows 712 us, where the products alone need 172.
// k_quantize4: 4096 x 4096 15 us, 128256 x 4096 422 to 453 us, 3.0 TB/s of reading and writing where a copy reaches
// 6.5: a thread has one load of 16 bytes on its way, then eight divisions.  Weights are made once.
#pragma once

#include "ops_common.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kRowTiles4 = 32;  // sixteens of rows of a block, at most

struct Linear4Args {
    const uint16_t *x;
    const uint8_t *q;
    const uint16_t *scales, *zeros;  // zeros: or NULL
    uint16_t *y;
    uint64_t x_stride, q_row, y_stride;  // q_row in bytes
    uint32_t m, rows, cols, groups;
    uint32_t row_tiles;  // sixteens of rows of a block
    uint32_t row_blocks;
};

// Pair j of a word's eight weights, j and j + 4, as 16-bit floats 16 + q: 16 has
// the exponent in which the four bits below the leading one are whole numbers.
template <int T>
__device__ __forceinline__ uint32_t pair4(uint32_t w, int j)
{
    constexpr int kAt = T == WC_T_BF16 ? 3 : 6;  // the lowest of those bits
    constexpr uint32_t kMask = 0x000F000Fu << kAt, kSixteen = T == WC_T_BF16 ? 0x41804180u : 0x4C004C00u;
    const int up = kAt - 4 * j;
    return ((up >= 0 ? w << (up >= 0 ? up : 0) : w >> (up >= 0 ? 0 : -up)) & kMask) | kSixteen;
}

// Weights, scales and zero points of sixteen rows and a slice of the columns.
// A wave loads them as they lie, 16 bytes a lane, the lanes along a row, and turns them in LDS: read for the
// matrix cores, 4 to 16 bytes of each of sixteen rows at a time, they came at 1.5 TB/s, and so at 4.
template <int GROUP, int SLICE, bool kZeros>
struct Sixteen {
    static constexpr int V = GROUP / 32;     // words of a lane in a group
    static constexpr int G = SLICE / GROUP;  // groups of a slice
    static constexpr int U = SLICE / 32;     // sixteens of bytes of a row
    static constexpr int L = U > 4 ? U / 4 : 1, LS = G > 4 ? G / 4 : 1;  // loads

    struct Place {  // of a wave
        u32x4 q[16 * U];
        alignas(16) uint16_t s[16][G], z[kZeros ? 16 : 1][G];
    };
    u32x4 q[L];
    uint16_t s[LS], z[kZeros ? LS : 1];

    // Of the rows from n and the columns from k0 on; past the last, the last one's and the last group's.
    __device__ __forceinline__ void fetch(const Linear4Args &g, uint32_t n, uint32_t k0)
    {
        const uint32_t lane = threadIdx.x & 63;
        n = min(n, g.rows - 1);
        const uint32_t rows = g.rows - 1 - n;  // places of a lane in 32 bits from where the wave reads
        const uint8_t *from = g.q + (uint64_t)n * g.q_row;
        const uint16_t *scales = g.scales + (uint64_t)n * g.groups, *zeros = g.zeros + (uint64_t)n * g.groups;
#pragma unroll
        for (int j = 0; j < L; j++) {
            const uint32_t f = (64 * j + lane) % (16 * U);
            q[j] = load16<16>(from + (min(f / U, rows) * (uint32_t)g.q_row + 16 * min(k0 / 32 + f % U, g.cols / 32 - 1)));
        }
#pragma unroll
        for (int j = 0; j < LS; j++) {
            const uint32_t f = (64 * j + lane) % (16 * G), at = min(f / G, rows) * g.groups + min(k0 / GROUP + f % G, g.groups - 1);
            s[j] = scales[at];
            if constexpr (kZeros) z[j] = zeros[at];
        }
    }
    // where a row's sixteen of bytes lies: so that the lanes that read together touch all banks once
    __device__ __forceinline__ static uint32_t place(uint32_t row, uint32_t unit)
    {
        const uint32_t top = row >> 3 & 1;
        const uint32_t other = U == 8 ? row >> 1 : U == 4 ? ((row >> 2 & 1) ^ top) << 1 | top : 0;
        return row * U + (unit ^ other);
    }
    __device__ __forceinline__ void put(Place &to) const
    {
        const uint32_t lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < L; j++) {
            const uint32_t f = (64 * j + lane) % (16 * U);
            to.q[place(f / U, f % U)] = q[j];
        }
#pragma unroll
        for (int j = 0; j < LS; j++) {
            const uint32_t f = (64 * j + lane) % (16 * G);
            to.s[f / G][f % G] = s[j];
            if constexpr (kZeros) to.z[f / G][f % G] = z[j];
        }
    }
    // lane 16 gr + i's words of group c: of row i, the columns from 8 V gr on
    __device__ __forceinline__ static void words(const Place &at, int c, uint32_t *w)
    {
        const uint32_t lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4, byte = GROUP / 2 * c + 4 * V * gr;
        struct alignas(4 * V) Words {
            uint32_t w[V];
        };
        const Words v = *reinterpret_cast<const Words *>(reinterpret_cast<const uint8_t *>(&at.q[place(i, byte / 16)]) + byte % 16);
#pragma unroll
        for (int e = 0; e < V; e++) w[e] = v.w[e];
    }
};

// y of 16 row_tiles rows of weights and 16 NT rows of x.  A block's waves share
// the columns, SLICE of them each at a time; for every sixteen of rows their
// sums meet in LDS, where all of them add them up (one wave alone kept the others waiting: 50 us against 37 for 61 rows
// at the time).  A slice that would pass the last column begins earlier and leaves out the groups that it
// shares with the one before.
// Grid: row_blocks x ceil(m / (16 NT)), those with the same rows of weights on the same XCD, one
// after the other.
template <int T, int GROUP, int NT, int SLICE, int WAVES, bool kZeros>
__global__ __launch_bounds__(64 * WAVES) void k_linear4(Linear4Args g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    using Some = Sixteen<GROUP, SLICE, kZeros>;
    constexpr int V = Some::V, G = Some::G;
    // x is loaded as it lies and turned in LDS, in S parts of P eights of a row, by L loads
    constexpr int P = SLICE < 128 ? SLICE / 8 : 16, S = SLICE / (8 * P), L = 16 * P / 64;
    constexpr uint32_t kSums = 256 * NT;  // of a sixteen of rows
    __shared__ u32x4 turned[WAVES][16 * P];
    __shared__ f32x4 parts[2][WAVES][NT][64];
    __shared__ float sums[kRowTiles4][kSums];   // of the columns before, where they are more than the waves take at once
    __shared__ f32x4 of_x[WAVES][G][NT][4];     // each wave's sums of x
    static_assert(sizeof(typename Some::Place) <= sizeof(turned[0]), "weights are turned where x was");
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), waves = blockDim.x >> 6;
    const uint32_t lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t turns = (g.m + 16 * NT - 1) / (16 * NT), xcd = blockIdx.x % 8, at = blockIdx.x / 8;
    const uint32_t row_block = at / turns * 8 + xcd, t0 = 16 * NT * (at % turns);
    if (row_block >= g.row_blocks) return;
    const uint32_t n0 = 16 * g.row_tiles * row_block, tiles = min(g.row_tiles, (g.rows - n0 + 15) / 16);
    constexpr uint32_t kOnes = T == WC_T_BF16 ? 0x3F803F80u : 0x3C003C00u;
    const X8 one = __builtin_bit_cast(X8, u32x4{kOnes, kOnes, kOnes, kOnes});

    const uint32_t passes = (g.cols + SLICE * waves - 1) / (SLICE * waves);
    // neighbours begin at other columns, so that they do not all read the same memory channels
    uint32_t k0 = SLICE * (row_block % passes * waves + wave);
    uint32_t turn = 0;
    for (uint32_t pass = 0; pass < passes; pass++) {
        const uint32_t from = min(k0, g.cols - SLICE), k1 = k0 + SLICE * waves < SLICE * waves * passes ? k0 + SLICE * waves : SLICE * wave;
        const bool last = pass + 1 == passes;
        Some a, b, c;
        a.fetch(g, n0, from);
        if (tiles > 1) b.fetch(g, n0 + 16, from);
        u32x4 xv[G][V][NT];  // x of the slice: for each word of weights, its eight columns in the order of the pairs
        u32x4 raw[NT][S][L];
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int h = 0; h < S; h++)
#pragma unroll
                for (int j = 0; j < L; j++) {
                    const uint32_t f = 64 * j + lane;
                    raw[t][h][j] = load16<16>(g.x + min(t0 + 16 * t + f / P, g.m - 1) * g.x_stride + from + 8 * P * h + 8 * (f % P));
                }
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int h = 0; h < S; h++) {
#pragma unroll
                for (int j = 0; j < L; j++) {
                    const uint32_t f = 64 * j + lane, row = f / P;
                    turned[wave][row * P + ((f ^ row) & (P - 1))] = raw[t][h][j];
                }
#pragma unroll
                for (int c = 0; c < P * 8 / GROUP; c++)
#pragma unroll
                    for (int e = 0; e < V; e++)
                        xv[P * 8 / GROUP * h + c][e][t] = turned[wave][i * P + ((GROUP / 8 * c + V * gr + e) ^ (i & (P - 1)))];
            }
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int c = 0; c < G; c++) {
                f32x4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < V; e++) {
                    const u32x4 v = xv[c][e][t];
                    xv[c][e][t] = u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                                        __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
                    d = Ty::mfma(__builtin_bit_cast(X8, v), one, d);
                }
                if (i == 0) of_x[wave][c][t][gr] = (kZeros ? -1.f : -24.f) * d;
                __builtin_amdgcn_sched_barrier(0);
            }
        typename Some::Place &place = *reinterpret_cast<typename Some::Place *>(turned[wave]);
        asm volatile("" ::: "memory");  // x has been read from there
        const auto step = [&](uint32_t r, const Some &now) {
            f32x4 acc[NT];
            now.put(place);
#pragma unroll
            for (int t = 0; t < NT; t++) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < G; c++) {
                __builtin_amdgcn_sched_barrier(0);
                if (k0 > from + GROUP * c) continue;
                const float scale = Ty::to_f32(place.s[i][c]), zero = kZeros ? 16.f + Ty::to_f32(place.z[i][c]) : 1.f;
                uint32_t w[V];
                Some::words(place, c, w);
                f32x4 d[NT];
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    d[t] = of_x[wave][c][t][gr];
                    if (kZeros) d[t] = zero * d[t];
                }
#pragma unroll
                for (int e = 0; e < V; e++) {
                    const uint32_t v = w[e];
                    const X8 p = __builtin_bit_cast(X8, u32x4{pair4<T>(v, 0), pair4<T>(v, 1), pair4<T>(v, 2), pair4<T>(v, 3)});
#pragma unroll
                    for (int t = 0; t < NT; t++) d[t] = Ty::mfma(__builtin_bit_cast(X8, xv[c][e][t]), p, d[t]);
                }
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[t][e] = __builtin_fmaf(scale, d[t][e], acc[t][e]);
            }
#pragma unroll
            for (int t = 0; t < NT; t++) parts[turn][wave][t][lane] = acc[t];
            __builtin_amdgcn_s_waitcnt(0xC07F);  // LDS, and not the weights on their way
            asm volatile("s_barrier" ::: "memory");
            for (uint32_t f = threadIdx.x; f < kSums; f += 64 * waves) {
                float v = reinterpret_cast<const float *>(parts[turn][0])[f];
#pragma unroll
                for (uint32_t q = 1; q < WAVES; q++) {
                    const float p = reinterpret_cast<const float *>(parts[turn][min(q, waves - 1)])[f];
                    v += q < waves ? p : 0.f;
                }
                if (pass) v += sums[r][f];
                if (!last) {
                    sums[r][f] = v;
                    continue;
                }
                const uint32_t n = n0 + 16 * r + f / 4 % 16, token = t0 + f / 256 * 16 + f / 64 % 4 * 4 + f % 4;
                if (n < g.rows && token < g.m) g.y[token * g.y_stride + n] = Ty::from_f32(v);
            }
            turn ^= 1;
        };
        // Two sixteens ahead, in each of the three's places, and past the last one its own once more: a load
        // under a condition would have every wait taken for those after it as well (38 us against 29 for
        // 61 rows at the time).
        uint32_t r = 0;
        for (; r + 3 <= tiles; r += 3) {
            c.fetch(g, n0 + 16 * (r + 2), from);
            step(r, a);
            a.fetch(g, n0 + 16 * min(r + 3, tiles - 1), from);
            step(r + 1, b);
            b.fetch(g, n0 + 16 * min(r + 4, tiles - 1), from);
            step(r + 2, c);
        }
        if (r < tiles) step(r, a);
        if (r + 1 < tiles) step(r + 1, b);
        asm volatile("" ::: "memory");  // and the weights
        k0 = k1;
    }
}

struct Quantize4Args {
    const uint16_t *w;
    uint64_t w_stride;
    uint8_t *q;
    uint16_t *scales, *zeros;
    uint64_t rows;
    uint32_t cols;
};

// q, s and z of eight columns by a lane, a group by GROUP / 8 lanes.  s is what
// its 16 bits say when w is divided by it, so that q is the nearest there is.
template <int T, int GROUP>
__global__ __launch_bounds__(256) void k_quantize4(Quantize4Args g)
{
    using Ty = Type<T>;
    const uint32_t per = g.cols / 8;
    const uint64_t at = (uint64_t)blockIdx.x * 256 + threadIdx.x, row = at / per;
    if (row >= g.rows) return;  // whole groups of lanes: per is a multiple of theirs
    const uint32_t col = 8 * (uint32_t)(at % per);
    float f[8];
    Ty::unpack(load16<2>(g.w + row * g.w_stride + col), f);
    float lo = 0.f, hi = 0.f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        lo = fminf(lo, f[e]);
        hi = fmaxf(hi, f[e]);
        bad |= f[e] != f[e];
    }
#pragma unroll
    for (int o = 1; o < GROUP / 8; o *= 2) {
        lo = fminf(lo, __shfl_xor(lo, o, 64));
        hi = fmaxf(hi, __shfl_xor(hi, o, 64));
        bad |= __shfl_xor((int)bad, o, 64) != 0;
    }
    const float range = hi - lo;  // of finite numbers it may be past the largest, its fifteenth is not
    const float step = bad ? nan32() : !g.zeros ? fmaxf(hi, -lo) / 7.f : range < kInf ? range / 15.f : hi / 15.f - lo / 15.f;
    const uint16_t scale = Ty::from_f32(step);
    const float s = Ty::to_f32(scale);
    float zero = 8.f;
    if (g.zeros) zero = s > 0.f && s < kInf ? fminf(rintf(-lo / s), 15.f) : 0.f;
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const float v = s > 0.f && s < kInf ? rintf(f[e] / s) + zero : zero;
        q |= (uint32_t)fminf(fmaxf(v, 0.f), 15.f) << (4 * e);
    }
    *reinterpret_cast<uint32_t *>(g.q + row * (g.cols / 2) + col / 2) = q;
    if (col % GROUP == 0) {
        const uint64_t group = row * (g.cols / GROUP) + col / GROUP;
        g.scales[group] = scale;
        if (g.zeros) g.zeros[group] = Ty::from_f32(zero);
    }
}

}  // namespace ops
}  // namespace wc

// ops_fourbit.hpp -- products of few rows with weights of 4 bits and group
// scales, and their making:
//   w_rk = s_rg (q_rk - z_rg),  g = k / group,   y = x w^T
// with q in 0..15, two of them in a byte (the even column in the low half), and z 8 where none is given.
//
//   k_linear4    y
//   k_quantize4  q, s and z of 16-bit weights
// What bounds it: reading the weights, half a byte for a column, so that
// little may be done for each.  A wave keeps its 256 columns of x in registers, in
// operand order, and reads those of one 16 rows of weights after the other, whole lines
// past the caches.  Eight weights are a word; two shifts and masks with a
// constant make a pair of them the 16-bit numbers 16 + q, exactly, and the
// matrix cores sum (16 + q) x over a group in fp32.  The group's result is
// s (that - (16 + z) sum x), the sum of x having been made once by a product with ones.
// So a weight takes 1 to 1.5 vector instructions, and s and z meet it in fp32.
#pragma once

#include "ops_common.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kSlice4 = 256;      // columns of a wave at a time
constexpr uint32_t kRowTiles4 = 4;     // sixteens of rows of a block

struct Linear4Args {
    const uint16_t *x;
    const uint8_t *q;
    const uint16_t *scales, *zeros;  // zeros: or NULL
    uint16_t *y;
    uint64_t x_stride, q_row, y_stride;  // q_row in bytes
    uint32_t m, rows, cols, groups;
    uint32_t row_tiles;  // sixteens of rows of a block, up to kRowTiles4
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

// n consecutive 16-bit values at any of their addresses
template <int n>
__device__ __forceinline__ void load_halves(const uint16_t *p, uint32_t *v)
{
    if constexpr (n == 8) {
        const u32x4 q = load16<2>(p);
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = q[e];
    } else {
        struct __attribute__((packed, aligned(2))) Words {
            uint32_t w[n / 2];
        };
        const Words q = *reinterpret_cast<const Words *>(p);
#pragma unroll
        for (int e = 0; e < n / 2; e++) v[e] = q.w[e];
    }
}

// Weights, scales and zero points of sixteen rows and a slice of the columns.
template <int GROUP>
struct Sixteen {
    static constexpr int V = GROUP / 32;       // words of a lane in a group
    static constexpr int G = kSlice4 / GROUP;  // groups of a slice

    uint32_t w[G][V], s[4][(G + 1) / 2], z[4][(G + 1) / 2];

    __device__ __forceinline__ void fetch(const Linear4Args &g, uint32_t n, uint32_t k0, uint32_t g0, bool whole)
    {
        const uint32_t lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
        const uint8_t *row = g.q + (uint64_t)min(n + i, g.rows - 1) * g.q_row;
#pragma unroll
        for (int c = 0; c < G; c++) {
            const uint8_t *p = row + min((k0 + GROUP * c) / 2, g.cols / 2 - GROUP / 2) + 4 * V * gr;
            if constexpr (V == 4) {
                const u32x4 v = read16<16, true>(p);
#pragma unroll
                for (int e = 0; e < 4; e++) w[c][e] = v[e];
            } else if constexpr (V == 2) {
                const uint64_t v = __builtin_nontemporal_load(reinterpret_cast<const uint64_t *>(p));
                w[c][0] = (uint32_t)v;
                w[c][1] = (uint32_t)(v >> 32);
            } else {
                w[c][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p));
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const uint64_t first = (uint64_t)min(n + 4 * gr + e, g.rows - 1) * g.groups + g0;
            if (whole) {
                load_halves<G>(g.scales + first, s[e]);
                if (g.zeros) load_halves<G>(g.zeros + first, z[e]);
            } else {  // groups past the last have a scale of 0
#pragma unroll
                for (int c = 0; c < G; c++) {
                    const bool in = g0 + c < g.groups;
                    const uint32_t a = in ? g.scales[first + c] : 0u, b = in && g.zeros ? g.zeros[first + c] : 0u;
                    s[e][c / 2] = c % 2 ? s[e][c / 2] | a << 16 : a;
                    z[e][c / 2] = c % 2 ? z[e][c / 2] | b << 16 : b;
                }
            }
        }
    }
};

// y of 16 row_tiles rows of weights and 16 NT rows of x.  A block's waves share
// the columns, 256 of them each at a time, and add up in LDS.  Grid: row_blocks x ceil(m / (16 NT)),
// those with the same rows of weights on the same XCD, one after the other.
template <int T, int GROUP, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_linear4(Linear4Args g)
{
    using Ty = Type<T>;
    using X8 = typename Ty::x8;
    constexpr int V = Sixteen<GROUP>::V, G = Sixteen<GROUP>::G;
    __shared__ f32x4 part[WAVES][kRowTiles4][NT][64];
    const uint32_t wave = threadIdx.x >> 6, waves = blockDim.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
    const uint32_t turns = (g.m + 16 * NT - 1) / (16 * NT), xcd = blockIdx.x % 8, at = blockIdx.x / 8;
    const uint32_t row_block = at / turns * 8 + xcd, t0 = 16 * NT * (at % turns);
    if (row_block >= g.row_blocks) return;
    const uint32_t n0 = 16 * g.row_tiles * row_block;
    f32x4 acc[kRowTiles4][NT];
#pragma unroll
    for (int r = 0; r < (int)kRowTiles4; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t ones = T == WC_T_BF16 ? 0x3F803F80u : 0x3C003C00u;

    for (uint32_t k0 = kSlice4 * wave; k0 < g.cols; k0 += kSlice4 * waves) {
        const uint32_t g0 = k0 / GROUP;
        const bool whole = g0 + G <= g.groups;  // the same for the whole wave
        Sixteen<GROUP> now, next;
        now.fetch(g, n0, k0, g0, whole);
        // x of the slice as operands: for each word of weights, its eight columns in the order of the pairs
        u32x4 xv[G][V][NT];
        float sx[G][NT];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const uint16_t *row = g.x + min(t0 + 16 * t + i, g.m - 1) * g.x_stride;
#pragma unroll
            for (int c = 0; c < G; c++)
#pragma unroll
                for (int e = 0; e < V; e++) {
                    const uint32_t k = k0 + GROUP * c + 8 * V * gr + 8 * e;
                    const u32x4 v = only(k < g.cols, load16<16>(row + min(k, g.cols - 8)));
                    xv[c][e][t] = u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                                        __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
                }
        }
        const X8 one = __builtin_bit_cast(X8, u32x4{ones, ones, ones, ones});
#pragma unroll
        for (int c = 0; c < G; c++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
                f32x4 d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < V; e++) d = Ty::mfma(one, __builtin_bit_cast(X8, xv[c][e][t]), d);
                sx[c][t] = d[0];  // the same in all rows
            }
#pragma unroll
        for (int r = 0; r < (int)kRowTiles4; r++) {
            if (r < (int)g.row_tiles) {
                if (r + 1 < (int)g.row_tiles) next.fetch(g, n0 + 16 * (r + 1), k0, g0, whole);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int c = 0; c < G; c++) {
                    f32x4 d[NT];
#pragma unroll
                    for (int t = 0; t < NT; t++) d[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        const uint32_t v = now.w[c][e];
                        const X8 a = __builtin_bit_cast(X8, u32x4{pair4<T>(v, 0), pair4<T>(v, 1), pair4<T>(v, 2), pair4<T>(v, 3)});
#pragma unroll
                        for (int t = 0; t < NT; t++) d[t] = Ty::mfma(a, __builtin_bit_cast(X8, xv[c][e][t]), d[t]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float scale = Ty::to_f32((uint16_t)(now.s[e][c / 2] >> (c % 2 * 16)));
                        const float zero = g.zeros ? 16.f + Ty::to_f32((uint16_t)(now.z[e][c / 2] >> (c % 2 * 16))) : 24.f;
#pragma unroll
                        for (int t = 0; t < NT; t++) acc[r][t][e] = __builtin_fmaf(scale, d[t][e] - zero * sx[c][t], acc[r][t][e]);
                    }
                }
                now = next;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < (int)kRowTiles4; r++)
        if (r < (int)g.row_tiles)
#pragma unroll
            for (int t = 0; t < NT; t++) part[wave][r][t][lane] = acc[r][t];
    __syncthreads();
    // lane l of sixteen r and tile t
    const bool fours = g.rows % 4 == 0 && g.y_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(g.y) & 7) == 0;
    for (uint32_t o = threadIdx.x; o < g.row_tiles * NT * 64; o += blockDim.x) {
        const uint32_t r = o / (NT * 64), t = o / 64 % NT, l = o % 64, token = t0 + 16 * t + (l & 15), n = n0 + 16 * r + 4 * (l >> 4);
        if (token >= g.m || n >= g.rows) continue;
        f32x4 v = part[0][r][t][l];
        for (uint32_t q = 1; q < waves; q++) v += part[q][r][t][l];
        uint16_t *y = g.y + token * g.y_stride + n;
        if (fours) {
            *reinterpret_cast<uint64_t *>(y) = (uint64_t)Ty::from_f32(v[0]) | (uint64_t)Ty::from_f32(v[1]) << 16 |
                                               (uint64_t)Ty::from_f32(v[2]) << 32 | (uint64_t)Ty::from_f32(v[3]) << 48;
        } else {
#pragma unroll
            for (uint32_t e = 0; e < 4; e++)
                if (n + e < g.rows) y[e] = Ty::from_f32(v[e]);
        }
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
    const float step = bad ? nan32() : g.zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
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

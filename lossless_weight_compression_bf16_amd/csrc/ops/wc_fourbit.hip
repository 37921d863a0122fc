// wc_fourbit.hip -- C ABI of the products with weights of 4 bits (see
// include/wc.h): argument checks and launch shapes; like the other calls these only
// enqueue on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wc.h"
#include "ops_common.hpp"
#include "ops_fourbit.hpp"
#include "ops_host.hpp"

using namespace wc::ops;

namespace {

bool valid_fourbit(uint64_t rows, uint32_t cols, uint32_t group)
{
    return (group == 32 || group == 64 || group == 128) && rows >= 1 && rows <= (1u << 24) && cols >= group && cols % group == 0 &&
           cols <= (1u << 20);
}

template <int T, int GROUP, int NT, int SLICE, int WAVES>
void launch_linear4(Linear4Args g, hipStream_t stream)
{
    const uint64_t tiles = ceil_div(g.rows, 16), turns = ceil_div(g.m, 16 * NT), slices = ceil_div(g.cols, SLICE);
    const uint32_t waves = (uint32_t)(slices < WAVES ? slices : WAVES);
    // a block for each compute unit, whose LDS has room for one, and as many for each XCD, which has 32 units (14336 x 4096, groups
    // of 64: 65 rows, 85 blocks a turn are 33 on two XCDs, 75 us, 80 are 30 at most, 44; 129 rows 119 and 64, 224 rows 161 and 91)
    const uint64_t each = turns < kCus ? kCus / turns : 1, blocks = each < 8 ? each : each / 8 * 8;
    g.row_tiles = (uint32_t)ceil_div(tiles, blocks);
    if (g.row_tiles > kRowTiles4) g.row_tiles = kRowTiles4;
    g.row_blocks = (uint32_t)ceil_div(tiles, g.row_tiles);
    const dim3 grid((uint32_t)(8 * ceil_div(g.row_blocks, 8) * turns)), block(64 * waves);
    if (g.zeros) hipLaunchKernelGGL((k_linear4<T, GROUP, NT, SLICE, WAVES, true>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_linear4<T, GROUP, NT, SLICE, WAVES, false>), grid, block, 0, stream, g);
}

template <int T, int GROUP>
void launch_linear4(const Linear4Args &g, hipStream_t stream)
{
    // A wave takes 256 columns, or as many as a group has where there are not so many.  Rows of x: 16 by 16 waves, whose registers
    // hold no more, and from 17 on 32 by 8 (4096 x 4096, groups of 64: 17 rows 10.2 us against 17.7 as two times
    // 16, 64 rows 12.8 against 32; with 64 rows at once a wave has room for 128 columns only: 17.4).
    if (g.cols < 256) launch_linear4<T, GROUP, 1, GROUP, 8>(g, stream);
    else if (g.m <= 16) launch_linear4<T, GROUP, 1, 256, 16>(g, stream);
    else launch_linear4<T, GROUP, 2, 256, 8>(g, stream);
}

template <int T>
void launch_linear4(const Linear4Args &g, uint32_t group, hipStream_t stream)
{
    if (group == 32) launch_linear4<T, 32>(g, stream);
    else if (group == 64) launch_linear4<T, 64>(g, stream);
    else launch_linear4<T, 128>(g, stream);
}

template <int T>
void launch_quantize4(const Quantize4Args &g, uint32_t group, hipStream_t stream)
{
    const dim3 grid((uint32_t)ceil_div(g.rows * (g.cols / 8), 256)), block(256);
    if (group == 32) hipLaunchKernelGGL((k_quantize4<T, 32>), grid, block, 0, stream, g);
    else if (group == 64) hipLaunchKernelGGL((k_quantize4<T, 64>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_quantize4<T, 128>), grid, block, 0, stream, g);
}

}  // namespace

extern "C" {

wc_status wc_linear4(const wc_fourbit *a, hipStream_t stream)
{
    if (!a || (a->type != WC_T_BF16 && a->type != WC_T_FP16) || !valid_fourbit(a->rows, a->cols, a->group) || a->m > kMaxRows)
        return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (!a->x || !aligned(a->x, 16) || (a->m > 1 && (a->x_stride < a->cols || a->x_stride % 8))) return WC_ERR_ARG;
    if (!a->q || !aligned(a->q, 16) || !a->scales || !aligned(a->scales, 2) || !aligned(a->zeros, 2)) return WC_ERR_ARG;
    if (!a->y || !aligned(a->y, 2) || (a->m > 1 && a->y_stride < a->rows)) return WC_ERR_ARG;
    if (!rows_apart(a->x, 2 * a->x_stride, 2ull * a->cols, a->y, 2 * a->y_stride, 2ull * a->rows, a->m)) return WC_ERR_ARG;
    const uint64_t groups = 2ull * a->rows * (a->cols / a->group);
    if (!apart(rows_of(a->y, a->y_stride, a->rows, a->m), line(a->q, (uint64_t)a->rows * a->cols / 2), line(a->scales, groups),
               line(a->zeros, groups)))
        return WC_ERR_ARG;
    // blocks of 32 sixteens of rows, or fewer where that makes no more blocks than compute units; every XCD the same number
    if ((ceil_div(a->rows, 16 * kRowTiles4) + 16) * ceil_div(a->m, 16) + kCus > max_blocks(1024)) return WC_ERR_ARG;
    Linear4Args g{};
    g.x = static_cast<const uint16_t *>(a->x);
    g.q = static_cast<const uint8_t *>(a->q);
    g.scales = static_cast<const uint16_t *>(a->scales);
    g.zeros = static_cast<const uint16_t *>(a->zeros);
    g.y = static_cast<uint16_t *>(a->y);
    g.x_stride = a->x_stride;
    g.q_row = a->cols / 2;
    g.y_stride = a->y_stride;
    g.m = (uint32_t)a->m;
    g.rows = a->rows;
    g.cols = a->cols;
    g.groups = a->cols / a->group;
    if (a->type == WC_T_BF16) launch_linear4<WC_T_BF16>(g, a->group, stream);
    else launch_linear4<WC_T_FP16>(g, a->group, stream);
    return launched();
}

wc_status wc_quantize4(const void *w, uint64_t w_stride, uint64_t rows, uint32_t cols, uint32_t group, uint32_t type, void *q,
                       void *scales, void *zeros, hipStream_t stream)
{
    if ((type != WC_T_BF16 && type != WC_T_FP16) || !valid_fourbit(rows, cols, group)) return WC_ERR_ARG;
    if (!w || !aligned(w, 2) || (rows > 1 && w_stride < cols) || !q || !aligned(q, 16) || !scales || !aligned(scales, 2) ||
        !aligned(zeros, 2) || ceil_div(rows * (cols / 8), 256) > max_blocks(256))
        return WC_ERR_ARG;
    const Rows from = rows_of(w, w_stride, cols, rows), to = line(q, rows * cols / 2), s = line(scales, 2 * rows * (cols / group)),
               z = line(zeros, 2 * rows * (cols / group));
    if (!apart(from, to, s, z) || !apart(to, s, z) || !apart(s, z)) return WC_ERR_ARG;
    const Quantize4Args g{static_cast<const uint16_t *>(w), w_stride, static_cast<uint8_t *>(q), static_cast<uint16_t *>(scales),
                          static_cast<uint16_t *>(zeros), rows, cols};
    if (type == WC_T_BF16) launch_quantize4<WC_T_BF16>(g, group, stream);
    else launch_quantize4<WC_T_FP16>(g, group, stream);
    return launched();
}

}  // extern "C"

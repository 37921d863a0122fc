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

template <int T, int GROUP>
void launch_linear4(Linear4Args g, hipStream_t stream)
{
    // enough sixteens of rows for a block that all have a compute unit
    const uint64_t tiles = ceil_div(g.rows, 16);
    g.row_tiles = (uint32_t)ceil_div(tiles, kCus);
    if (g.row_tiles > kRowTiles4) g.row_tiles = kRowTiles4;
    g.row_blocks = (uint32_t)ceil_div(tiles, g.row_tiles);
    const uint32_t slices = (uint32_t)ceil_div(g.cols, kSlice4);
    const bool one = g.m <= 16;
    constexpr int kOne = GROUP == 32 ? 8 : 16;  // waves: groups of 32 take registers for their scales
    const uint32_t most = one ? kOne : 8, waves = slices < most ? slices : most;
    const dim3 grid((uint32_t)(8 * ceil_div(g.row_blocks, 8) * ceil_div(g.m, one ? 16 : 32))), block(64 * waves);
    if (one) hipLaunchKernelGGL((k_linear4<T, GROUP, 1, kOne>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_linear4<T, GROUP, 2, 8>), grid, block, 0, stream, g);
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
    if (8 * ceil_div(ceil_div(a->rows, 16), 8) * ceil_div(a->m, 16) > max_blocks(1024)) return WC_ERR_ARG;
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
    const Quantize4Args g{static_cast<const uint16_t *>(w), w_stride, static_cast<uint8_t *>(q), static_cast<uint16_t *>(scales),
                          static_cast<uint16_t *>(zeros), rows, cols};
    if (type == WC_T_BF16) launch_quantize4<WC_T_BF16>(g, group, stream);
    else launch_quantize4<WC_T_FP16>(g, group, stream);
    return launched();
}

}  // extern "C"

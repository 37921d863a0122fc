// ops_deal.hpp -- how the tiles of a grouped product are dealt to the blocks of
// a launch: plain arithmetic, the same on the host, where it can be enumerated.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define WC_ANYWHERE __host__ __device__ __forceinline__
#else
#define WC_ANYWHERE inline
#endif

namespace wc {
namespace ops {

enum PieceKind : uint32_t {
    kWhole,   // a tile
    kPart,    // a part along k of one of the last tiles
    kZeros,   // a tile of the rows behind the last expert's, only to be zeros
    kHole,    // nothing, but pieces of this block may come after it
    kNoMore,  // nothing, and nothing after it
};

// As many whole tiles as fill the `slots` (a multiple of 8) some number of times; the tiles that are
// left, if they would leave half of the slots or more without one, in parts along k;
// then tiles of zeros.  Block b's pieces are b, b + grid and so on (both of them
// multiples of 8 apart): of each kind every XCD (b % 8) has a contiguous range, and
// where a kind's pieces are no multiple of 8, the last of these ranges end in holes.
struct Dealing {
    uint32_t whole, left, splits, zeros;

    WC_ANYWHERE static Dealing of(uint32_t tiles, uint32_t stages, uint32_t slots, bool parts, uint32_t zeros)
    {
        Dealing d;
        d.whole = tiles / slots * slots;
        d.left = tiles - d.whole;
        d.splits = 1;
        if (parts && d.left) {  // at least 8 stages in a part
            const uint32_t each = slots / d.left, most = stages / 8 < 16 ? stages / 8 : 16;
            d.splits = each < most ? each : most;
            if (d.splits < 1) d.splits = 1;
        }
        d.zeros = zeros;
        return d;
    }
    // Piece b, and its number t among those of its kind.
    WC_ANYWHERE PieceKind piece(uint32_t b, uint32_t &t) const
    {
        uint32_t at = b / 8;
        if (at < whole / 8) {
            t = b % 8 * (whole / 8) + at;
            return kWhole;
        }
        at -= whole / 8;
        const uint32_t parts = (left * splits + 7) / 8, behind = (zeros + 7) / 8;
        if (at < parts) {
            t = b % 8 * parts + at;
            return t < left * splits ? kPart : kHole;
        }
        at -= parts;
        t = b % 8 * behind + at;
        return at >= behind ? kNoMore : t < zeros ? kZeros : kHole;
    }
    // The next piece of a block that has had `turn` of its places; kNoMore when there is none.
    WC_ANYWHERE PieceKind next(uint32_t block, uint32_t grid, uint32_t &turn, uint32_t &t) const
    {
        for (;; turn++) {
            const PieceKind kind = piece(block + turn * grid, t);
            if (kind == kHole) continue;
            if (kind != kNoMore) turn++;
            return kind;
        }
    }
};

}  // namespace ops
}  // namespace wc

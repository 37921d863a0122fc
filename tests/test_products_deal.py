"""How the tiles of a grouped product are dealt to the blocks of a launch,
enumerated on the host from the kernels' own text: every whole tile, every
part and every tile of zeros exactly once, by blocks that take one piece and by
blocks that take one after the other."""
import os
import shutil
import subprocess

import pytest

from lossless_weight_compression_bf16_amd import build as W

SOURCE = r"""
#include <stdint.h>
#include <stdio.h>
#include <algorithm>
#include <random>
#include <vector>
#include "ops_deal.hpp"
using namespace wc::ops;

static long cases = 0;

// The pieces that `grid` blocks take, or the first one that is not taken once.
static int check(uint32_t tiles, uint32_t stages, uint32_t slots, bool parts, uint32_t zeros, uint32_t grid)
{
    const Dealing d = Dealing::of(tiles, stages, slots, parts, zeros);
    const uint32_t sizes[3] = {d.whole, d.left * d.splits, d.zeros};
    std::vector<uint32_t> had[3];
    for (int q = 0; q < 3; q++) had[q].assign(sizes[q], 0);
    bool ok = d.whole + d.left == tiles && d.splits >= 1 && (d.splits == 1 || d.left * d.splits <= slots) && d.zeros == zeros;
    for (uint32_t b = 0; b < grid; b++) {
        uint32_t turn = 0, t = 0;
        for (PieceKind kind; (kind = d.next(b, grid, turn, t)) != kNoMore;) {
            if (kind > kZeros || t >= sizes[kind]) ok = false;
            else had[kind][t]++;
        }
        ok = ok && d.next(b, grid, turn, t) == kNoMore;  // and stays so
    }
    cases++;
    uint32_t wrong = 0;
    for (auto &h : had)
        for (uint32_t n : h) wrong += n != 1;
    if (!ok || wrong) {
        printf("%u tiles of %u stages, %u slots, %s, %u of zeros, %u blocks: %u pieces of %u + %u + %u not had once\n", tiles, stages,
               slots, parts ? "parts" : "whole", zeros, grid, wrong, sizes[0], sizes[1], sizes[2]);
        return 1;
    }
    return 0;
}

int main()
{
    std::mt19937 rng(7);
    auto upto = [&](uint32_t n) { return (uint32_t)(rng() % (n + 1)); };
    int bad = 0;
    // experts of 2000 and 2100 rows and 20000 rows behind, 4104 x 136: 17 rows of tiles of 256 by 17, and 79 by 17 of zeros
    bad += check(17 * 17, 3, 256, false, 79 * 17, 256);
    // seven experts of 1000 rows and 9384 behind, 7176 x 4096
    bad += check(28 * 29, 64, 256, true, 37 * 29, 256);
    for (int n = 0; n < 4000 && bad < 5; n++) {
        const uint32_t slots = n % 2 ? 256 : 512, tiles = upto(n % 3 ? 4 * slots : 40), stages = upto(300);
        const uint32_t zeros = n % 5 ? upto(n % 3 ? 3000 : 20) : 0, grid = 8 * (1 + upto(40));
        const bool parts = n % 7 < 4;
        // one block after the other, from any number of blocks, and a block for every place
        const uint32_t all = 8 * ((tiles + (parts ? slots : 0) + zeros + 7) / 8 + 3);
        bad += check(tiles, stages, slots, parts, zeros, std::min(256u, all));
        bad += check(tiles, stages, slots, parts, zeros, grid);
        bad += check(tiles, stages, slots, parts, zeros, all);
    }
    printf("%ld cases\n", cases);
    return bad ? 1 : 0;
}
"""


def test_every_piece_once(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    (tmp_path / "deal.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{os.path.join(W.CSRC, 'ops')}", str(tmp_path / "deal.cpp"), "-o", str(tmp_path / "deal")], check=True)
    r = subprocess.run([str(tmp_path / "deal")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert "12002 cases" in r.stdout


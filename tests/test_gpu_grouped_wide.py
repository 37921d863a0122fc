"""Few rows of experts with many weights and short rows, which go by tiles of 64
rows as those with long ones do.

Tolerances: as in test_gpu_grouped.py."""
import pytest

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
import test_gpu_grouped as GR  # noqa: E402
from test_gpu_grouped import BF, HF, dev  # noqa: E402, F401


def test_which_experts_go_by_tiles():
    """Scratch for the last round's parts, at k = 1024, is the tiles' alone."""
    L = wc.lib()
    for rows in (1, 2, 8):
        assert L.wc_grouped_linear_scratch(16 * rows, 16, 4096, 1024) == 0  # 2^26 weights
        assert L.wc_grouped_linear_scratch(17 * rows, 17, 4096, 1024) > 0
        assert L.wc_grouped_linear_scratch(rows, 4096, 4096, 1024) == 0     # no experts of that number
    assert L.wc_grouped_linear_scratch(16, 64, 4096, 1024) == 0             # 16 of 64 experts can have rows


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,rows,cols", [([1] * 34, 8200, 264), ([8] * 34, 8200, 264), ([0, 1, 2, 20, 0, 30, 1, 1] * 5, 2056, 1016),
                                              ([2] * 300, 904, 264), ([1, 0, 9, 3], 20008, 1024)])
def test_against_64_bits(dev, dtype, counts, rows, cols):  # noqa: F811
    GR._check(counts, 0, rows, cols, dtype, dev)
    GR._check(counts, 5, rows, cols, dtype, dev)


@pytest.mark.gpu
def test_masks_and_strides(dev):  # noqa: F811
    counts, rows, cols = [3, 8, 5], 30008, 1000
    GR.test_what_is_not_read_does_not_matter(dev, [3, 0, 5], 9, rows, cols)
    GR.test_a_row_of_infinities_and_nan_stays_alone(dev, counts, rows, cols)
    GR.test_strides_and_alignment(dev, counts, rows, cols)
    GR.test_out_keeps_what_is_behind(dev, counts, rows, cols)

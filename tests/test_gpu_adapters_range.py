"""Adapters whose scaled A x is near the end of fp32's range, or far below
half precision's: it is held in 32 bits, and y as well, so y is the formula's.
Tolerances and the formula are those of test_gpu_adapters.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from test_gpu_adapters import BF, F32, HF, _check, _inputs  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


# one launch, two, two for the blocks of ranks, three
@pytest.mark.parametrize("m,n,rank", [(1, 2, 16), (40, 2, 24), (40, 2, 100), (600, 3, 24), (600, 3, 100)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("power", [116, 110, 60, -60, -80])
def test_scales_of_any_size(dev, dtype, m, n, rank, power):
    """u = s A x of about 2^(power + 8), in y through B of 2^-10."""
    x, y, a, b, ids, s = _inputs(m, n, rank, 256, 64, dtype, F32, m + rank)
    ids.clamp_(min=0)
    x, b = (x * 2.0 ** 8).to(dtype), (b * 2.0 ** -10).to(dtype)
    y.zero_()
    _check((x, y, a, b, ids, s * 2.0 ** power), dev, f"{dtype} {m} tokens, rank {rank}, scales 2^{power}")

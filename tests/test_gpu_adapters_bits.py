"""What the adapters keep of u = s A x.

The cases' numbers are whole, so that u is exact in fp32: a whole number below
2^21.  A row of B takes the difference of two values of u, -7..7, which is
exact in every type of y, if u is kept whole, and off by several where u keeps
16 bits.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import adapters as A  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _whole(m, n, rank, cols, rows, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(30, 91, (m, cols), generator=g).double()
    x[:, 0] = torch.randint(-7, 8, (m,), generator=g)
    half = rank // 2
    a = torch.randint(30, 91, (n, rank, cols), generator=g).double()
    a[:, half:2 * half] = a[:, :half]
    a[:, half:, 0] += 1.0  # u of the second half is the first half's and x[0]
    at = torch.randint(0, half, (n, rows, 1), generator=g)
    sign = (torch.randint(0, 2, (n, rows, 1), generator=g) * 2 - 1).double()
    b = torch.zeros((n, rows, rank), dtype=torch.float64).scatter_(2, at, -sign).scatter_(2, at + half, sign)
    ids = torch.randint(-1, n, (m,), generator=g).sort().values
    want = x[:, :1] * sign[ids.clamp(min=0), :, 0] * (ids >= 0)[:, None]
    assert float((x @ a.flatten(0, 1).T).max()) < 2.0 ** 21
    return x, a, b, ids, want


# one launch, two, two for blocks of ranks, three; partial tiles and ranks
@pytest.mark.parametrize("m,n,rank,rows", [(1, 1, 16, 64), (3, 2, 20, 65), (61, 5, 50, 1100), (70, 30, 16, 300),
                                           (70, 3, 130, 70), (300, 200, 24, 96), (600, 3, 24, 300), (600, 3, 64, 130),
                                           (520, 2, 200, 96)])
@pytest.mark.parametrize("dtype,ydtype", [(BF, F32), (BF, BF), (HF, F32), (HF, HF)])
def test_u_is_kept_whole(dev, dtype, ydtype, m, n, rank, rows):
    print(f"[adapters bits] {dtype} {ydtype} {m} tokens of {n}, rank {rank}, {rows} rows", flush=True)
    sys.stdout.flush()
    x, a, b, ids, want = _whole(m, n, rank, 232, rows, m + rank)
    xd, ad, bd = (t.to(dtype).to(dev) for t in (x, a, b))
    assert all(torch.equal(d.double().cpu(), t) for d, t in zip((xd, ad, bd), (x, a, b)))
    y = A.add_adapters(xd, torch.zeros((m, rows), dtype=ydtype, device=dev), ad, bd, ids.to(dev))
    assert torch.equal(y.double().cpu(), want)

"""The products by tiles of 64 rows, which are taken where there are few rows
and more than 2^26 weights, and by smaller ones beside them: the masks, edges and odd sizes at which tiles can go
wrong, with the tolerances of the other sizes' tests."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_grouped as GR  # noqa: E402
import test_gpu_loss as LO  # noqa: E402
from test_gpu_grouped import dev  # noqa: E402,F401

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import grouped as G, loss as L  # noqa: E402

BF, HF = torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")
# rows of an expert below, at and above whole tiles and sixteens; columns that end within a stage of 64, and weights
# with rows that end within a tile; the last two hold few enough weights at k > 1024 for k_grouped_few
RAGGED = [([1, 0, 64, 65, 16, 17], 2056, 5576), ([9] * 40, 520, 4104), ([0, 63, 0, 1, 128], 2056, 8200), ([48] * 3, 4104, 8192),
          ([9] * 40, 520, 2056), ([12, 0, 3], 136, 1032), ([5, 2, 9], 1040, 1096)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,rows,cols", RAGGED)
def test_grouped_against_64_bits(dev, dtype, counts, rows, cols):  # noqa: F811
    GR._check(counts, 0, rows, cols, dtype, dev)
    GR._check(counts, 7, rows, cols, dtype, dev)


@pytest.mark.parametrize("counts,rows,cols", [([20, 30, 11], 4104, 4104), ([60, 3, 17], 264, 100008), ([20, 30, 11], 264, 4104)])
def test_grouped_masks_and_strides(dev, counts, rows, cols):  # noqa: F811
    GR.test_what_is_not_read_does_not_matter(dev, [counts[0], 0, counts[2]], 9, rows, cols)
    GR.test_a_row_of_infinities_and_nan_stays_alone(dev, counts, rows, cols)
    GR.test_strides_and_alignment(dev, counts, rows, cols)
    GR.test_out_keeps_what_is_behind(dev, counts, rows, cols)


def test_grouped_ends_out_of_range(dev):  # noqa: F811
    m, rows, cols = 100, 4104, 4104  # 4 x 4104 x 4104 > 2^26
    x, w = torch.ones((m, cols), device=dev, dtype=BF), torch.ones((4, rows, cols), device=dev, dtype=BF)
    for ends in ([5, 3, 10, m], [1, 2, 3, m + 1], [-1, 2, 3, 4], [m, 0, m, 0], [1 << 40, -(1 << 40), 1 << 62, 5]):
        t = torch.tensor(ends, device=dev)
        with pytest.raises(wc.WcError, match="index out of range"):
            G.grouped_linear(x, w, t)
        with pytest.raises(wc.WcError, match="index out of range"):
            G.grouped_linear_backward(x, w, t, x)
        G.grouped_linear(x, w, t, check=False)
    torch.cuda.synchronize()
    y = G.grouped_linear(x, w, torch.tensor([5, 5, 10, m - 1], device=dev))
    assert bool((y[:-1] == torch.full((), cols, dtype=BF)).all()) and not bool(y[-1].any())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,v,k", [(17, 70001, 968), (18, 16411, 4104), (61, 20011, 3480), (64, 2 ** 18 + 3, 264), (33, 257, 4104), (63, 1, 1040)])
def test_loss_against_64_bits(dev, dtype, m, v, k):  # noqa: F811
    LO.test_against_64_bits(dev, dtype, m, v, k)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_loss_rows_without_a_part(dev, dtype):  # noqa: F811
    LO.test_rows_without_a_part(dev, dtype, 40, 70001, 1000)


def test_loss_infinities_and_nan(dev):  # noqa: F811
    m, k, v = 40, 1096, 70001
    h, w = torch.zeros((m, k), device=dev, dtype=BF), torch.ones((v, k), device=dev, dtype=BF)
    h[:, 0] = 1
    t = torch.full((m,), 5, device=dev)
    w[:, 0] = -INF                                  # every logit -inf (0 times 1 of the others)
    r = L.linear_cross_entropy(h, w, t)
    assert bool((r.lse == -INF).all()) and bool((r.loss == INF).all())
    w[5, 0] = 1                                     # every one but the token's: the loss is 0
    r = L.linear_cross_entropy(h, w, t)
    assert bool((r.lse == 1).all()) and bool((r.loss == 0).all())
    w[5, 0] = INF
    r = L.linear_cross_entropy(h, w, t)
    assert bool(r.lse.isnan().all()) and bool(r.loss.isnan().all())
    w[:, 0] = 1
    h[0] = NAN
    r = L.linear_cross_entropy(h, w, t)
    assert bool(r.lse[0].isnan()) and bool(r.lse[1:].isfinite().all())


def test_loss_strides_and_tokens(dev):  # noqa: F811
    m, v, k = 40, 70001, 1000
    h, w, t, gl, gz = LO._inputs(m, v, k, HF, dev)
    want = L.linear_cross_entropy(h, w, t)
    wh, ww = L.linear_cross_entropy_backward(h, w, t, want.lse, gl, gz)
    wide = torch.full((v, k + 16), NAN, device=dev, dtype=HF)
    wide[:, 8:8 + k] = w
    odd = torch.zeros(m * k + 1, device=dev, dtype=HF)
    odd[1:] = h.flatten()
    for z in (h.t().contiguous().t(), odd[1:].view(m, k)):
        r = L.linear_cross_entropy(z, wide[:, 8:8 + k], t)
        assert torch.equal(r.loss, want.loss) and torch.equal(r.lse, want.lse)
        gh, gw = L.linear_cross_entropy_backward(z, wide[:, 8:8 + k], t, want.lse, gl, gz)
        assert torch.equal(gh, wh) and torch.equal(gw, ww)
    t[2] = v
    with pytest.raises(wc.WcError, match="index out of range"):
        L.linear_cross_entropy(h, w, t)
    r = L.linear_cross_entropy(h, w, t, check=False)
    assert bool(r.loss[2].isnan()) and torch.equal(r.lse, want.lse) and torch.equal(r.loss[3:], want.loss[3:])

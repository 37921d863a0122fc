"""Products grouped by expert of no rows: ends past them raise, as they do where there are rows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import grouped as G  # noqa: E402
from test_gpu_grouped import BF, dev  # noqa: E402, F401


@pytest.mark.parametrize("ends", [[0, 3], [1, 0], [-1, 0], [0, 1 << 40], [0, -1]])
def test_ends_out_of_range(dev, ends):  # noqa: F811
    x, w, d = torch.empty((0, 24), device=dev, dtype=BF), torch.ones((2, 16, 24), device=dev, dtype=BF), torch.empty((0, 16), device=dev, dtype=BF)
    t = torch.tensor(ends, device=dev)
    with pytest.raises(wc.WcError, match="index out of range"):
        G.grouped_linear(x, w, t)
    with pytest.raises(wc.WcError, match="index out of range"):
        G.grouped_linear(x, w, t, out=d)
    with pytest.raises(wc.WcError, match="index out of range"):
        G.grouped_linear(x.clone().requires_grad_(), w, t)
    for need in ((True, True), (True, False), (False, True)):
        with pytest.raises(wc.WcError, match="index out of range"):
            G.grouped_linear_backward(x, w, t, d, *need)
    assert G.grouped_linear(x, w, t, check=False).shape == (0, 16)
    assert not bool(G.grouped_linear_backward(x, w, t, d, check=False)[1].any())


def test_ends_in_range(dev):  # noqa: F811
    x, w, d = torch.empty((0, 24), device=dev, dtype=BF), torch.ones((700, 16, 24), device=dev, dtype=BF), torch.empty((0, 16), device=dev, dtype=BF)
    t = torch.zeros(700, dtype=torch.int64, device=dev)
    assert G.grouped_linear(x, w, t).shape == (0, 16)
    dx, dw = G.grouped_linear_backward(x, w, t, d)
    assert dx.shape == (0, 24) and not bool(dw.any())
    t[699] = 1
    with pytest.raises(wc.WcError, match="index out of range"):
        G.grouped_linear(x, w, t)

"""The cross entropy of more rows than one set of its launches takes (32768): the
last set's rows by each of its kernels, against the definition in 64 bits.

Tolerances: as in test_gpu_loss.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import loss as L  # noqa: E402
from test_gpu_loss import BF, HF, _check_loss, _inputs, _say, dev  # noqa: E402, F401

SLICE = 1 << 15


# of the last rows: one, a few (k_loss_few, waves apart and together), tiles of 128, of 256, of 64 with the weights past the caches
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("behind,v,k", [(1, 301, 40), (2, 70, 1032), (16, 1003, 72), (40, 301, 72), (SLICE + 300, 301, 24),
                                        (SLICE - 1, 1003, 16), (2 * SLICE, 130, 16), (33, 65537, 1032)])
def test_last_rows(dev, dtype, behind, v, k):  # noqa: F811
    m = SLICE + behind
    _say(f"[slices] {dtype} {m} rows, {v} x {k}")
    h, w, t, _, _ = _inputs(m, v, k, dtype, dev)
    if m * v > 1 << 26:  # the first rows are others' to test: their tokens and values as in the last ones
        head = L.linear_cross_entropy(h, w, t)
        last = _check_loss(h[SLICE:], w, t[SLICE:], "last rows")
        assert torch.equal(head.lse[SLICE:], last.lse) and torch.equal(head.loss[SLICE:], last.loss)
        first = _check_loss(h[:64], w, t[:64], "first rows")
        assert float((head.lse[:64] - first.lse).abs().max()) < 1e-3
        return
    _check_loss(h, w, t, f"{m} rows")


@pytest.mark.parametrize("behind", [1, 40, SLICE + 300])
def test_tokens_out_of_range_in_the_last_rows(dev, behind):  # noqa: F811
    m, v = SLICE + behind, 50
    h, w, t, _, _ = _inputs(m, v, 16, BF, dev)
    good = L.linear_cross_entropy(h, w, t)
    for at in (SLICE, m - 1):
        for bad in (v, -2, 1 << 40):
            u = t.clone()
            u[at] = bad
            with pytest.raises(wc.WcError, match="index out of range"):
                L.linear_cross_entropy(h, w, u)
            r = L.linear_cross_entropy(h, w, u, check=False)
            rest = torch.arange(m, device=dev) != at
            assert bool(r.loss[at].isnan()) and torch.equal(r.lse, good.lse) and torch.equal(r.loss[rest], good.loss[rest])


def test_strides(dev):  # noqa: F811
    m, v, k = SLICE + 300, 301, 24
    h, w, t, _, _ = _inputs(m, v, k, HF, dev)
    want = L.linear_cross_entropy(h, w, t)
    wide = torch.full((m, k + 16), float("nan"), device=dev, dtype=HF)
    wide[:, 8:8 + k] = h
    r = L.linear_cross_entropy(wide[:, 8:8 + k], w, torch.stack([t, t], 1)[:, 0])
    assert torch.equal(r.loss, want.loss) and torch.equal(r.lse, want.lse)

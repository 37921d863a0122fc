"""Rows behind the last expert's where there are many of them, so that a block of the
large tiles has tiles of zeros to write after its own: y and the gradient of x
are zeros there, and what the definition gives before.

Tolerance: as in test_gpu_grouped.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from lossless_weight_compression_bf16_amd import grouped as G  # noqa: E402
from test_gpu_grouped import BF, HF, NAN, _groups, _inputs, _near, _say, dev  # noqa: E402, F401


def _filled(*shape, dtype, dev):
    """Memory that the call's result will be given, full of NaN."""
    t = torch.full(shape, NAN, dtype=dtype, device=dev)
    del t


# the number of tiles, and of their parts, is no multiple of 8, and there are more than 256 tiles of zeros
@pytest.mark.parametrize("counts,rest,rows,cols", [
    ([2000, 2100], 20000, 4104, 136),      # y: 17 x 17 tiles, 33 of them in the last round, and 79 x 17 of zeros
    ([2000, 2100], 20000, 136, 4104),      # the same for the gradient of x
    ([1000] * 7, 9384, 7176, 1032),        # 28 x 29 tiles, of which 44 in parts along k
    ([1000] * 7, 9384, 1032, 7176),
    ([1900, 0, 2300, 1], 8192, 2056, 2056),
])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_many_rows_behind(dev, dtype, counts, rest, rows, cols):  # noqa: F811
    used = sum(counts)
    _say(f"[behind] {dtype} {counts} + {rest} rows, {rows} x {cols}")
    x, w, ends, dy = _inputs(counts, rest, rows, cols, dtype, dev)
    x[used:] = dy[used:] = NAN
    _filled(used + rest, rows, dtype=dtype, dev=dev)
    y = G.grouped_linear(x, w, ends)
    assert not bool(y[used:].any()), "y behind"
    _filled(used + rest, cols, dtype=dtype, dev=dev)
    dx, dw = G.grouped_linear_backward(x, w, ends, dy)
    assert not bool(dx[used:].any()), "gradient of x behind"
    for e, at in _groups(counts):
        if at.start == at.stop:
            assert not bool(dw[e].any())
            continue
        a, b, d = x[at].double(), w[e].double(), dy[at].double()
        _near(y[at], a @ b.T, a.abs() @ b.abs().T, cols, f"y of expert {e}")
        _near(dx[at], d @ b, d.abs() @ b.abs(), rows, f"gradient of x of expert {e}")
        _near(dw[e], d.T @ a, d.abs().T @ a.abs(), a.shape[0], f"gradient of expert {e}")
    out = torch.full_like(y, 5.0)
    assert G.grouped_linear(x, w, ends, out=out) is out
    assert torch.equal(out[:used], y[:used]) and bool((out[used:] == 5).all())
    # and through autograd
    x, w = x.requires_grad_(), w.requires_grad_()
    _filled(used + rest, rows, dtype=dtype, dev=dev)
    r = G.grouped_linear(x, w, ends)
    assert torch.equal(r, y)
    del y
    r.backward(dy)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)

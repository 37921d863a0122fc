"""The gradients of the cross entropy where the gradient of the logits, G, is held
whole: as near to the definition in 64 bits as their own single rounding lets
them be; and, with `rounded`, as near as one more rounding lets them be.

Tolerances.  Each element: as in test_gpu_loss.py, but for G, which in two
terms is off by 2^-16 of its size in BF16 (half a step of what half a step
leaves), by 2^-22 in FP16, or by 2^-39 of the largest row's gradient.  All
elements together: the correctly rounded gradient's own distance from the exact
one, which the test has, is D in the root mean square; an error d before the
rounding makes sqrt(D^2 + d^2) of it.  D is 0.17% in BF16 and 0.021% in FP16;
d, of logits whose sums of k <= 768 products are off like a random walk, by
sqrt(k) 2^-24 |z| < 1e-5 for |z| < 6, is below 3e-5, and 1% more than D leaves
room for 0.14 D = 2.9e-5 in FP16.  A G rounded once adds 0.1 and 0.01%: 13% or more."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from lossless_weight_compression_bf16_amd import _binding as B, loss as L  # noqa: E402
from test_gpu_loss import BF, EPS, HF, INF, NAN, _check_gradient, _inputs, _near, _say, dev  # noqa: E402, F401


def _want(h, w, t, lse, gl, gz):
    """G, its possible error before any rounding to the type, and both gradients, in 64 bits."""
    k = h.shape[1]
    hd, wd = h.double(), w.double()
    z, size = hd @ wd.T, hd.abs() @ wd.abs().T
    of_token = torch.where(t < 0, 0.0, gl.double())
    of_lse = of_token + (gz.double() if gz is not None else 0)
    d = z - lse.double()[:, None]
    p = d.exp()
    g = p * of_lse[:, None]
    dg = g.abs() * ((k + 24) * EPS * size + (3 * d.abs() + 8) * EPS)
    hot = torch.zeros_like(g).scatter_(1, t.clamp(min=0)[:, None], 1.0) * (t >= 0)[:, None]
    g = g - of_token[:, None] * hot
    dg += 2 * EPS * (g.abs() + of_lse.abs()[:, None] * p)
    most = float(torch.maximum(of_token.abs(), of_lse.abs()).max())
    return g, dg, most, g @ wd, g.T @ hd


def _rms(t):
    return float(t.square().mean().sqrt())


def _check_whole(h, w, t, lse, gl, gz, what):
    f = torch.finfo(h.dtype)
    g, dg, most, want_h, want_w = _want(h, w, t, lse, gl, gz)
    dg = dg + (2.0 ** -16 * g.abs() if h.dtype == BF else 2.0 ** -22 * g.abs() + 2.0 ** -39 * most)
    got = L.linear_cross_entropy_backward(h, w, t, lse, gl, gz)
    for got, want, off, n, sizes, name in ((got[0], want_h, dg @ w.double().abs(), w.shape[0], g.abs() @ w.double().abs(), "hidden"),
                                           (got[1], want_w, dg.T @ h.double().abs(), h.shape[0], g.abs().T @ h.double().abs(), "weight")):
        off = off + (n + 24) * EPS * sizes
        _near(got, want, off + (f.eps / 2) * 1.01 * (want.abs() + off) + f.tiny * f.eps, f"{what}, {name}")
        own, had = _rms(want.to(h.dtype).double() - want), _rms(got.double() - want)
        _say(f"[whole]   {name}: {had / _rms(want):.3e} off, the correctly rounded one {own / _rms(want):.3e}")
        assert had <= 1.01 * own, f"{what}, {name}: {had / own} of the correctly rounded one's"


SIZES = [(8, 5003, 264), (16, 3001, 768), (40, 9001, 264), (61, 70001, 520), (100, 5021, 768), (129, 2003, 136), (300, 4003, 328),
         (1000, 3007, 96)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,v,k", SIZES)
def test_as_near_as_one_rounding(dev, dtype, m, v, k):  # noqa: F811
    what = f"{dtype} {m} rows, {v} x {k}"
    _say(f"[whole] {what}")
    h, w, t, gl, gz = _inputs(m, v, k, dtype, dev)
    lse = L.linear_cross_entropy(h, w, t).lse
    gl, gz = 1024 * gl, 1024 * gz  # so that the smallest gradients are no subnormal numbers
    _check_whole(h, w, t, lse, gl, gz, what)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_tiles_and_pieces(dev, dtype):  # noqa: F811
    """Tiles of 256 x 256, and more than one piece of the vocabulary."""
    for m, v, k in ((2100, 30011, 136), (9000, 20003, 24)):
        _say(f"[whole] {dtype} {m} rows, {v} x {k}")
        h, w, t, gl, gz = _inputs(m, v, k, dtype, dev)
        _check_whole(h, w, t, L.linear_cross_entropy(h, w, t).lse, 1024 * gl, 1024 * gz, f"{dtype} {m} rows, {v} x {k}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,v,k", [(8, 1003, 64), (61, 70001, 520), (100, 1001, 520), (2100, 12011, 136), (9000, 40003, 24)])
def test_rounded(dev, dtype, m, v, k, monkeypatch):  # noqa: F811
    """G as one number: test_gpu_loss.py's tolerances, which have room for its rounding."""
    _say(f"[rounded] {dtype} {m} rows, {v} x {k}")
    h, w, t, gl, gz = _inputs(m, v, k, dtype, dev)
    lse = L.linear_cross_entropy(h, w, t).lse
    whole = L.linear_cross_entropy_backward
    monkeypatch.setattr(L, "linear_cross_entropy_backward", lambda *a: whole(*a, rounded=True))
    got = _check_gradient(h, w, t, lse, gl, gz, f"rounded, {dtype} {m} rows, {v} x {k}")
    monkeypatch.undo()
    assert not all(torch.equal(a, b) for a, b in zip(got, L.linear_cross_entropy_backward(h, w, t, lse, gl, gz)))
    x, y = h.clone().requires_grad_(), w.clone().requires_grad_()
    r = L.linear_cross_entropy(x, y, t, rounded=True)
    ((gl * r.loss).sum() + (gz * r.lse).sum()).backward()
    assert torch.equal(x.grad, got[0]) and torch.equal(y.grad, got[1])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m", [5, 40, 300])
def test_infinities_in_gradients_stay(dev, dtype, m):  # noqa: F811
    """A gradient of the loss that is an infinity: what the formula has of it, an infinity of its sign and no NaN, where
    nothing else is one."""
    v, k = 300, 64
    h = torch.ones((m, k), device=dev, dtype=dtype)
    w = torch.zeros((v, k), device=dev, dtype=dtype)
    w[:, 0] = 1.0
    t = torch.full((m,), -1, device=dev)
    lse = L.linear_cross_entropy(h, w, t).lse
    gz = torch.zeros(m, device=dev)
    gz[1] = INF
    for rounded in (False, True):
        dh, dw = L.linear_cross_entropy_backward(h, w, t, lse, None, gz, rounded=rounded)
        assert bool((dh[1, 0] == INF).all()) and not bool(dh[0].any()) and not bool(dh[2:].any())
        assert bool((dw == INF).all())
        gz[1] = NAN
        dh, dw = L.linear_cross_entropy_backward(h, w, t, lse, None, gz, rounded=rounded)
        assert bool(dh[1].isnan().all()) and not bool(dh[0].any()) and bool(dw.isnan().all())
        gz[1] = INF


def test_rounded_through_the_binding(dev):  # noqa: F811
    m, v, k = 70, 900, 64
    h, w, t, gl, gz = _inputs(m, v, k, BF, dev)
    lse = L.linear_cross_entropy(h, w, t).lse
    need = B.wc_linear_cross_entropy_backward_scratch(m, v, k)
    scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    for rounded in (0, 1):
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        B.wc_linear_cross_entropy_backward(B.wc_linear_loss_grad(
            h.data_ptr(), k, w.data_ptr(), k, t.data_ptr(), lse.data_ptr(), gl.data_ptr(), gz.data_ptr(), dh.data_ptr(), k,
            dw.data_ptr(), m, v, k, B.WC_T_BF16, rounded), scratch, need)
        a, b = L.linear_cross_entropy_backward(h, w, t, lse, gl, gz, rounded=bool(rounded))
        assert torch.equal(a, dh) and torch.equal(b, dw)


@pytest.mark.parametrize("m", [3, 90, 700])
def test_captured(dev, m):  # noqa: F811
    """Replayed several times, with other calls between, on the memory of one pool."""
    h, w, t, gl, gz = _inputs(m, 3001, 136, BF, dev)
    lse = L.linear_cross_entropy(h, w, t).lse
    want = L.linear_cross_entropy_backward(h, w, t, lse, gl, gz)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.linear_cross_entropy_backward(h, w, t, lse, gl, gz, check=False)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = L.linear_cross_entropy_backward(h, w, t, lse, gl, gz, check=False)
    for _ in range(3):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        L.linear_cross_entropy_backward(h, w, t, lse, gl, None)

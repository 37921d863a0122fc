"""Products grouped by expert over ragged rows, and their gradients, against
their definition in 64 bits.

Tolerance.  A product of n exact terms summed in fp32, in any order, is off by
at most (n + 24) 2^-24 times the sum of their sizes (the 24 for sums that are
joined), and its one rounding to the type by half a step of it, or of the
smallest number.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import grouped as G  # noqa: E402

EPS = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _near(got, want, size, n, what):
    f = torch.finfo(got.dtype)
    tol = (n + 24) * EPS * size + (f.eps / 2) * want.abs() * 1.01 + f.tiny * f.eps
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).nan_to_num(9e9).max())} of its tolerance"


def _inputs(counts, rest, rows, cols, dtype, dev, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    m = sum(counts) + rest

    def n(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)
    ends = torch.tensor(counts, device=dev).cumsum(0)
    return n(m, cols), n(len(counts), rows, cols, std=cols ** -0.5), ends, n(m, rows)


def _groups(counts):
    lo = 0
    for e, n in enumerate(counts):
        yield e, slice(lo, lo + n)
        lo += n


def _expect(x, w, counts, dy):
    """y, dx and dw in 64 bits, each with the sum of its terms' sizes."""
    m, (_, rows, cols) = x.shape[0], w.shape
    z = dict(dtype=torch.float64, device=x.device)
    y, ys, dx, dxs = torch.zeros((m, rows), **z), torch.zeros((m, rows), **z), torch.zeros((m, cols), **z), torch.zeros((m, cols), **z)
    dw, dws = torch.zeros(w.shape, **z), torch.zeros(w.shape, **z)
    for e, at in _groups(counts):
        if at.start == at.stop:
            continue
        a, b, d = x[at].double(), w[e].double(), dy[at].double()
        y[at], ys[at] = a @ b.T, a.abs() @ b.abs().T
        dx[at], dxs[at] = d @ b, d.abs() @ b.abs()
        dw[e], dws[e] = d.T @ a, d.abs().T @ a.abs()
    return (y, ys), (dx, dxs), (dw, dws)


def _check(counts, rest, rows, cols, dtype, dev, args=None):
    what = f"{dtype} {counts[:12]}{'...' if len(counts) > 12 else ''} + {rest} rows, {rows} x {cols}"
    _say(f"[grouped] {what}")
    x, w, ends, dy = args or _inputs(counts, rest, rows, cols, dtype, dev)
    (y, ys), (dx, dxs), (dw, dws) = _expect(x, w, counts, dy)
    got = G.grouped_linear(x, w, ends)
    assert got.dtype == dtype and got.shape == y.shape
    _near(got, y, ys, cols, what + ", y")
    _say("[grouped]   gradient")
    gx, gw = G.grouped_linear_backward(x, w, ends, dy)
    _near(gx, dx, dxs, rows, what + ", dx")
    most = max(counts)
    _near(gw, dw, dws, most, what + ", dw")
    for t, behind in ((got, sum(counts)), (gx, sum(counts))):
        assert not bool(t[behind:].any())
    return got, gx, gw


FEW = [([1], 8, 8), ([0, 1, 0], 16, 24), ([3, 0, 5, 64, 65], 40, 264), ([1] * 9, 1024, 2048), ([2, 1, 15, 16, 17, 33, 0], 72, 1032),
       ([48] * 3, 136, 2304), ([0, 0, 140, 0, 1, 1], 24, 40), ([1, 0] * 150, 16, 32), ([1] * 1024, 8, 16), ([63, 1], 520, 768)]
MANY = [([49], 8, 8), ([200, 0, 1, 300], 136, 520), ([64, 128, 127, 129], 256, 64), ([257, 255, 1, 700], 264, 1032),
        ([1000], 72, 2048), ([0, 0, 500], 128, 128), ([130] * 40, 40, 72), ([3000, 0, 50], 512, 96)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,rows,cols", FEW + MANY)
def test_against_64_bits(dev, dtype, counts, rows, cols):
    _check(counts, 0, rows, cols, dtype, dev)
    _check(counts, 77, rows, cols, dtype, dev)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_tiles(dev, dtype):
    """Sizes at which 256 x 256 tiles are taken for y, dx and dw, ends and edges within them."""
    _check([2100, 1, 0, 5000, 700], 100, 4104, 136, dtype, dev)
    _check([6000, 3001], 3, 200, 4120, dtype, dev)


def test_few_rows_of_many_experts_by_size(dev):
    """A random number of rows for each of 300 experts, some without any, some with over 64."""
    g = torch.Generator().manual_seed(4)
    counts = (torch.rand(300, generator=g) ** 6 * 300).int().tolist()
    assert 0 in counts and max(counts) > 128
    _check(counts, 5, 48, 88, BF, dev)


def test_no_rows(dev):
    x, w, ends, dy = _inputs([0, 0], 0, 16, 24, BF, dev)
    assert G.grouped_linear(x, w, ends).shape == (0, 16)
    gx, gw = G.grouped_linear_backward(x, w, ends, dy)
    assert gx.shape == (0, 24) and gw.shape == w.shape and not bool(gw.any())
    _check([0, 0, 0], 9, 16, 24, BF, dev)
    _check([0] * 70, 130, 264, 520, HF, dev)


@pytest.mark.parametrize("counts,rest,rows,cols", [([5, 0, 20], 6, 40, 264), ([300, 0, 170], 200, 136, 200)])
def test_what_is_not_read_does_not_matter(dev, counts, rest, rows, cols):
    """NaN in the rows behind the last expert's, and in the weights of experts without rows."""
    for dtype in (BF, HF):
        x, w, ends, dy = _inputs(counts, rest, rows, cols, dtype, dev)
        x[sum(counts):] = NAN
        dy[sum(counts):] = NAN
        w[1] = NAN
        _check(counts, rest, rows, cols, dtype, dev, (x, w, ends, dy))


@pytest.mark.parametrize("counts,rows,cols", [([2, 30, 1], 40, 264), ([400, 3, 170], 136, 200)])
def test_a_row_of_infinities_and_nan_stays_alone(dev, counts, rows, cols):
    x, w, ends, dy = _inputs(counts, 0, rows, cols, BF, dev)
    clean = G.grouped_linear(x, w, ends)
    clean_x, clean_w = G.grouped_linear_backward(x, w, ends, dy)
    x[1], dy[1] = float("inf"), NAN
    y = G.grouped_linear(x, w, ends)
    gx, gw = G.grouped_linear_backward(x, w, ends, dy)
    others = torch.arange(x.shape[0], device=dev) != 1
    assert torch.equal(y[others], clean[others]) and not bool(y[1].isfinite().any())
    assert torch.equal(gx[others], clean_x[others]) and bool(gx[1].isnan().all())
    assert torch.equal(gw[1:], clean_w[1:]) and bool(gw[0].isnan().all())


@pytest.mark.parametrize("counts,rows,cols", [([2, 30, 1], 40, 264), ([400, 3, 170], 136, 200)])
def test_strides_and_alignment(dev, counts, rows, cols):
    x, w, ends, dy = _inputs(counts, 10, rows, cols, BF, dev)
    want = G.grouped_linear(x, w, ends)
    wx, ww = G.grouped_linear_backward(x, w, ends, dy)
    m = x.shape[0]
    wide = torch.full((m, cols + 24), NAN, device=dev, dtype=BF)
    wide[:, 8:8 + cols] = x
    odd = torch.full((m * cols + 1,), NAN, device=dev, dtype=BF)
    odd[1:] = x.flatten()
    every = torch.empty((m, cols, 2), device=dev, dtype=BF)
    every[..., 0] = x
    stacked = torch.full((w.shape[0], 2, rows, cols + 8), NAN, device=dev, dtype=BF)
    stacked[:, 1, :, :cols] = w
    for z in (wide[:, 8:8 + cols], odd[1:].view(m, cols), every[..., 0], x.t().contiguous().t()):
        for v in (w, stacked[:, 1, :, :cols]):
            assert torch.equal(G.grouped_linear(z, v, ends), want)
            gx, gw = G.grouped_linear_backward(z, v, ends, dy.t().contiguous().t())
            assert torch.equal(gx, wx) and torch.equal(gw, ww)
    pairs = torch.stack([ends, ends], 1)
    assert torch.equal(G.grouped_linear(x, w, pairs[:, 0]), want)
    one = dy[:1].expand(m, rows)
    gx, _ = G.grouped_linear_backward(x, w, ends, one)
    assert torch.equal(gx, G.grouped_linear_backward(x, w, ends, one.contiguous())[0])


@pytest.mark.parametrize("counts,rows,cols", [([2, 30, 1], 40, 264), ([400, 3, 170], 136, 200), ([300], 64, 8192)])
def test_out_keeps_what_is_behind(dev, counts, rows, cols):
    x, w, ends, _ = _inputs(counts, 10, rows, cols, BF, dev)
    want, used = G.grouped_linear(x, w, ends), sum(counts)
    big = torch.full((x.shape[0], rows + 16), 3.0, device=dev, dtype=BF)
    out = big[:, 8:8 + rows]
    version = out._version
    assert G.grouped_linear(x, w, ends, out=out) is out and out._version > version
    assert torch.equal(out[:used], want[:used])
    assert bool((out[used:] == 3).all()) and bool((big[:, :8] == 3).all()) and bool((big[:, 8 + rows:] == 3).all())


def test_out_across_x(dev):
    """x's own memory as out: from a copy of x."""
    for counts in ([2, 30, 1], [400, 3, 170]):
        x, w, ends, _ = _inputs(counts, 0, 64, 64, BF, dev)
        want = G.grouped_linear(x, w, ends)
        assert torch.equal(G.grouped_linear(x, w, ends, out=x), want)


def test_ends_out_of_range(dev):
    for m, rows in ((20, 24), (900, 264)):
        x = torch.ones((m, 40), device=dev, dtype=BF)
        w = torch.ones((4, rows, 40), device=dev, dtype=BF)
        dy = torch.ones((m, rows), device=dev, dtype=BF)
        for ends in ([5, 3, 10, m], [1, 2, 3, m + 1], [-1, 2, 3, 4], [m, 0, m, 0], [1 << 40, -(1 << 40), 1 << 62, 5]):
            _say(f"[grouped] ends {ends} of {m} rows")
            t = torch.tensor(ends, device=dev)
            with pytest.raises(wc.WcError, match="index out of range"):
                G.grouped_linear(x, w, t)
            with pytest.raises(wc.WcError, match="index out of range"):
                G.grouped_linear_backward(x, w, t, dy)
            G.grouped_linear(x, w, t, check=False)
            G.grouped_linear_backward(x, w, t, dy, check=False)
        torch.cuda.synchronize()
        t = torch.tensor([5, 5, 10, m], device=dev)
        assert bool((G.grouped_linear(x, w, t) == 40).all())


@pytest.mark.parametrize("counts,rows,cols", [([3, 0, 20, 1], 40, 264), ([400, 0, 170], 136, 200)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_autograd(dev, dtype, counts, rows, cols):
    x, w, ends, dy = _inputs(counts, 4, rows, cols, dtype, dev)
    dx, dw = G.grouped_linear_backward(x, w, ends, dy)
    for need in ((True, True), (True, False), (False, True)):
        a, b = x.clone().requires_grad_(need[0]), w.clone().requires_grad_(need[1])
        y = G.grouped_linear(a, b, ends)
        y.backward(dy)
        assert torch.equal(y, G.grouped_linear(x, w, ends))
        assert torch.equal(a.grad, dx) if need[0] else a.grad is None
        assert torch.equal(b.grad, dw) if need[1] else b.grad is None
    # a view of stacked weights, and a gradient that is one number
    both = torch.stack([w, w], 1).requires_grad_()
    G.grouped_linear(x, both[:, 1], ends).sum().backward()
    assert torch.equal(both.grad[:, 1], G.grouped_linear_backward(x, w, ends, torch.ones_like(dy))[1])
    assert not bool(both.grad[:, 0].any())


def test_gradient_against_differences(dev):
    """The gradient of sum (c y) along a direction against differences of the definition in 64 bits."""
    counts, rows, cols = [70, 0, 201], 72, 88
    x, w, ends, c = _inputs(counts, 0, rows, cols, HF, dev)
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    G.grouped_linear(a, b, ends).backward(c)
    g = torch.Generator(device=dev).manual_seed(9)

    def f(x, w):
        return sum(float((c[at].double() * (x[at] @ w[e].T)).sum()) for e, at in _groups(counts))
    for which, at, grad in ((0, x, a.grad), (1, w, b.grad)):
        d = torch.randn(at.shape, generator=g, device=dev, dtype=torch.float64)
        lo, hi = ([x.double(), w.double()] for _ in range(2))
        lo[which], hi[which] = lo[which] - 0.5 * d, hi[which] + 0.5 * d
        along = f(*hi) - f(*lo)  # f is linear in either: the difference is exact but for 64-bit sums
        got = float((grad.double() * d).sum())
        # each element of the gradient is rounded to half precision (and summed in fp32: less than that)
        assert abs(got - along) <= 2 * 2.0 ** -11 * float((grad.double().abs() * d.abs()).sum())


def test_what_autograd_cannot_do_raises(dev):
    x, w, ends, dy = _inputs([3, 4], 0, 16, 24, BF, dev)
    a = x.clone().requires_grad_()
    with pytest.raises(ValueError, match="no out"):
        G.grouped_linear(a, w, ends, out=torch.empty_like(dy))
    with pytest.raises(ValueError, match="current stream"):
        G.grouped_linear(a, w, ends, stream=torch.cuda.Stream())
    with pytest.raises(RuntimeError, match="no backward pass"):
        G.grouped_linear_backward(a, w, ends, dy)
    g, = torch.autograd.grad(G.grouped_linear(a, w, ends).float().square().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        g.sum().backward()
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            G.grouped_linear(forward_ad.make_dual(x, x), w, ends)
    y = G.grouped_linear(a, w, ends)
    a.data.add_(0)
    with torch.no_grad():
        a.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy)


def test_refusals(dev):
    x, w, ends, dy = _inputs([3, 4], 0, 16, 24, BF, dev)
    bad = [((x.float(), w, ends), TypeError), ((x, w.half(), ends), TypeError), ((x[:, :16], w, ends), ValueError),
           ((x[0], w, ends), ValueError), ((x, w[0], ends), ValueError), ((x, w, ends.int()), ValueError),
           ((x, w, ends[:1]), ValueError), ((x[:, :20], w[:, :, :20], ends), ValueError), ((x, w[:, :12], ends), ValueError),
           ((x.cpu(), w, ends), ValueError), ((x, w, ends.cpu()), ValueError), ((x, w[:0], ends[:0]), ValueError),
           ((x, w.transpose(1, 2).contiguous().transpose(1, 2), ends), ValueError)]
    for args, kind in bad:
        with pytest.raises(kind):
            G.grouped_linear(*args)
        with pytest.raises(kind):
            G.grouped_linear_backward(*args, dy)
    for out in (torch.empty((7, 15), device=dev, dtype=BF), torch.empty((7, 16), device=dev), torch.empty((7, 17), device=dev, dtype=BF)[:, :16],
                torch.empty(7 * 16 + 1, device=dev, dtype=BF)[1:].view(7, 16), torch.empty((1, 16), device=dev, dtype=BF).expand(7, 16)):
        with pytest.raises(ValueError):
            G.grouped_linear(x, w, ends, out=out)
    both = torch.zeros(2 * 16 * 24, device=dev, dtype=BF)
    with pytest.raises(ValueError, match="memory in common"):
        G.grouped_linear(x, both.view(2, 16, 24), ends, out=both[:112].view(7, 16))
    for grad in (dy[:, :8], dy.float(), dy[:3]):
        with pytest.raises(ValueError):
            G.grouped_linear_backward(x, w, ends, grad)
    assert G.grouped_linear_backward(x, w, ends, dy, need_x=False, need_w=False) == (None, None)

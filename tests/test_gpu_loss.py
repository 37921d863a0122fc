"""Cross entropy from hidden states, and its gradients, against the definition
in 64 bits.

Tolerances.  A logit, k exact products summed in fp32, is off by
(k + 24) 2^-24 times the sum of their sizes.  An exponential of a difference d
has a relative error of (3 |d| + 8) 2^-24, and the sum of them, joined from
at most vocabulary / 2048 + 16 parts in a row after chains of 64, another of
(64 + 12 (vocabulary / 2048 + 16)) 2^-24; |d| exp(-|d|) is below 0.4, so that
all the far ones add less than 3 2^-24 each.  The gradient of a logit is
rounded once to the type (FP16: after a scaling, or by 2^-38 of the largest),
its products with W and H are sums in fp32, and their results are rounded once.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import logprobs, loss as L  # noqa: E402

EPS = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _inputs(m, v, k, dtype, dev, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    w = (torch.randn((v, k), generator=g, device=dev) * (1.5 * k ** -0.5)).to(dtype)
    t = torch.randint(0, v, (m,), generator=g, device=dev)
    h = (torch.randn((m, k), generator=g, device=dev) + 2 * w[t].float()).to(dtype)
    t[3::5] = -1
    gl = torch.randn(m, generator=g, device=dev)
    gz = 0.01 * torch.randn(m, generator=g, device=dev)
    return h, w, t, gl, gz


def _near(got, want, tol, what):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).nan_to_num(9e9).max())} of its tolerance"


def _check_loss(h, w, t, what):
    k, v = h.shape[1], w.shape[0]
    z, size = h.double() @ w.double().T, h.double().abs() @ w.double().abs().T
    lse = torch.logsumexp(z, 1)
    given = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    want = torch.where(t < 0, 0.0, lse - given)
    dz = (k + 24) * EPS * size.amax(1)
    ds = (64 + 12 * (v / 2048 + 16) + 11) * EPS + dz
    r = L.linear_cross_entropy(h, w, t)
    assert r.loss.dtype == r.lse.dtype == torch.float32 and r.loss.shape == r.lse.shape == t.shape
    most = z.amax(1)
    _near(r.lse, lse, ds + 2 * EPS * (lse.abs() + most.abs() + (lse - most).abs()), what + ", lse")
    _near(r.loss, want, 2 * dz + ds + 2 * EPS * ((most - given).abs() + 2 * (lse - most).abs() + want.abs()), what + ", loss")
    assert bool((r.loss[t < 0] == 0).all())
    return r


def _check_gradient(h, w, t, lse, gl, gz, what):
    k, v, dtype = h.shape[1], w.shape[0], h.dtype
    f = torch.finfo(dtype)
    hd, wd = h.double(), w.double()
    z, size = hd @ wd.T, hd.abs() @ wd.abs().T
    of_token = torch.where(t < 0, 0.0, gl.double()) if gl is not None else torch.zeros(h.shape[0], dtype=torch.float64, device=h.device)
    of_lse = of_token + (gz.double() if gz is not None else 0)
    d = z - lse.double()[:, None]
    p = d.exp()
    g = p * of_lse[:, None]
    dg = g.abs() * ((k + 24) * EPS * size + (3 * d.abs() + 8) * EPS)
    hot = torch.zeros_like(g).scatter_(1, t.clamp(min=0)[:, None], 1.0) * (t >= 0)[:, None]
    g = g - of_token[:, None] * hot
    dg += 2 * EPS * (g.abs() + of_lse.abs()[:, None] * p) + (f.eps / 2) * 1.01 * g.abs()
    if dtype == HF:
        dg += 2.0 ** -38 * float(torch.maximum(of_token.abs(), of_lse.abs()).max())
    got_h, got_w = L.linear_cross_entropy_backward(h, w, t, lse, gl, gz)
    assert got_h.dtype == got_w.dtype == dtype and got_h.shape == h.shape and got_w.shape == w.shape

    def tol(want, off, n, sizes):
        return off + (n + 24) * EPS * sizes + (f.eps / 2) * 1.01 * (want.abs() + off) + f.tiny * f.eps
    want = g @ wd
    _near(got_h, want, tol(want, dg @ wd.abs(), v, g.abs() @ wd.abs()), what + ", hidden")
    want = g.T @ hd
    _near(got_w, want, tol(want, dg.T @ hd.abs(), h.shape[0], g.abs().T @ hd.abs()), what + ", weight")
    return got_h, got_w


SIZES = [(1, 1, 8), (1, 1003, 64), (1, 50257, 768), (2, 17, 16), (5, 31, 2056), (16, 100, 40), (17, 1000, 1032), (33, 4097, 264),
         (64, 513, 2304), (61, 12345, 128), (65, 40, 72), (100, 1001, 520), (129, 300, 264), (200, 2049, 136), (300, 33, 1000),
         (1000, 777, 96), (70, 20000, 64)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,v,k", SIZES)
def test_against_64_bits(dev, dtype, m, v, k):
    what = f"{dtype} {m} rows, {v} x {k}"
    _say(f"[loss] {what}")
    h, w, t, gl, gz = _inputs(m, v, k, dtype, dev)
    r = _check_loss(h, w, t, what)
    _say("[loss]   gradient")
    _check_gradient(h, w, t, r.lse, gl, gz, what)
    _check_gradient(h, w, t, r.lse, gl, None, what + ", of the loss alone")
    _check_gradient(h, w, t, r.lse, None, gz, what + ", of lse alone")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_tiles(dev, dtype):
    """Sizes at which 256 x 256 tiles are taken, with edges within them."""
    h, w, t, gl, gz = _inputs(2100, 30011, 136, dtype, dev)
    _say(f"[loss] large tiles {dtype}")
    r = _check_loss(h, w, t, "large tiles")
    _say("[loss]   gradient")
    _check_gradient(h, w, t, r.lse, gl, gz, "large tiles")


def test_pieces_of_the_vocabulary(dev):
    """More rows times vocabulary than one piece holds (2^27): the hidden gradient adds up over three of them."""
    m, v, k = 9000, 40003, 24
    h, w, t, gl, gz = _inputs(m, v, k, BF, dev)
    _say("[loss] pieces")
    lse = L.linear_cross_entropy(h, w, t).lse
    _check_gradient(h, w, t, lse, gl, gz, "pieces")


def test_as_token_logprobs_on_logits(dev):
    """Whole numbers: the logits are exact in any type, so that both agree to the last roundings."""
    g = torch.Generator(device=dev).manual_seed(2)
    h = torch.randint(-2, 3, (70, 16), generator=g, device=dev).to(BF)
    w = torch.randint(-1, 2, (900, 16), generator=g, device=dev).to(BF)
    t = torch.randint(0, 900, (70,), generator=g, device=dev)
    a, b = L.linear_cross_entropy(h, w, t), logprobs.token_logprobs(h.float() @ w.float().T, t)
    _near(a.loss, -b.logprob.double(), 2e-5, "loss")
    _near(a.lse, b.lse.double(), 2e-5, "lse")


@pytest.mark.parametrize("m", [3, 90])
def test_far_logits(dev, m):
    """Logits of thousands: the loss of the largest one is 0, of the others their distance."""
    k, v = 32, 300
    h = torch.zeros((m, k), device=dev, dtype=BF)
    w = torch.zeros((v, k), device=dev, dtype=BF)
    h[:, 0], w[:, 0] = 64.0, torch.arange(v, device=dev).remainder(97).to(BF) * 2
    w[17, 0] = 256
    t = torch.full((m,), 17, device=dev)
    t[1] = 2
    r = L.linear_cross_entropy(h, w, t)
    assert bool((r.lse == 64.0 * 256).all())
    assert float(r.loss[0]) == 0 and float(r.loss[1]) == 64.0 * (256 - 4)
    one = torch.ones(m, device=dev)
    gh, gw = L.linear_cross_entropy_backward(h, w, t, r.lse, one)
    assert not bool(gh[0].any()) and float(gh[1, 0]) == 256 - 4
    assert float(gw[17, 0]) == 64 and float(gw[2, 0]) == -64 and not bool(gw[3].any())


@pytest.mark.parametrize("m", [1, 3, 90, 300])
def test_infinities_and_nan(dev, m):
    k, v = 32, 700
    h = torch.ones((m, k), device=dev, dtype=BF)
    w = torch.ones((v, k), device=dev, dtype=BF)
    t = torch.full((m,), 5, device=dev)
    w[:, 0] = -INF                                  # every logit -inf
    r = L.linear_cross_entropy(h, w, t)
    assert bool((r.lse == -INF).all()) and bool((r.loss == INF).all())
    gh, gw = L.linear_cross_entropy_backward(h, torch.ones_like(w), t, r.lse, torch.ones(m, device=dev))
    assert not bool(gh.any()) and not bool(gw.any())
    w[5, 0] = 1                                     # every one but the token's: the loss is 0
    r = L.linear_cross_entropy(h, w, t)
    assert bool((r.lse == k).all()) and bool((r.loss == 0).all())
    w[5, 0] = INF
    r = L.linear_cross_entropy(h, w, t)
    assert bool(r.lse.isnan().all()) and bool(r.loss.isnan().all())
    w[:, 0] = 1
    h[0] = NAN
    r = L.linear_cross_entropy(h, w, t)
    assert bool(r.lse[0].isnan()) and bool(r.lse[1:].isfinite().all())


@pytest.mark.parametrize("m,v,k", [(5, 100, 40), (90, 1000, 64), (600, 9000, 64)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_without_a_part(dev, dtype, m, v, k):
    """Rows without a token whose hidden values are NaN: loss 0, and no part in either gradient."""
    h, w, t, gl, _ = _inputs(m, v, k, dtype, dev)
    h[t < 0] = NAN
    r = L.linear_cross_entropy(h, w, t)
    assert bool((r.loss[t < 0] == 0).all()) and bool(r.lse[t < 0].isnan().all()) and bool(r.lse[t >= 0].isfinite().all())
    gh, gw = L.linear_cross_entropy_backward(h, w, t, r.lse, gl)
    assert not bool(gh[t < 0].any()) and bool(gh.isfinite().all()) and bool(gw.isfinite().all())
    clean = torch.where((t < 0)[:, None], 0, h)
    bh, bw = L.linear_cross_entropy_backward(clean, w, t, torch.where(t < 0, 0, r.lse), gl)
    assert torch.equal(gh, bh) and torch.equal(gw, bw)
    none = torch.full_like(t, -1)
    gh, gw = L.linear_cross_entropy_backward(h, w, none, r.lse, gl)
    assert not bool(gh.any()) and not bool(gw.any())


@pytest.mark.parametrize("m", [4, 100])
def test_tokens_out_of_range(dev, m):
    h, w, t, gl, _ = _inputs(m, 50, 16, BF, dev)
    good = L.linear_cross_entropy(h, w, t)
    for bad in (50, -2, 1 << 40):
        u = t.clone()
        u[2] = bad
        with pytest.raises(wc.WcError, match="index out of range"):
            L.linear_cross_entropy(h, w, u)
        with pytest.raises(wc.WcError, match="index out of range"):
            L.linear_cross_entropy_backward(h, w, u, good.lse, gl)
        r = L.linear_cross_entropy(h, w, u, check=False)
        assert bool(r.loss[2].isnan()) and torch.equal(r.lse, good.lse) and torch.equal(r.loss[3:], good.loss[3:])
        gh, gw = L.linear_cross_entropy_backward(h, w, u, good.lse, gl, check=False)
        u[2] = -1
        bh, bw = L.linear_cross_entropy_backward(h, w, u, good.lse, gl)
        assert torch.equal(gh, bh) and torch.equal(gw, bw)


@pytest.mark.parametrize("m", [5, 90])
def test_strides_and_alignment(dev, m):
    v, k = 301, 72
    h, w, t, gl, gz = _inputs(m, v, k, HF, dev)
    want = L.linear_cross_entropy(h, w, t)
    wh, ww = L.linear_cross_entropy_backward(h, w, t, want.lse, gl, gz)
    wide = torch.full((v, k + 16), NAN, device=dev, dtype=HF)
    wide[:, 8:8 + k] = w
    odd = torch.zeros(m * k + 1, device=dev, dtype=HF)
    odd[1:] = h.flatten()
    pair = torch.stack([t, t], 1)[:, 0]
    for z in (h.t().contiguous().t(), odd[1:].view(m, k)):
        r = L.linear_cross_entropy(z, wide[:, 8:8 + k], pair)
        assert torch.equal(r.loss, want.loss) and torch.equal(r.lse, want.lse)
        gh, gw = L.linear_cross_entropy_backward(z, wide[:, 8:8 + k], pair, torch.stack([want.lse, gl], 1)[:, 0],
                                                 torch.stack([gl, gl], 1)[:, 0], torch.stack([gz, gl], 1)[:, 0])
        assert torch.equal(gh, wh) and torch.equal(gw, ww)
    same = L.linear_cross_entropy(h[:1].expand(m, k), w, t)
    assert torch.equal(same.lse, same.lse[:1].expand(m))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,v,k", [(1, 301, 72), (7, 301, 72), (300, 2000, 64)])
def test_autograd(dev, dtype, m, v, k):
    h, w, t, gl, gz = _inputs(m, v, k, dtype, dev)
    plain = L.linear_cross_entropy(h, w, t)
    for need in ((True, True), (True, False), (False, True)):
        for a, b in ((gl, gz), (gl, None), (None, gz)):
            x, y = h.clone().requires_grad_(need[0]), w.clone().requires_grad_(need[1])
            r = L.linear_cross_entropy(x, y, t)
            assert torch.equal(r.loss, plain.loss) and torch.equal(r.lse, plain.lse)
            total = (0 if a is None else (a * r.loss).sum()) + (0 if b is None else (b * r.lse).sum())
            total.backward()
            dh, dw = L.linear_cross_entropy_backward(h, w, t, plain.lse, a, b)
            assert torch.equal(x.grad, dh) if need[0] else x.grad is None
            assert torch.equal(y.grad, dw) if need[1] else y.grad is None
    x = h.clone().requires_grad_()
    L.linear_cross_entropy(x, w, t).loss.sum().backward()
    assert torch.equal(x.grad, L.linear_cross_entropy_backward(h, w, t, plain.lse, torch.ones(m, device=dev))[0])


@pytest.mark.parametrize("m,v,k", [(7, 301, 72), (150, 1500, 64)])
def test_gradient_against_differences(dev, m, v, k):
    """The gradient along a direction against central differences of the definition in 64 bits."""
    h, w, t, gl, gz = _inputs(m, v, k, HF, dev)
    x, y = h.clone().requires_grad_(), w.clone().requires_grad_()
    r = L.linear_cross_entropy(x, y, t)
    ((gl * r.loss).sum() + (gz * r.lse).sum()).backward()
    g = torch.Generator(device=dev).manual_seed(9)

    def f(h, w):
        z = h @ w.T
        lse = torch.logsumexp(z, 1)
        loss = torch.where(t < 0, 0.0, lse - z.gather(1, t.clamp(min=0)[:, None])[:, 0])
        return float((gl.double() * loss).sum() + (gz.double() * lse).sum())
    for which, at, grad in ((0, h, x.grad), (1, w, y.grad)):
        d = torch.randn(at.shape, generator=g, device=dev, dtype=torch.float64)
        s = 1e-4
        lo, hi = ([h.double(), w.double()] for _ in range(2))
        lo[which], hi[which] = lo[which] - s * d, hi[which] + s * d
        along, got = (f(*hi) - f(*lo)) / (2 * s), float((grad.double() * d).sum())
        # roundings of G and of the result, half a step each, of numbers whose sizes add up to at most:
        p = torch.softmax(h.double() @ w.double().T, 1) * (gl.abs() + gz.abs()).double()[:, None]
        p += torch.zeros_like(p).scatter_(1, t.clamp(min=0)[:, None], gl.abs().double()[:, None])
        sizes = p @ w.double().abs() if which == 0 else p.T @ h.double().abs()
        # and the third derivative's part of the differences, s^2 / 6 of it, far below them
        assert abs(got - along) <= 2 * 2.0 ** -11 * float((sizes * d.abs()).sum())


def test_what_autograd_cannot_do_raises(dev):
    h, w, t, gl, _ = _inputs(7, 50, 16, BF, dev)
    x = h.clone().requires_grad_()
    with pytest.raises(ValueError, match="current stream"):
        L.linear_cross_entropy(x, w, t, stream=torch.cuda.Stream())
    r = L.linear_cross_entropy(x, w, t)
    with pytest.raises(RuntimeError, match="no backward pass"):
        L.linear_cross_entropy_backward(x, w, t, r.lse.detach(), gl)
    g, = torch.autograd.grad(r.loss.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        g.sum().backward()
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            L.linear_cross_entropy(forward_ad.make_dual(h, h), w, t)


def test_no_rows(dev):
    h, w, t = torch.empty((0, 16), device=dev, dtype=BF), torch.ones((9, 16), device=dev, dtype=BF), torch.empty(0, device=dev, dtype=torch.int64)
    r = L.linear_cross_entropy(h, w, t)
    assert r.loss.shape == r.lse.shape == (0,)
    gh, gw = L.linear_cross_entropy_backward(h, w, t, r.lse, r.loss)
    assert gh.shape == (0, 16) and gw.shape == (9, 16) and not bool(gw.any())


def test_refusals(dev):
    h, w, t, gl, _ = _inputs(7, 50, 16, BF, dev)
    bad = [((h.float(), w, t), TypeError), ((h, w.half(), t), TypeError), ((h[:, :8], w, t), ValueError), ((h[0], w, t), ValueError),
           ((h, w[0], t), ValueError), ((h, w, t.int()), ValueError), ((h, w, t[:3]), ValueError), ((h, w[:0], t), ValueError),
           ((h[:, :12], w[:, :12], t), ValueError), ((h.cpu(), w, t), ValueError), ((h, w.cpu(), t), ValueError),
           ((h, w.t().contiguous().t(), t), ValueError), ((h, w[:1].expand(50, 16), t), ValueError),
           ((h[:1].expand((1 << 19) + 1, 16), w, t[:1].expand((1 << 19) + 1)), ValueError)]
    for args, kind in bad:
        with pytest.raises(kind):
            L.linear_cross_entropy(*args)
        with pytest.raises(kind):
            L.linear_cross_entropy_backward(*args, gl, gl)
    for lse, g, z in ((None, gl, None), (gl[:3], gl, None), (gl, gl.double(), None), (gl, gl, gl[:1]), (gl.cpu(), gl, None)):
        with pytest.raises(ValueError):
            L.linear_cross_entropy_backward(h, w, t, lse, g, z)
    assert L.linear_cross_entropy_backward(h, w, t, gl, gl, need_hidden=False, need_weight=False) == (None, None)

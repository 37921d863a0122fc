"""Products with weights of 4 bits, and their making, against the definition
in 64 bits.

Tolerance.  With w = s (q - z) the kernel sums (16 + q) x over a group, takes
(16 + z) sum x from it, scales, and sums the groups: all in fp32, of exact
products.  Each of these sums of n terms is off by at most (n + 24) 2^-24 times
the sum of their sizes, which is that of s (|16 + q| + |16 + z|) |x|; the two
products with z and s add 3 2^-24 of it.  Then one rounding to the type.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import fourbit as F  # noqa: E402

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


def _inputs(m, rows, cols, group, dtype, zeros, dev, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    q = torch.randint(0, 256, (rows, cols // 2), generator=g, device=dev, dtype=torch.uint8)
    s = ((0.5 + torch.rand((rows, cols // group), generator=g, device=dev)) * cols ** -0.5 / 4).to(dtype)
    z = (7 + 2 * torch.randn(s.shape, generator=g, device=dev)).to(dtype) if zeros else None
    x = torch.randn((m, cols), generator=g, device=dev).to(dtype)
    return x, F.Weights4(q, s, z, group)


def _values(w):
    """q and the zeros as rows x groups x group, in 64 bits."""
    rows, groups = w.scales.shape
    q = torch.stack([w.q & 15, w.q >> 4], 2).view(rows, groups, w.group).double()
    z = (torch.full_like(w.scales, 8) if w.zeros is None else w.zeros).double()[..., None]
    return q, z, w.scales.double()[..., None]


def _expect(x, w):
    q, z, s = _values(w)
    rows, cols = q.shape[0], x.shape[1]
    xd = x.double()
    want = xd @ (s * (q - z)).reshape(rows, cols).T
    size = xd.abs() @ (s.abs() * ((16 + q) + (16 + z).abs())).reshape(rows, cols).T
    f = torch.finfo(x.dtype)
    return want, (cols + 27) * EPS * size + (f.eps / 2) * 1.01 * want.abs() + f.tiny * f.eps


def _check(x, w, what):
    _say(f"[4 bits] {what}")
    want, tol = _expect(x, w)
    y = F.linear4(x, w)
    assert y.dtype == x.dtype and y.shape == want.shape
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).nan_to_num(9e9).max())} of its tolerance"
    return y


SIZES = [(1, 1, 1), (1, 16, 4), (1, 4096, 32), (2, 17, 8), (5, 100, 3), (16, 33, 40), (17, 4100, 2), (31, 65, 9), (33, 250, 17),
         (61, 300, 5), (64, 8200, 1), (70, 40, 6), (200, 24, 2), (3, 16500, 2), (1, 9, 300)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,rows,groups", SIZES)
def test_against_64_bits(dev, dtype, group, m, rows, groups):
    for zeros in (False, True):
        x, w = _inputs(m, rows, groups * group, group, dtype, zeros, dev)
        _check(x, w, f"{dtype} {m} rows, {rows} x {groups} groups of {group}, zeros {zeros}")


def test_every_value_in_every_place(dev):
    """A weight at a time: x is one column, so that y is that column of the weights, exactly."""
    for dtype in (BF, HF):
        for group in (32, 64, 128):
            q = torch.arange(16, device=dev).repeat_interleave(1)[:, None].repeat(1, group).to(torch.uint8)
            q = (q + torch.arange(group, device=dev)) % 16
            w = F.Weights4((q[:, ::2] | (q[:, 1::2] << 4)).to(torch.uint8).contiguous(), torch.full((16, 1), 0.5, device=dev, dtype=dtype), None, group)
            y = F.linear4(torch.eye(group, device=dev, dtype=dtype), w)
            assert torch.equal(y, ((q.float() - 8) / 2).T.to(dtype))


def test_strides_and_outputs(dev):
    for m in (3, 40):
        x, w = _inputs(m, 75, 192, 64, BF, True, dev)
        want = F.linear4(x, w)
        wide = torch.full((m, 200), NAN, device=dev, dtype=BF)
        wide[:, 8:] = x
        odd = torch.zeros(m * 192 + 1, device=dev, dtype=BF)
        odd[1:] = x.flatten()
        for z in (wide[:, 8:], odd[1:].view(m, 192), x.t().contiguous().t()):
            assert torch.equal(F.linear4(z, w), want)
        big = torch.full((m, 90), 3.0, device=dev, dtype=BF)
        out = big[:, 5:80]
        version = out._version
        assert F.linear4(x, w, out=out) is out and out._version > version
        assert torch.equal(out, want) and bool((big[:, :5] == 3).all()) and bool((big[:, 80:] == 3).all())
        square, v = _inputs(m, 128, 128, 64, BF, False, dev)
        want = F.linear4(square, v)
        assert torch.equal(F.linear4(square, v, out=square), want)  # across x: from a copy of it


def test_no_rows(dev):
    x, w = _inputs(0, 16, 64, 64, BF, False, dev)
    assert F.linear4(x, w).shape == (0, 16)


def test_infinities_and_nan_stay_where_they_are(dev):
    for m in (4, 20):
        x, w = _inputs(m, 64, 320, 64, HF, False, dev)
        clean = F.linear4(x, w)
        x[1, 7] = float("inf")
        w.scales[5, 4] = NAN  # of the last slice, which is not whole
        y = F.linear4(x, w)
        rows = torch.arange(64, device=dev) != 5
        others = torch.arange(m, device=dev) != 1
        assert torch.equal(y[others][:, rows], clean[others][:, rows])
        assert bool(y[:, 5].isnan().all()) and not bool(y[1].isfinite().any())


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(dev, dtype, group):
    g = torch.Generator(device=dev).manual_seed(group)
    w = torch.randn((37, 3 * group), generator=g, device=dev).to(dtype)
    w[3, :group] = 0
    w[4, :group] = 0.75
    w[5, :group] = w[5, :group].abs()
    w[6, :group] = -w[6, :group].abs()
    for zeros in (False, True):
        got = F.quantize4(w, group, zeros=zeros)
        v = w.view(37, 3, group).float()
        lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7).to(dtype)
        s = scale.float()
        zero = torch.where(s > 0, (-lo / s).round().clamp(max=15), 0.0) if zeros else torch.full_like(s, 8)
        q = torch.where(s[..., None] > 0, (v / s[..., None]).round() + zero[..., None], zero[..., None]).clamp(0, 15).view(37, -1)
        assert torch.equal(got.scales, scale) and got.group == group
        assert got.zeros is None if not zeros else torch.equal(got.zeros, zero.to(dtype))
        assert torch.equal(got.q & 15, q[:, ::2].to(torch.uint8)) and torch.equal(got.q >> 4, q[:, 1::2].to(torch.uint8))
        # every weight within half a step, and what the rounding of the scale moves the ends by
        _, z, _ = _values(got)
        back = (torch.stack([got.q & 15, got.q >> 4], 2).view(37, 3, group).double() - z) * s.double()[..., None]
        step = s.double()[..., None]
        assert bool(((back - v.double()).abs() <= step * (0.5 + 1e-6) + 15 * step * torch.finfo(dtype).eps + 0.5 * step * zeros).all())
    odd = torch.zeros(w.numel() + 1, device=dev, dtype=dtype)
    odd[1:] = w.flatten()
    for t in (odd[1:].view(w.shape), w.t().contiguous().t(), torch.cat([w, w], 1)[:, :3 * group]):
        same = F.quantize4(t, group, zeros=True)
        assert all(torch.equal(a, b) for a, b in zip(same[:3], got[:3]))


def test_quantize_then_multiply(dev):
    g = torch.Generator(device=dev).manual_seed(3)
    w = (torch.randn((200, 512), generator=g, device=dev) / 20).to(BF)
    x = torch.randn((9, 512), generator=g, device=dev).to(BF)
    for zeros in (False, True):
        w4 = F.quantize4(w, 64, zeros=zeros)
        y = _check(x, w4, "quantized")
        off = (y.double() - x.double() @ w.double().T).abs()
        step = w4.scales.double().repeat_interleave(64, 1)
        assert bool((off <= x.double().abs() @ (1.1 * step).T + 2.0 ** -8 * y.double().abs()).all())


def test_bad_groups_say_so(dev):
    w = torch.ones((2, 128), device=dev, dtype=HF)
    w[0, 5], w[1, 100] = NAN, float("inf")
    for zeros in (False, True):
        got = F.quantize4(w, 64, zeros=zeros)
        assert bool(got.scales[0, 0].isnan()) and bool(got.scales[1, 1].isinf()) and bool(got.scales[0, 1].isfinite())


def test_what_autograd_cannot_do_raises(dev):
    x, w = _inputs(3, 16, 64, 64, BF, True, dev)
    want = F.linear4(x, w)
    a = x.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="no backward pass"):
        F.linear4(a, w)
    with pytest.raises(RuntimeError, match="no backward pass"):
        F.linear4(x, w._replace(scales=w.scales.clone().requires_grad_()))
    with torch.no_grad():
        assert torch.equal(F.linear4(a, w), want)
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            F.linear4(forward_ad.make_dual(x, x), w)


def test_refusals(dev):
    x, w = _inputs(3, 16, 128, 64, BF, True, dev)
    bad = [((x.float(), w), TypeError), ((x.half(), w), TypeError), ((x[:, :64], w), ValueError), ((x[0], w), TypeError),
           ((x.cpu(), w), ValueError), ((x, w._replace(group=48)), ValueError), ((x, w._replace(group=32)), ValueError),
           ((x, w._replace(scales=w.scales[:, :1])), ValueError), ((x, w._replace(scales=w.scales.t().contiguous().t())), ValueError),
           ((x, w._replace(zeros=w.zeros[:4])), ValueError), ((x, w._replace(q=w.q.int())), TypeError),
           ((x, w._replace(q=w.q.cpu())), ValueError)]
    for args, kind in bad:
        with pytest.raises(kind):
            F.linear4(*args)
    for out in (torch.empty((3, 15), device=dev, dtype=BF), torch.empty((3, 16), device=dev), torch.empty((1, 16), device=dev, dtype=BF).expand(3, 16)):
        with pytest.raises(ValueError):
            F.linear4(x, w, out=out)
    for args, kind in (((x.float(),), TypeError), ((x[0],), TypeError), ((x, 48), ValueError), ((x[:, :100],), ValueError), ((x.cpu(),), ValueError)):
        with pytest.raises(kind):
            F.quantize4(*args)

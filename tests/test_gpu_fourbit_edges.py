"""4-bit weights at the edges of what the types hold, and what cannot be followed by autograd.

Tolerances: as in test_gpu_fourbit.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from lossless_weight_compression_bf16_amd import fourbit as F  # noqa: E402
from test_gpu_fourbit import BF, HF, _check, _inputs, _say, dev  # noqa: E402, F401


@pytest.mark.parametrize("zeros", [False, True])
def test_making_them_has_no_gradient_and_says_so(dev, zeros):  # noqa: F811
    w = torch.randn((16, 128), generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(BF)
    want = F.quantize4(w, 64, zeros)
    p = torch.nn.Parameter(w.clone())
    for t in (p, 2 * p):
        with pytest.raises(RuntimeError, match="quantize4 has no backward pass"):
            F.quantize4(t, 64, zeros)
    with torch.no_grad():
        got = F.quantize4(p, 64, zeros)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    assert all(a is None or torch.equal(a, b) for a, b in zip(F.quantize4(p.detach(), 64, zeros)[:3], want[:3]))
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            F.quantize4(forward_ad.make_dual(w, w), 64, zeros)
        assert torch.equal(F.quantize4(w, 64, zeros).q, want.q)


def _edges(dev):  # noqa: F811
    big = torch.finfo(BF).max
    w = torch.zeros((4, 128), device=dev, dtype=BF)
    w[0, 3], w[0, 60] = big, -big
    w[1] = torch.linspace(-0.9 * big, big, 128, device=dev).to(BF)  # whose own steps overflow: infinities and NaN
    w[2, 64:], w[2, 70] = big, -0.5 * big
    w[3, 5], w[3, 6], w[3, 100] = float("inf"), -float("inf"), big
    return w


def _spread(dev):  # noqa: F811
    """Normal numbers up to the largest, of both signs."""
    w = torch.randn((4, 128), generator=torch.Generator(device=dev).manual_seed(5), device=dev, dtype=torch.float64).clamp_(-2, 2)
    w[:, ::32], w[:, 1::32] = 2, -2
    return (w * (0.5 * torch.finfo(BF).max)).to(BF)


@pytest.mark.parametrize("inputs", [_edges, _spread])
def test_a_range_past_the_largest_number(dev, inputs):  # noqa: F811
    """hi - lo overflows fp32 where the scale, a fifteenth of it, does not: finite weights have a finite scale."""
    w = inputs(dev)
    for group in (32, 64, 128):
        _say(f"[4 bits] ranges past the largest number, groups of {group}")
        got = F.quantize4(w, group, zeros=True)
        v = w.double().view(4, -1, group)
        lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
        finite = v.abs().amax(2) < float("inf")
        assert torch.equal(got.scales.isfinite(), finite)
        s, step = got.scales.double(), (hi - lo) / 15
        # half a step of BF16 and the quotients' and the difference's roundings
        assert bool(((s - step).abs()[finite] <= (2.0 ** -8 + 3 * 2.0 ** -24) * step[finite]).all())
        q = torch.stack([got.q & 15, got.q >> 4], 2).view(v.shape).double()
        some = finite & (step > 0)
        zero = (-lo / s).round().clamp(max=15)
        # a quotient next to a half may round either way in fp32
        assert bool(((got.zeros.double() - zero).abs()[some] <= ((-lo / s - zero).abs() > 0.4999)[some]).all())
        back = (q - got.zeros.double()[..., None]) * s[..., None]
        assert bool(((back - v).abs()[some] <= (s * (1.0 + 1e-6 + 15 * torch.finfo(BF).eps))[..., None][some]).all())
        near = F.quantize4((w[:3].float() / 2).to(BF), group, zeros=True)  # whose range does not overflow
        assert torch.equal(near.q, got.q[:3]) and torch.equal(near.zeros, got.zeros[:3])
        assert torch.equal((near.scales.float() * 2).nan_to_num(7.0), got.scales[:3].float().nan_to_num(7.0))


@pytest.mark.parametrize("m", [1, 16, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_large_x_is_finite_up_to_what_is_said(dev, m, group):  # noqa: F811
    """31 |x| summed over a group below 2^128: BF16 x of 2^128 / (32 group) at most."""
    for zeros in (False, True):
        x, w = _inputs(m, 200, 4 * group, group, BF, zeros, dev)
        if zeros:
            w.zeros.clamp_(0, 15)
        x = x.clamp(-1, 1)
        x[0] = 1
        scale = 2.0 ** 128 / (32 * group)
        w = w._replace(scales=(w.scales.float() * 2.0 ** -60).to(BF))
        want = F.linear4(x, w)
        got = _check((x.double() * scale).to(BF), w, f"{m} rows of numbers up to {scale}, groups of {group}, zeros {zeros}")
        assert bool(got.isfinite().all()) and torch.equal(got.double(), want.double() * scale)

"""Operators without a backward pass among tensors that autograd follows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad  # noqa: E402

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import adapters as A, logprobs as L, moe as M  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _adapters(dev, m=4):
    n, rank, c, rows = 2, 8, 64, 32
    g = torch.Generator().manual_seed(m)
    x, y, a, b = (torch.randn(s, generator=g).to(BF).to(dev) for s in ((m, c), (m, rows), (n, rank, c), (n, rows, rank)))
    return x, y, a, b, torch.arange(m, device=dev) % n, torch.rand(n, generator=g).to(dev)


def _experts(dev, m=4):
    e, h, i = 3, 16, 8
    g = torch.Generator().manual_seed(m)
    return [torch.randn(s, generator=g).to(BF).to(dev) for s in ((m, h), (e, h), (e, i, h), (e, i, h), (e, h, i))]


def test_tensors_that_require_a_gradient_raise(dev):
    args = _adapters(dev)
    want = A.add_adapters(args[0], args[1].clone(), *args[2:])
    for k in (0, 1, 2, 3, 5):
        some = [t.clone() for t in args]
        some[k].requires_grad_()
        with pytest.raises(RuntimeError, match="no backward pass"):
            A.add_adapters(*some)
        assert torch.equal(some[1], args[1])
        with torch.no_grad():
            assert torch.equal(A.add_adapters(*some), want)
    args = _experts(dev)
    want = M.moe_layer(*args, 2)
    for k in range(5):
        some = [t.clone() for t in args]
        some[k].requires_grad_()
        with pytest.raises(RuntimeError, match="no backward pass"):
            M.moe_layer(*some, 2)
        with torch.no_grad():
            assert torch.equal(M.moe_layer(*some, 2), want)
    with pytest.raises(RuntimeError, match="no backward pass"):
        M.moe_layer(*args, 2, out=torch.zeros_like(want).requires_grad_())


def _saved(t):
    """A loss whose backward pass needs t as it is now."""
    w = torch.ones_like(t).requires_grad_()
    return (w * t).sum()


def test_what_is_written_in_place_is_known_to_autograd(dev):
    x, y, a, b, ids, s = _adapters(dev)
    loss = _saved(y)
    A.add_adapters(x, y, a, b, ids, s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    args = _experts(dev)
    out = torch.zeros_like(args[0])
    loss = _saved(out)
    M.moe_layer(*args, 2, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    z, t = torch.randn((3, 100), device=dev), torch.arange(3, device=dev)
    r = L.token_logprobs(z, t)
    loss = _saved(z)
    L.token_logprobs_backward(z, t, r.lse, r.entropy, torch.ones(3, device=dev), out=z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_a_gradient_is_not_written_over_a_tensor_that_requires_one(dev):
    z, t = torch.randn((3, 100), device=dev).requires_grad_(), torch.arange(3, device=dev)
    one = torch.ones(3, device=dev)
    r = L.token_logprobs(z.detach(), t)
    before = z.detach().clone()
    want = L.token_logprobs_backward(z, t, r.lse, r.entropy, one)
    with pytest.raises(RuntimeError, match="requires a gradient"):
        L.token_logprobs_backward(z, t, r.lse, r.entropy, one, out=z)
    assert torch.equal(z.detach(), before)
    with torch.no_grad():
        assert torch.equal(L.token_logprobs_backward(z, t, r.lse, r.entropy, one, out=z), want)
    with torch.inference_mode():  # tensors without versions
        z = before.clone()
        assert torch.equal(L.token_logprobs_backward(z, t, r.lse, r.entropy, one, out=z), want)


def test_forward_mode_raises(dev):
    z, t = torch.randn((3, 100), device=dev), torch.arange(3, device=dev)
    r = L.token_logprobs(z, t)
    one = torch.ones(3, device=dev)
    ad, ex = _adapters(dev), _experts(dev)
    calls = [(lambda v: L.token_logprobs(v, t, top=2), z),
             (lambda v: L.token_logprobs_backward(z, t, r.lse, r.entropy, v), one),
             (lambda v: A.add_adapters(v, *ad[1:]), ad[0]), (lambda v: A.add_adapters(ad[0], v, *ad[2:]), ad[1]),
             (lambda v: M.moe_layer(v, *ex[1:], 2), ex[0]), (lambda v: M.moe_layer(*ex[:4], v, 2), ex[4])]
    with forward_ad.dual_level():
        for call, at in calls:
            call(at)  # no tangent
            with pytest.raises(RuntimeError, match="no forward-mode derivative"):
                call(forward_ad.make_dual(at, torch.ones_like(at)))

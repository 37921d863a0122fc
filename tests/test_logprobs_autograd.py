"""What autograd sees of token_logprobs, on the CPU: the node around the
kernels, with the formulas in 64 bits in the kernels' place."""
import pytest

torch = pytest.importorskip("torch")

from lossless_weight_compression_bf16_amd import logprobs as L  # noqa: E402


@pytest.fixture
def node(monkeypatch):
    def forward(logits, tokens, top, check, stream, views=True):
        logp = torch.log_softmax(logits, 1)
        best = torch.sort(logp, dim=1, descending=True, stable=True)
        return L.TokenLogprobs(logp.gather(1, tokens[:, None])[:, 0], -(logp.exp() * logp).sum(1),
                               torch.logsumexp(logits, 1), best.values[:, :top].clone() if top else None,
                               best.indices[:, :top].clone() if top else None)

    def backward(logits, tokens, lse, entropy, grad_logprob=None, grad_entropy=None, out=None, check=True, stream=None):
        logp = logits - lse[:, None]
        zero = torch.zeros_like(lse)
        g = (zero if grad_logprob is None else grad_logprob)[:, None]
        h = (zero if grad_entropy is None else grad_entropy)[:, None]
        d = -logp.exp() * (g + h * (logp + entropy[:, None]))
        return d.scatter_add(1, tokens[:, None], g)
    monkeypatch.setattr(L, "_forward", forward)
    monkeypatch.setattr(L, "token_logprobs_backward", backward)

    def call(logits, tokens, top=0):
        return L.TokenLogprobs(*L._TokenLogprobs.apply(logits, tokens, top, True))
    return call


def _case():
    g = torch.Generator().manual_seed(0)
    z = torch.randn((4, 9), generator=g, dtype=torch.float64).requires_grad_()
    return z, torch.tensor([0, 8, 3, 3])


def test_first_order(node):
    z, t = _case()
    r = node(z, t, top=2)
    got, = torch.autograd.grad(r.logprob.sum() - 0.3 * r.entropy.sum(), z)
    logp = torch.log_softmax(z, 1)
    want, = torch.autograd.grad(logp.gather(1, t[:, None]).sum() + 0.3 * (logp.exp() * logp).sum(), z)
    assert torch.allclose(got, want, rtol=0, atol=1e-12)


def test_second_order_raises(node):
    z, t = _case()
    r = node(z, t)
    d, = torch.autograd.grad(r.logprob.sum(), z, create_graph=True)
    assert torch.equal(d.detach(), torch.autograd.grad(node(z, t).logprob.sum(), z)[0])
    # the penalty's part of the gradient must not be left out of the sum
    with pytest.raises(RuntimeError, match="differentiated twice"):
        torch.autograd.grad(d.square().sum() + z.square().sum(), z)
    weight = torch.ones(4, dtype=torch.float64, requires_grad=True)
    d, = torch.autograd.grad((weight * node(z, t).logprob).sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated twice"):
        torch.autograd.grad(d.sum() + weight.sum(), weight)


def test_gradients_of_the_other_outputs_raise(node):
    z, t = _case()
    for loss in (lambda r: 0.1 * r.lse.square().sum() - r.logprob.sum(),
                 lambda r: r.top_logprobs.sum() - r.logprob.sum(), lambda r: r.lse.sum()):
        with pytest.raises(RuntimeError, match="logprob and entropy only"):
            torch.autograd.grad(loss(node(z, t, top=2)), z)
    r = node(z, t, top=2)
    assert not r.top_ids.requires_grad
    got, = torch.autograd.grad((r.logprob * r.lse.detach()).sum() + r.top_logprobs.detach().sum(), z)
    logp, lse = torch.log_softmax(z, 1), torch.logsumexp(z, 1).detach()
    want, = torch.autograd.grad((logp.gather(1, t[:, None])[:, 0] * lse).sum(), z)
    assert torch.allclose(got, want, rtol=0, atol=1e-12)


@pytest.mark.gpu
def test_the_kernels_node():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    z = torch.randn((5, 3001), generator=torch.Generator().manual_seed(1)).cuda().requires_grad_()
    t = torch.arange(5, device="cuda")
    r = L.token_logprobs(z, t, top=3)
    assert torch.autograd.grad(r.logprob.sum(), z, retain_graph=True)[0].isfinite().all()
    for loss in (r.logprob.sum() + r.lse.sum(), r.logprob.sum() + r.top_logprobs.sum()):
        with pytest.raises(RuntimeError, match="logprob and entropy only"):
            torch.autograd.grad(loss, z, retain_graph=True)
    d, = torch.autograd.grad(r.logprob.sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated twice"):
        d.square().sum().backward()

"""The example's serving step from compressed weights against the same step
in 64 bits on the uncompressed ones.  Each BF16 rounding on the way (y before
the experts, their sum, h) is 2^-9 of a value of its row's size; through the
output layer, whose rows have norm 3, a logit is off by a few times 3 * 2^-9 of
the size of h's elements, about 0.02, and 0.1 is allowed."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_step_against_64_bits():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import serve_step as S
    w = S.random_weights(seed=3)
    model = S.compress(w)
    g = torch.Generator(device="cuda").manual_seed(4)
    m, top_k = 9, 2
    x = torch.empty((m, 512), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.tensor([0, 1, -1, 2, 3, 1, 1, -1, 0], device="cuda")
    tokens = torch.randint(0, 1024, (m,), generator=g, device="cuda")
    scores, logits, gradient = S.step(model, x, ids, tokens, top_k=top_k, top=5)
    d = {k: v.double() for k, v in w.items()}
    y = x.double() @ d["projection"].T
    for t in range(m):
        if ids[t] >= 0:
            i = int(ids[t])
            y[t] += d["scales"][i] * (d["b"][i] @ (d["a"][i] @ x[t].double()))
    y = y.float().to(torch.bfloat16).double()
    h = x.double().clone()
    for t in range(m):
        l = d["router"] @ y[t]
        e = torch.argsort(l, descending=True)[:top_k]
        p = torch.softmax(l[e], 0)
        for w_e, i in zip(p, e):
            gate = d["w1"][i] @ y[t]
            h[t] += w_e * (d["w2"][i] @ (gate * torch.sigmoid(gate) * (d["w3"][i] @ y[t])))
    want = h @ d["output"].T
    assert float((logits.double() - want).abs().max()) < 0.1
    # the scores are those of the step's own logits
    z = logits.double()
    lse = torch.logsumexp(z, 1)
    assert torch.allclose(scores.logprob.double(), z.gather(1, tokens[:, None])[:, 0] - lse, atol=1e-5)
    assert torch.equal(scores.top_ids, torch.sort(z, dim=1, descending=True, stable=True).indices[:, :5])
    z.requires_grad_()
    logp = torch.log_softmax(z, 1)
    loss = -logp.gather(1, tokens[:, None]).mean() - 0.1 * -(logp.exp() * logp).sum(1).mean()
    loss.backward()
    assert torch.allclose(gradient.double(), z.grad, atol=1e-6)

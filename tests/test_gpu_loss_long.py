"""The cross entropy of so many rows that its calls take several launches for a
step of theirs, against 64 bits.

Tolerances, in the root mean square: half a unit of the type for the gradients' one
rounding (0.3 of that would do), as much again for the sums."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import loss as L  # noqa: E402

BF = torch.bfloat16
EPS = torch.finfo(BF).eps


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _normal(seed, dev, *shape, scale=1.0):
    t = torch.empty(shape, dtype=BF, device=dev)
    return t.normal_(0, scale, generator=torch.Generator(device=dev).manual_seed(seed))


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_gradient_of_more_numbers_than_threads(dev):
    """2^34 numbers of the hidden gradient, joined from fp32 sums by four a thread: a launch holds fewer than 2^32 threads."""
    m, v, k, few = 1 << 19, 264, 1 << 15, 1024
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info(dev)[0] < 230 << 30:
        pytest.skip("needs 230 GiB")
    w, base = _normal(1, dev, v, k, scale=k ** -0.5), _normal(2, dev, few, k)
    t = torch.randint(0, v, (few,), generator=torch.Generator(device=dev).manual_seed(3), device=dev)
    _say(f"[long] {m} rows of {k}")
    h = torch.empty((m, k), dtype=BF, device=dev)
    h.view(m // few, few, k).copy_(base)
    tokens = t.repeat(m // few)
    z = base.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    r = L.linear_cross_entropy(h, w, tokens)
    # logits of size up to 6, off by at most k 2^-24 of about 150
    assert float((r.lse.view(-1, few).double() - lse).abs().max()) < 0.3
    assert bool((r.lse.view(-1, few) == r.lse[:few]).all()) and bool((r.loss.view(-1, few) == r.loss[:few]).all())
    g = torch.softmax(z, 1)
    g.scatter_add_(1, t[:, None], torch.full((few, 1), -1.0, dtype=torch.float64, device=dev))
    one = torch.ones(m, device=dev)
    for rounded in (False, True):
        _say(f"[long]   gradients, rounded {rounded}")
        dh, dw = L.linear_cross_entropy_backward(h, w, tokens, r.lse, one, rounded=rounded)
        want = g @ w.double()
        for at in range(0, m // few, 37):  # every 37th of the repetitions, and the last
            assert _off(dh[few * at:few * (at + 1)], want) <= EPS, at
        assert _off(dh[m - few:], want) <= EPS
        assert _off(dw, (m // few) * (g.T @ base.double())) <= EPS
        del dh, dw

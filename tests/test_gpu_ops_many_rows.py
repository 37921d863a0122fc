"""Sizes whose blocks, times their threads, pass the 2^32 that one launch takes:
the calls make several launches of them.  Whole numbers, so that results are
exact or nearly so."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import adapters as A, logprobs as L  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def test_rows_of_logits(dev):
    m, v = (1 << 24) + 9, 5
    _say(f"[many rows] logits {m} x {v}")
    g = torch.Generator(device=dev).manual_seed(1)
    z = torch.randint(-4, 5, (m, v), generator=g, device=dev).to(HF)
    t = torch.randint(0, v, (m,), generator=g, device=dev)
    r = L.token_logprobs(z, t, top=2)
    logp = torch.log_softmax(z.double(), 1)
    assert float((r.logprob - logp.gather(1, t[:, None])[:, 0]).abs().max()) < 1e-5
    assert float((r.entropy + (logp.exp() * logp).sum(1)).abs().max()) < 1e-5
    key = z.to(torch.int64) * 8 - torch.arange(v, device=dev)  # equal logits by their index
    assert torch.equal(r.top_ids, key.topk(2, dim=1).indices)
    gl = torch.randint(1, 4, (m,), generator=g, device=dev).float()
    d = L.token_logprobs_backward(z, t, r.lse, r.entropy, gl)
    want = (torch.nn.functional.one_hot(t, v) - logp.exp()) * gl.double()[:, None]
    assert float((d - want).abs().max()) < 2.0 ** -9  # values up to 3, rounded to half precision


@pytest.mark.parametrize("n", [3, (1 << 18) + 5])
def test_tokens_with_adapters(dev, n):
    """Tiles of 128 tokens, and of 16."""
    m, cols = (1 << 24) + 37, 8
    _say(f"[many rows] {m} tokens of {n} adapters")
    g = torch.Generator(device=dev).manual_seed(2)
    x, a, b = (torch.randint(-3, 4, s, generator=g, device=dev).to(BF) for s in ((m, cols), (n, 1, cols), (n, 1, 1)))
    ids = torch.randint(-1, n, (m,), generator=g, device=dev).sort().values
    y = torch.ones((m, 1), device=dev)
    A.add_adapters(x, y, a, b, ids)
    at = ids.clamp(min=0)
    want = 1 + (x.float() * a[at, 0].float()).sum(1) * b[at, 0, 0].float() * (ids >= 0)
    assert torch.equal(y[:, 0], want)


def test_rows_of_one_token(dev):
    rows = (1 << 29) + 3
    _say(f"[many rows] one token, {rows} rows")
    x, a = torch.full((1, 8), 2.0, dtype=BF, device=dev), torch.full((1, 1, 8), 3.0, dtype=BF, device=dev)
    b = (torch.arange(rows, device=dev, dtype=torch.int32) % 7).to(BF).view(1, rows, 1)
    y = torch.ones((1, rows), dtype=BF, device=dev)
    A.add_adapters(x, y, a, b, torch.zeros(1, dtype=torch.int64, device=dev))
    want = (1 + 48 * b.view(1, rows).float()).to(BF)  # 1 + 288 at most: rounded once
    assert torch.equal(y, want)

"""Operators on a stream of the caller's, with arguments that have to be
copied first (strided, not 16-byte aligned, expanded), while the current
stream is busy: copies and kernels belong to the given stream, so the results
are there when that stream is done, whatever the current one does."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import adapters as A, logprobs as L, moe as M  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def busy(dev):
    """Keeps the current stream at work for some tens of milliseconds."""
    w = torch.randn((4096, 4096), device=dev, dtype=BF) / 64
    out = torch.empty_like(w)

    def go():
        for _ in range(300):
            torch.mm(w, w, out=out)
    go()
    torch.cuda.synchronize()
    return go


def _shifted(t):
    """t in memory that is not 16-byte aligned."""
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.flatten()
    return flat[1:].view(t.shape)


def _apart(t):
    """t with a stride of two elements in its last dimension."""
    wide = torch.zeros((*t.shape, 2), dtype=t.dtype, device=t.device)
    wide[..., 0] = t
    return wide[..., 0]


def _on_stream(call, want, busy, what):
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        _say(f"[streams] {what} on {stream}")
        torch.cuda.synchronize()
        busy()
        got = call(stream)
        side.synchronize()
        with torch.cuda.stream(side):
            same = [torch.equal(g, w) for g, w in zip(got, want)]
        torch.cuda.synchronize()
        assert all(same), f"{what}: {same}"


def test_token_logprobs(dev, busy):
    z = torch.randn((33, 5003), device=dev)
    t = torch.arange(33, device=dev)
    want = L.token_logprobs(z, t, top=5)
    zt, ta = z.t().contiguous().t(), _apart(t)
    _on_stream(lambda s: L.token_logprobs(zt, ta, top=5, check=False, stream=s), want, busy, "token_logprobs")
    _on_stream(lambda s: L.token_logprobs(zt, ta, top=5, stream=s), want, busy, "token_logprobs, checked")


def test_token_logprobs_backward(dev, busy):
    z = torch.randn((33, 5003), device=dev)
    t = torch.arange(33, device=dev)
    r = L.token_logprobs(z, t)
    one = torch.full((1,), 0.25, device=dev).expand(33)
    want = L.token_logprobs_backward(z, t, r.lse, r.entropy, one.contiguous(), one.contiguous())
    zt, ta, lse, ent = z.t().contiguous().t(), _apart(t), _apart(r.lse), _apart(r.entropy)
    _on_stream(lambda s: [L.token_logprobs_backward(zt, ta, lse, ent, one, one, check=False, stream=s)], [want], busy,
               "token_logprobs_backward")


@pytest.mark.parametrize("m", [5, 700])
def test_add_adapters(dev, busy, m):
    n, rank, cols, rows = 3, 20, 520, 300
    x, a, b = (torch.randn(s, device=dev).to(BF) for s in ((m, cols), (n, rank, cols), (n, rows, rank)))
    ids, scales = torch.arange(m, device=dev) % n, torch.rand(n, device=dev)
    y = torch.randn((m, rows), device=dev)
    want = A.add_adapters(x, y.clone(), a, b, ids, scales)
    xs, ia, sa = _shifted(x), _apart(ids), _apart(scales)
    out = [y.clone() for _ in range(2)]
    _on_stream(lambda s: [A.add_adapters(xs, out.pop(), a, b, ia, sa, check=False, stream=s)], [want], busy,
               f"add_adapters of {m} tokens")


@pytest.mark.parametrize("m", [1, 40])
def test_moe_layer(dev, busy, m):
    e, h, i = 6, 512, 264
    x, r, w1, w3, w2 = (torch.randn(s, device=dev).to(BF) / 16 for s in ((m, h), (e, h), (e, i, h), (e, i, h), (e, h, i)))
    want = M.moe_layer(x, r, w1, w3, w2, 2)
    xs, rs = _shifted(x), _shifted(r)
    _on_stream(lambda s: [M.moe_layer(xs, rs, w1, w3, w2, 2, stream=s)], [want], busy, f"moe_layer of {m} tokens")

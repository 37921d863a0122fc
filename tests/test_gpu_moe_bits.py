"""What the experts' layer keeps of h = silu(W1 x) * (W3 x).

The cases' numbers are whole (times a power of two), so that every product
and sum before h is exact in fp32: with a gate of 41, 1 + exp(-41) is 1 and
h = 41 times a whole number below 2^16, which has up to 22 bits.  A row of W2
takes the difference of two such h, 41 d with d = -6..6: exact in every type,
if h is kept whole, and off by 41 or more where h keeps 16 bits.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import moe as M  # noqa: E402

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _whole(m, inner, experts, dtype, size, seed):
    """Tokens, router and experts as above; h is 41 size whole numbers, y the differences d 41."""
    g = torch.Generator().manual_seed(seed)
    cols, pairs = 16, inner // 2
    x = torch.randint(-80, 81, (m, cols), generator=g).double()
    x[:, 0] = x[:, 1] = 1.0
    router = torch.zeros((experts, cols), dtype=torch.float64)
    router[:, 2:] = torch.randint(-3, 4, (experts, cols - 2), generator=g)
    w1 = torch.zeros((experts, inner, cols), dtype=torch.float64)
    w1[:, :, 0] = 41.0
    w3 = torch.randint(-50, 51, (experts, inner, cols), generator=g).double()
    w3[:, :, 0] = 0.0
    w3[:, pairs:] = w3[:, :pairs]
    d = torch.randint(1, 7, (experts, pairs), generator=g).double()
    w3[:, pairs:, 1] += d
    w2 = torch.zeros((experts, cols, inner), dtype=torch.float64)
    at = torch.randint(0, pairs, (experts, cols), generator=g)
    sign = torch.randint(0, 2, (experts, cols), generator=g).double() * 2 - 1
    w2.scatter_(2, at[:, :, None], -sign[:, :, None])
    w2.scatter_(2, at[:, :, None] + pairs, sign[:, :, None])
    best = torch.sort(x @ router.T, dim=1, descending=True, stable=True).indices[:, 0]
    want = (41.0 * sign * d.gather(1, at))[best]
    args = (x, router, w1, w3 * size, w2 / size)
    cast = [a.to(dtype) for a in args]
    assert all(torch.equal(c.double(), a) for c, a in zip(cast, args))
    assert float((x @ w3.flatten(0, 1).T).abs().max()) < 2.0 ** 16
    return cast, want


# the last of inner's strips of 256 partial, and tokens over one, two and four tiles
@pytest.mark.parametrize("m,inner,experts", [(1, 64, 5), (1, 1032, 3), (2, 64, 5), (15, 1032, 3), (16, 8, 1), (33, 264, 2),
                                             (64, 520, 1), (64, 2056, 40)])
@pytest.mark.parametrize("dtype,size", [(BF, 1.0), (BF, 2.0 ** 40), (BF, 2.0 ** -60), (HF, 1.0), (HF, 2.0 ** 9),
                                        (HF, 2.0 ** -8)])
def test_h_is_kept_whole(dev, dtype, size, m, inner, experts):
    _say(f"[moe bits] {dtype} h times {size}, {m} tokens, {experts} experts, inner {inner}")
    args, want = _whole(m, inner, experts, dtype, size, m + inner)
    for renorm in (True,) if experts > 1 else (True, False):
        y = M.moe_layer(*[a.to(dev) for a in args], 1, renormalize=renorm)
        assert torch.equal(y.double().cpu(), want)


@pytest.mark.parametrize("m", [1, 2, 17, 40])
def test_half_precision_h_far_above_and_below_one(dev, m):
    """h of about 2^25 with W2 of 2^-14, and of 2^-21 with W2 of 2^14: the error
    is that of fp32 sums and of one rounding, at any size of h."""
    g = torch.Generator().manual_seed(m)
    cols, inner, eps = 64, 136, 2.0 ** -24

    def values(*shape):  # of half to one, either sign: none is subnormal after the scaling
        return (0.5 + 0.5 * torch.rand(shape, generator=g)) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    for f0, f1, f3, f2 in ((1.0, 2.0 ** 10, 2.0 ** 10, 2.0 ** -14), (2.0 ** -6, 2.0 ** -6, 2.0 ** -7, 2.0 ** 14)):
        x = (values(m, cols) * f0).to(HF)
        w1, w3 = (values(1, inner, cols) * f1).to(HF), (values(1, inner, cols) * f3).to(HF)
        w2 = (torch.randn((1, cols, inner), generator=g).sign() * f2).to(HF)
        w2 *= torch.rand(w2.shape, generator=g) < 0.02  # few terms: h's own error is not averaged away
        a, b, c, v = w1[0].double(), w3[0].double(), w2[0].double(), x.double()
        gate, up = v @ a.T, v @ b.T
        dg, du = (cols + 24) * eps * (v.abs() @ a.abs().T), (cols + 24) * eps * (v.abs() @ b.abs().T)
        s = gate / (1 + (-gate).exp())
        h = s * up
        dh = 1.1 * dg * (up.abs() + du) + (s.abs() + 1.1 * dg) * du + h.abs() * eps * (2 * gate.abs() + 8)
        dh += 2.0 ** -21 * h.abs() + 2.0 ** -37 * h.abs().amax(1, keepdim=True)
        want = h @ c.T
        tol = dh @ c.abs().T + (4 * inner + 24) * eps * (h.abs() @ c.abs().T) + 1.01 * 2.0 ** -11 * want.abs() + 2.0 ** -24
        assert float(want.abs().max()) < 65504
        y = M.moe_layer(x.to(dev), torch.zeros((1, cols), dtype=HF, device=dev), w1.to(dev), w3.to(dev), w2.to(dev), 1)
        err = (y.double().cpu() - want).abs()
        assert bool((err <= tol).all()), f"weights times {f1}: worst {float((err / tol).max())} of its tolerance"


def test_an_infinite_h_is_the_infinity_of_its_sum(dev):
    """h past fp32's range: y is its infinity, not NaN, where W2 gives it a sign and no other infinity meets it."""
    for m in (1, 3):
        x = torch.zeros((m, 8), dtype=BF)
        x[:, 0] = 2.0 ** 40
        w1 = torch.zeros((1, 8, 8), dtype=BF)
        w3 = torch.zeros((1, 8, 8), dtype=BF)
        w1[0, 3, 0] = w3[0, 3, 0] = 2.0 ** 30
        w2 = torch.full((1, 8, 8), -0.5, dtype=BF)
        y = M.moe_layer(x.to(dev), torch.zeros((1, 8), dtype=BF, device=dev), w1.to(dev), w3.to(dev), w2.to(dev), 1)
        assert bool((y == -float("inf")).all())


def test_half_precision_repeats_and_graph(dev):
    """FP16's scaling comes from each call's own h: nothing of a call with larger h is left for the next."""
    g = torch.Generator().manual_seed(3)
    m, e, h, i = 40, 6, 256, 264
    x, r, w1, w3, w2 = ((torch.randn(s, generator=g) / f).to(HF).to(dev) for s, f in (
        ((m, h), 1.0), ((e, h), 16.0), ((e, i, h), 16.0), ((e, i, h), 16.0), ((e, h, i), 16.0)))
    y1 = M.moe_layer(x, r, w1, w3, w2, 2)
    assert torch.equal(M.moe_layer(x, r, w1, w3, w2, 2), y1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = M.moe_layer(x, r, w1, w3, w2, 2)
    for k, f in enumerate((1.0, 2.0 ** 10, 2.0 ** -10, 1.0, 2.0 ** -12)):
        w3.copy_((torch.randn((e, i, h), generator=g) * f / 16).to(HF))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, M.moe_layer(x, r, w1, w3, w2, 2)), f"replay {k}"

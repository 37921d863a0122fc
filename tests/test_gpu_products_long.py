"""The products on operands and results of more than 2^32 bytes, where a place
in 32 bits would come round: against 64 bits, in pieces, whole or in the rows
where it would show (the first, the last, and those after 2^31 and 2^32 bytes).

Tolerances.  Of single results: half a unit of the type, and of n products
summed in fp32 n 2^-24 of their sizes' sum (their root mean square would do).
Of whole gradients, in the root mean square: G's and the result's roundings, eps / 2
each, and eps / 2 more for the sums."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd.fourbit import Weights4, linear4, quantize4  # noqa: E402
from lossless_weight_compression_bf16_amd.grouped import grouped_linear, grouped_linear_backward  # noqa: E402
from lossless_weight_compression_bf16_amd.loss import linear_cross_entropy, linear_cross_entropy_backward  # noqa: E402

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


def _near(got, want, size, n, what):
    err, tol = (got.double() - want).abs(), EPS / 2 * 1.01 * want.abs() + n * 2.0 ** -24 * size
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).max())} of its tolerance"


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_a_large_vocabulary(dev):
    v, k = 600_000, 4096  # 4.9 GB
    w = _normal(1, dev, v, k, scale=k ** -0.5)
    for m in (1, 3, 40, 300):
        _say(f"[long] loss of {m} rows, vocabulary of {v}")
        h = _normal(2, dev, m, k)
        tokens = v - 1 - torch.arange(m, device=dev) * (v // 300)
        z = torch.cat([h.double() @ c.double().T for c in w.split(50_000)], 1)
        lse = torch.logsumexp(z, 1)
        loss = lse - z.gather(1, tokens[:, None])[:, 0]
        r = linear_cross_entropy(h, w, tokens)
        # logits of size up to 6, off by at most k 2^-24 of about 60, and what exp and log add
        assert float((r.lse.double() - lse).abs().max()) < 2e-3 and float((r.loss.double() - loss).abs().max()) < 2e-3
        g = torch.softmax(z, 1)
        g.scatter_add_(1, tokens[:, None], torch.full((m, 1), -1.0, dtype=torch.float64, device=dev))
        dh, dw = linear_cross_entropy_backward(h, w, tokens, r.lse, torch.ones(m, device=dev))
        want = sum(g[:, i:i + 50_000] @ w[i:i + 50_000].double() for i in range(0, v, 50_000))
        assert _off(dh, want) <= 1.5 * EPS
        for rows in (slice(0, 512), slice(262_000, 263_000), slice(524_000, 525_000), slice(v - 512, v)):
            assert _off(dw[rows], g[:, rows].T @ h.double()) <= 1.5 * EPS, rows
        del z, g, dw


def test_many_rows_of_experts(dev):
    m, k, n = 1_100_000, 2048, 64  # x of 4.5 GB
    x, w = _normal(1, dev, m, k), _normal(2, dev, 3, n, k, scale=k ** -0.5)
    ends = torch.tensor([400_001, 1_050_003, m], device=dev)
    expert = torch.zeros(m, dtype=torch.int64, device=dev)
    expert[400_001:] += 1
    expert[1_050_003:] += 1
    _say("[long] grouped products of many rows")
    y = grouped_linear(x, w, ends)
    d = _normal(3, dev, m, n)
    dx, dw = grouped_linear_backward(x, w, ends, d)
    for rows in (slice(0, 300), slice(399_900, 400_100), slice(524_200, 524_400), slice(1_048_500, 1_050_100), slice(m - 300, m)):
        for e in expert[rows].unique().tolist():
            a, b, c = (t[rows][expert[rows] == e].double() for t in (x, d, dx))
            we = w[e].double()
            _near(y[rows][expert[rows] == e], a @ we.T, a.abs() @ we.abs().T, k, f"y {rows}")
            _near(c, b @ we, b.abs() @ we.abs(), n, f"dx {rows}")
    lo = 0
    for e, hi in enumerate(ends.tolist()):
        want = sum(d[i:min(i + 50_000, hi)].double().T @ x[i:min(i + 50_000, hi)].double() for i in range(lo, hi, 50_000))
        assert _off(dw[e], want) <= EPS
        lo = hi


@pytest.mark.parametrize("m", [2, 70, 900])
def test_many_experts_of_large_weights(dev, m):
    experts, n, k = 40, 8192, 8192  # 5.4 GB
    w = _normal(1, dev, experts, n, k, scale=k ** -0.5)
    x, d = _normal(2, dev, m, k), _normal(3, dev, m, n)
    used = {0: m // 2, 16: m // 2 + m // 4, 39: m}  # the rows of three experts end there
    ends = torch.tensor([max([0] + [h for f, h in used.items() if f <= e]) for e in range(experts)], device=dev)
    _say(f"[long] {m} rows of large experts")
    y = grouped_linear(x, w, ends)
    dx, dw = grouped_linear_backward(x, w, ends, d)
    lo = 0
    for e, hi in used.items():
        if hi == lo:
            continue
        we = w[e].double()
        a, b = x[lo:hi].double(), d[lo:hi].double()
        _near(y[lo:hi], a @ we.T, a.abs() @ we.abs().T, k, f"y of {e}")
        _near(dx[lo:hi], b @ we, b.abs() @ we.abs(), n, f"dx of {e}")
        _near(dw[e], b.T @ a, b.abs().T @ a.abs(), hi - lo, f"dw of {e}")
        lo = hi
    assert not bool(dw[1].any()) and not bool(dw[38].any())


def test_many_weights_of_4_bits(dev):
    rows, cols = (1 << 20) + 24, 8192  # 4.3 GB, and 8.6 GB of results for 4096 rows
    g = torch.Generator(device=dev).manual_seed(1)
    q = torch.randint(0, 256, (rows, cols // 2), generator=g, device=dev, dtype=torch.uint8)
    s = (torch.rand((rows, cols // 32), generator=g, device=dev) * cols ** -0.5).to(BF)
    z = (7 + torch.rand((rows, cols // 32), generator=g, device=dev)).to(BF)
    w = Weights4(q, s, z, 32)
    for m in (1, 20, 2100):
        _say(f"[long] {m} rows, {rows} rows of weights of 4 bits")
        x = _normal(2, dev, m, cols)
        y = linear4(x, w)
        for at in (slice(0, 64), slice(524_200, 524_400), slice(rows - 100, rows)):
            v = torch.stack([q[at] & 15, q[at] >> 4], 2).view(-1, cols // 32, 32).double()
            f = lambda t: t[at].double()[..., None]  # noqa: E731
            dense = (f(s) * (v - f(z))).reshape(-1, cols)
            size = (f(s) * (32 + v + f(z))).reshape(-1, cols)
            _near(y[:, at], x.double() @ dense.T, x.double().abs() @ size.T, cols, f"{m} {at}")
        del y
    dense = _normal(3, dev, 300_000, cols)  # 4.9 GB
    got = quantize4(dense, 128, True)
    want = quantize4(dense[-1000:], 128, True)
    assert all(torch.equal(a[-1000:], b) for a, b in zip(got[:3], want[:3]))

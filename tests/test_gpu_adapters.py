"""Low-rank adapters against y + s B (A x) in 64 bits.

Tolerance.  u = A x is summed in fp32 from exact products: off by at most
(cols + 24) 2^-24 sum |a x|.  It enters the second product as 16-bit terms:
of BF16 three (rest below 2^-24 of each value), of FP16 two after a scaling
per token (rest below 2^-21 of the token's largest value).  The second
product sums 3 rank_pad exact products in fp32.  Then one addition in fp32
and one rounding to the type of y.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import _binding as B, adapters as A  # noqa: E402

EPS = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
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


def _inputs(m, n, rank, cols, rows, dtype, ydtype, seed, order="mixed"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, cols), generator=g).to(dtype)
    a = (torch.randn((n, rank, cols), generator=g) / cols ** 0.5).to(dtype)
    b = torch.randn((n, rows, rank), generator=g).to(dtype)
    y = torch.randn((m, rows), generator=g).to(ydtype)
    ids = torch.randint(-1, n, (m,), generator=g)
    if order == "runs":
        ids = ids.sort().values[torch.randperm(1, generator=g)[0]:]
    s = 0.5 + torch.rand(n, generator=g)
    return x, y, a, b, ids, s


def _expect(x, y, a, b, ids, s):
    """The result and its tolerance, in 64 bits."""
    x, a, b = x.double(), a.double(), b.double()
    want, tol = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    cols, rank = x.shape[1], a.shape[1]
    pad = (rank + 15) // 16 * 16
    for i in range(a.shape[0]):
        t = torch.nonzero(ids == i)[:, 0]
        if not t.numel():
            continue
        f = 1.0 if s is None else float(s[i])
        u = f * (x[t] @ a[i].T)
        um = abs(f) * (x[t].abs() @ a[i].abs().T)
        want[t] += u @ b[i].T
        du = (cols + 24) * EPS * um + 2 ** -21 * u.abs().amax(1, keepdim=True)
        tol[t] += (du + 3 * pad * EPS * u.abs()) @ b[i].abs().T
    tol += ROUND[y.dtype] * want.abs() * 1.01 + EPS * (want.abs() + y.double().abs()) + torch.finfo(y.dtype).tiny
    return want, tol


def _check(args, dev, what):
    _say(f"[adapters] {what}")
    want, tol = _expect(*args)
    d = [None if t is None else t.to(dev) for t in args]
    y = A.add_adapters(*d)
    assert y is d[1]
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).max())} of its tolerance"
    none = args[4] < 0
    assert torch.equal(y.cpu()[none], args[1][none]), f"{what}: rows without an adapter changed"


SIZES = [(1, 1, 1, 8, 1), (1, 8, 16, 4096, 4096), (3, 2, 5, 40, 17), (16, 16, 16, 256, 64), (17, 3, 20, 264, 100),
         (61, 32, 16, 512, 1000), (64, 1, 33, 136, 72), (100, 7, 64, 520, 257), (5, 3, 256, 104, 50),
         (70, 5, 130, 64, 33), (513, 4, 16, 256, 65), (600, 700, 8, 64, 40), (700, 5, 20, 1032, 300),
         (1000, 3, 100, 72, 130), (520, 2, 200, 264, 96), (530, 3, 64, 96, 600), (256, 4, 48, 264, 130), (640, 11, 70, 136, 90),
         (700, 90, 40, 1064, 520)]


@pytest.mark.parametrize("dtype,ydtype", [(BF, F32), (BF, BF), (HF, F32), (HF, HF)])
@pytest.mark.parametrize("size", SIZES)
def test_against_64_bits(dev, dtype, ydtype, size):
    _check(_inputs(*size, dtype, ydtype, sum(size)), dev, f"{dtype} {ydtype} {size}")
    _check(_inputs(*size, dtype, ydtype, sum(size), "runs"), dev, f"{dtype} {ydtype} {size} in runs")


@pytest.mark.parametrize("ids", [[-1] * 5, [2] * 5, [0, 1, 2, 1, 0], [-1, -1, 0, -1, -1]])
def test_orders(dev, ids):
    x, y, a, b, _, s = _inputs(5, 3, 16, 128, 96, BF, F32, 1)
    _check((x, y, a, b, torch.tensor(ids), s), dev, f"ids {ids}")
    _check((x, y, a, b, torch.tensor(ids), None), dev, f"ids {ids}, no scales")


@pytest.mark.parametrize("m", [7, 600])
def test_strides(dev, m):
    x, y, a, b, ids, s = _inputs(m, 4, 16, 128, 96, BF, BF, 2)
    want, tol = _expect(x, y, a, b, ids, s)
    d = [t.to(dev) for t in (x, a, b, ids, s)]
    for xs, ys in ((136, 97), (129, 103), (128, 96)):
        for shift in (0, 1):
            wx = torch.zeros((m, xs + 8), dtype=BF, device=dev)
            vx = wx[:, shift:128 + shift]
            vx.copy_(d[0])
            wy = torch.full((m, ys + 2), 5.0, dtype=BF, device=dev)
            vy = wy[:, shift:96 + shift]
            vy.copy_(y)
            A.add_adapters(vx, vy, d[1], d[2], d[3], d[4])
            assert bool(((vy.double().cpu() - want).abs() <= tol).all()), (xs, ys, shift)
            rest = wy.clone()
            rest[:, shift:96 + shift] = 5.0
            assert bool((rest == 5.0).all()), "elements beside y changed"


@pytest.mark.parametrize("m", [6, 640])
def test_nan_and_infinity_stay_in_their_rows(dev, m):
    for dtype in (BF, HF):
        x, y, a, b, _, s = _inputs(m, 2, 16, 128, 96, dtype, F32, 3)
        ids = torch.zeros(m, dtype=torch.int64)
        ids[1] = 1
        want, tol = _expect(x, y, a, b, ids, s)
        x[2, 5] = float("nan")
        x[4, 7] = float("inf")
        got = A.add_adapters(*[t.to(dev) for t in (x, y, a, b, ids, s)]).double().cpu()
        ok = torch.ones(m, dtype=torch.bool)
        ok[[2, 4]] = False
        assert bool(((got - want).abs() <= tol)[ok].all())
        assert bool(got[2].isnan().all()) and not bool(got[4].isfinite().any())
        # a NaN in an adapter reaches its own tokens only
        a[1, 3, 3] = float("nan")
        x[2, 5] = x[4, 7] = 0.0
        want, tol = _expect(x, y, a, b, ids, s)
        got = A.add_adapters(*[t.to(dev) for t in (x, y, a, b, ids, s)]).double().cpu()
        ok = ids == 0
        assert bool(((got - want).abs() <= tol)[ok].all()) and bool(got[1].isnan().all())


def test_intermediate_beyond_half_range(dev):
    """A x past 65504 and far below 2^-24 with FP16 adapters: u is held in 32 bits."""
    for f in (2000.0, 2.0 ** -12):
        x, y, a, b, ids, s = _inputs(40, 2, 24, 256, 64, HF, F32, 4)
        ids.clamp_(min=0)
        x = (x * f).to(HF)
        a = (a * f).to(HF)
        y.zero_()
        _check((x, y, a, b, ids, s), dev, f"inputs times {f}")


def test_repeats_streams_and_graph(dev):
    for m in (33, 700):
        x, y, a, b, ids, s = [t.to(dev) for t in _inputs(m, 9, 20, 520, 300, BF, F32, 5)]
        want = A.add_adapters(x, y.clone(), a, b, ids, s)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        for stream in (None, st, st.cuda_stream):
            y2 = y.clone()
            torch.cuda.synchronize()
            assert torch.equal(A.add_adapters(x, y2, a, b, ids, s, stream=stream), want)
        y2 = y.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            A.add_adapters(x, y2, a, b, ids, s, check=False)
        for k in range(4):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)))
            y2.copy_(y)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y2, A.add_adapters(x, y.clone(), a, b, ids, s)), f"replay {k}"


def test_offsets_past_32_bits(dev):
    """y and the adapters' B of more than 2^32 bytes."""
    m, rows, n = 3, 1 << 20, 140
    x, _, a, _, _, s = _inputs(m, n, 16, 64, 8, BF, F32, 6)
    b = torch.zeros((n, rows, 16), dtype=BF, device=dev)
    assert b.numel() * 2 > 1 << 32
    b[-1, :, 3] = 1.0
    wide = torch.zeros((m, (1 << 30) + 8), dtype=BF, device=dev)
    y = wide[:, :rows]
    ids = torch.tensor([n - 1, -1, n - 1], device=dev)
    A.add_adapters(x.to(dev), y, a.to(dev), b, ids, s.to(dev))
    u = float(s[-1]) * (x.double() @ a[-1, 3].double())
    for t, w in ((0, float(u[0])), (1, 0.0), (2, float(u[2]))):
        assert bool(((y[t].double() - w).abs() <= abs(w) * 2.0 ** -8).all()), t


def test_no_rows_and_no_adapters(dev):
    x, y, a, b, ids, s = [t.to(dev) for t in _inputs(4, 2, 8, 64, 32, BF, F32, 7)]
    assert A.add_adapters(x[:0], y[:0], a, b, ids[:0], s).shape == (0, 32)
    z = y.clone()
    A.add_adapters(x, z, a[:0], b[:0], torch.full_like(ids, -1), s[:0])
    assert torch.equal(z, y)


def test_refusals(dev):
    x, y, a, b, ids, s = [t.to(dev) for t in _inputs(4, 2, 8, 64, 32, BF, F32, 7)]
    for args in ((x.cpu(), y, a, b, ids, s), (x, y.cpu(), a, b, ids, s), (x, y[:3], a, b, ids, s),
                 (x, y, a[:, :, :56], b, ids, s), (x, y, a, b[:, :31], ids, s), (x, y, a, b, ids[:3], s),
                 (x, y, a, b, ids.int(), s), (x, y, a, b, ids, s[:1]), (x, y, a, b, ids, s.half()),
                 (x, y[:1].expand(4, 32), a, b, ids, s), (x, y, a.transpose(0, 1), b, ids, s),
                 (x[:, :60], y, a[:, :, :60].contiguous(), b, ids, s), (x[0], y, a, b, ids, s),
                 (x, y, a[:, :0], b[:, :, :0], ids, s), (x, y[:, ::2], a, b[:, :16].contiguous(), ids, s),
                 (x, y, a.new_zeros((2, 257, 64)), b.new_zeros((2, 32, 257)), ids, s)):
        with pytest.raises(ValueError):
            A.add_adapters(*args)
    for args in ((x.float(), y, a, b, ids, s), (x, y.half(), a, b, ids, s), (x, y, a.half(), b, ids, s)):
        with pytest.raises(TypeError):
            A.add_adapters(*args)
    ids[2] = 2
    z = y.clone()
    with pytest.raises(B.WcError, match="index out of range"):
        A.add_adapters(x, z, a, b, ids, s)
    assert torch.equal(z[2], y[2])


@pytest.mark.parametrize("m", [5, 300])
def test_no_adapters_at_all(dev, m):
    x, y, a, b, _, _ = _inputs(m, 1, 16, 128, 96, BF, F32, 8)
    got = A.add_adapters(x.to(dev), y.to(dev), a[:0].to(dev), b[:0].to(dev), torch.full((m,), -1, device=dev))
    assert torch.equal(got.cpu(), y)

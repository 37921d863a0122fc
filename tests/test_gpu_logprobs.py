"""Log probabilities of given tokens against their definition in 64 bits.

Tolerances.  A row's S is a sum of V terms, V / 256 of them one after the
other in a thread, each 2^d with d = (z - m) log2 e rounded once and m log2 e
rounded once: relative errors of 2^-24 (V / 256 + |m| + |d| + a few joins),
where the terms' |d| weighted by their size stay below 30.  So lse, and with
it a log probability, is off by at most 2^-24 (V / 256 + 2 |m| + |result| +
64), and the entropy by twice that times (1 + H).  Indices are exact.
A gradient's element is p times a bracket: p is off by 2^-24 (|log p| + 4)
of itself, the bracket by as much of its terms, and one rounding to the type
follows.
"""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import _binding as B, logprobs as L  # noqa: E402

EPS = 2.0 ** -24
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _logits(m, v, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((m, v), generator=g) * std).to(dtype)


def _order(z, n):
    """The n best of a row: larger first, equal by index, NaN last."""
    z = np.where(z == 0, 0.0, z)
    nan = np.isnan(z)
    return np.lexsort((np.arange(z.size), np.where(nan, 0.0, -z), nan))[:n]


def _expect(z, t):
    """lse, logprob, entropy of one row (float64) for token t."""
    if np.isnan(z).any() or np.isposinf(z).any():
        lse = ent = math.nan
    elif np.isneginf(z).all():
        lse, ent = -math.inf, 0.0
    else:
        m = z.max()
        e = np.exp(z - m)
        lse = m + math.log(e.sum())
        d = z[e > 0] - m
        ent = math.log(e.sum()) - float((e[e > 0] * d).sum() / e.sum())
    if t == -1:
        return lse, 0.0, ent
    if not 0 <= t < z.size:
        return lse, math.nan, ent
    lp = -math.inf if np.isneginf(z[t]) and not math.isnan(lse) else z[t] - lse
    return lse, lp, ent


def _near(got, want, tol, what):
    if math.isnan(want) or math.isinf(want):
        assert (math.isnan(got) and math.isnan(want)) or got == want, f"{what}: got {got} want {want}"
    else:
        assert abs(got - want) <= tol, f"{what}: got {got} want {want} tolerance {tol}"


def _check(z, tokens, top, r, what, rows=None):
    zs = z.double().cpu().numpy()
    r = [None if t is None else t.cpu().numpy() for t in r]
    for i in range(zs.shape[0]) if rows is None else rows:
        row, t = zs[i], int(tokens[i])
        lse, lp, ent = _expect(row, t)
        fin = row[np.isfinite(row)]
        big = np.abs(fin).max() if fin.size else 0.0
        tol = EPS * (row.size / 256 + 2 * big + 64)
        _near(r[2][i], lse, tol + EPS * abs(lse if math.isfinite(lse) else 0), f"{what} row {i} lse")
        _near(r[0][i], lp, tol + EPS * abs(lp if math.isfinite(lp) else 0), f"{what} row {i} logprob")
        _near(r[1][i], ent, 2 * tol * (1 + (ent if ent == ent else 0)), f"{what} row {i} entropy")
        if top:
            want = _order(row, top)
            assert np.array_equal(r[4][i], want), f"{what} row {i}: top {r[4][i]} want {want}"
            for q, j in enumerate(want):
                _, w, _ = _expect(row, int(j))
                _near(r[3][i][q], w, tol + EPS * abs(w if math.isfinite(w) else 0), f"{what} row {i} top {q}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,v,top", [(1, 1, 1), (1, 1, 0), (3, 2, 2), (5, 7, 3), (2, 8, 8), (4, 63, 63), (3, 64, 64),
                                     (2, 255, 5), (7, 2048, 20), (3, 2049, 64), (2, 8192, 1), (2, 8193, 64),
                                     (1, 50257, 64), (5, 50257, 5), (3, 50257, 0), (2, 131073, 20), (1100, 1000, 6),
                                     (1, 300001, 33)])
def test_against_64_bits(dev, dtype, m, v, top):
    _say(f"[logprobs] {dtype} {m} x {v}, top {top}")
    z = _logits(m, v, dtype, 7 * m + v)
    g = torch.Generator().manual_seed(v)
    t = torch.randint(0, v, (m,), generator=g)
    t[m // 2] = -1
    r = L.token_logprobs(z.to(dev), t.to(dev), top=top)
    _check(z, t, top, r, f"{dtype} {m}x{v}", rows=range(0, m, 97) if m > 100 else None)


def _special_rows(v, dtype):
    g = torch.Generator().manual_seed(3)
    base = (torch.randn(v, generator=g) * 2).to(dtype)
    low = torch.finfo(dtype).min
    high = torch.finfo(dtype).max
    rows = {}
    rows["all -inf"] = torch.full((v,), -math.inf, dtype=dtype)
    rows["all lowest"] = torch.full((v,), low, dtype=dtype)
    rows["all highest"] = torch.full((v,), high, dtype=dtype)
    rows["equal"] = torch.full((v,), 1.5, dtype=dtype)
    one = rows["all -inf"].clone()
    one[v // 2] = 3.0
    rows["one token left"] = one
    few = rows["all lowest"].clone()
    few[[1, v // 3, v - 1]] = torch.tensor([0.5, 0.25, 0.5], dtype=dtype)
    rows["three tokens above the lowest"] = few
    half = base.clone()
    half[::2] = -math.inf
    rows["every second masked"] = half
    nan = base.clone()
    nan[v // 4] = math.nan
    rows["a NaN"] = nan
    mostly = torch.full((v,), math.nan, dtype=dtype)
    mostly[v // 5] = -math.inf
    mostly[v // 2] = 1.0
    rows["mostly NaN"] = mostly
    rows["all NaN"] = torch.full((v,), math.nan, dtype=dtype)
    inf = base.clone()
    inf[v - 2] = math.inf
    rows["an infinity"] = inf
    zeros = torch.zeros(v, dtype=dtype)
    zeros[::3] = -0.0
    rows["signed zeros"] = zeros
    rows["ascending"] = torch.arange(v, dtype=torch.float32).div(v / 8).to(dtype)
    rows["descending"] = rows["ascending"].flip(0)
    wide = base.clone()
    wide[0], wide[v - 1] = high, low
    rows["highest and lowest"] = wide
    return rows


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [65, 3001, 20011])
def test_special_rows(dev, dtype, v):
    rows = _special_rows(v, dtype)
    z = torch.stack(list(rows.values()))
    for k in (0, v // 2, -1):
        t = torch.full((z.shape[0],), k)
        r = L.token_logprobs(z.to(dev), t.to(dev), top=20)
        _check(z, t, 20, r, f"{dtype} {v} token {k} {list(rows)}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_rows_in_one_block(dev, dtype):
    """A thousand rows: a block takes a whole row, and no slices are joined."""
    v = 20011
    rows = list(_special_rows(v, dtype).values())
    z = torch.stack(rows + [rows[i % len(rows)] for i in range(1024 - len(rows))])
    t = torch.arange(1024) % v
    r = L.token_logprobs(z.to(dev), t.to(dev), top=64)
    _check(z, t, 64, r, f"{dtype} one block", rows=range(len(rows)))


@pytest.mark.parametrize("top", [1, 5, 64])
def test_the_largest_in_few_threads(dev, top):
    """1,536 of the largest logits at the places of three threads: more than
    the candidates' list holds."""
    v, m = 131072, 1024
    g = torch.Generator().manual_seed(top)
    row = torch.randn(v, generator=g)
    at = (torch.arange(v) // 8) % 256
    for k in (3, 70, 255):
        row[at == k] = 10 + 5 * torch.rand(int((at == k).sum()), generator=g)
    z = torch.empty((m, v), dtype=torch.bfloat16, device=dev)
    z[:] = row.to(torch.bfloat16)
    t = torch.zeros(m, dtype=torch.int64)
    r = L.token_logprobs(z, t.to(dev), top=top)
    host = row.to(torch.bfloat16)[None]
    _check(host, t[:1], top, [x[:1] for x in r], "first row")
    for x in r:
        assert torch.equal(x, x[:1].expand_as(x)), "equal rows give equal results"


@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_alignment(dev, dtype):
    wide = _logits(9, 5003, dtype, 5).to(dev)
    t = torch.arange(9, device=dev)
    for z in (wide[:, 1:5002], wide[:, 3:], wide[1::2, :4001], wide[:1].expand(9, 5003), wide.t().contiguous().t()):
        k = z.shape[0]
        r = L.token_logprobs(z, t[:k], top=5)
        _check(z, t[:k], 5, r, f"{dtype} stride {z.stride()} offset {z.storage_offset()}")
        gl = torch.ones(k, device=dev)
        a = L.token_logprobs_backward(z, t[:k], r.lse, r.entropy, gl)
        b = L.token_logprobs_backward(z.contiguous(), t[:k], r.lse, r.entropy, gl)
        assert torch.equal(a, b)


def test_repeats_are_equal_and_streams(dev):
    z = _logits(17, 50257, torch.bfloat16, 1).to(dev)
    t = torch.arange(17, device=dev)
    want = L.token_logprobs(z, t, top=20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s, s.cuda_stream):
        got = L.token_logprobs(z, t, top=20, stream=stream)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph_replays(dev):
    z = _logits(3, 50257, torch.float32, 2).to(dev)
    t = torch.tensor([4, 5, -1], device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.token_logprobs(z, t, top=7, check=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = L.token_logprobs(z, t, top=7, check=False)
        d = L.token_logprobs_backward(z, t, r.lse, r.entropy, r.entropy, r.lse, check=False)
    for k in range(4):
        z.copy_(_logits(3, 50257, torch.float32, 20 + k))
        graph.replay()
        torch.cuda.synchronize()
        want = L.token_logprobs(z, t, top=7)
        assert all(torch.equal(a, b) for a, b in zip(r, want)), f"replay {k}"
        assert torch.equal(d, L.token_logprobs_backward(z, t, want.lse, want.entropy, want.entropy, want.lse))


def _grad64(z, t, lse, ent, gl, ge):
    """The formula, and the size of its terms for the tolerance."""
    z = z.double()
    lp = z - lse.double()[:, None]
    p = lp.exp()
    v = z.shape[1]
    given = (t >= 0) & (t < v)
    gl = torch.where(given, gl.double(), 0.0)[:, None]
    ge = ge.double()[:, None]
    lpf = torch.where(p > 0, lp, 0.0)
    want = -p * (gl + ge * (lpf + ent.double()[:, None]))
    size = p * (gl.abs() + ge.abs() * (lpf.abs() + ent.double().abs()[:, None])) * (lpf.abs() + 6)
    hot = torch.zeros_like(want).scatter_(1, t.clamp(0, v - 1)[:, None], 1.0) * gl
    return want + hot, size + hot.abs()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,v", [(1, 1), (2, 7), (3, 2049), (5, 8193), (2, 50257)])
def test_gradient_against_the_formula(dev, dtype, m, v):
    z = _logits(m, v, dtype, v)
    if v > 4:
        z[:, 1::3] = -math.inf
    g = torch.Generator().manual_seed(v + m)
    t = torch.randint(0, v, (m,), generator=g) // 3 * 3
    if m > 1:
        t[1] = -1
    gl, ge = torch.randn(m, generator=g), torch.randn(m, generator=g)
    r = L.token_logprobs(z.to(dev), t.to(dev))
    lse, ent = r.lse.cpu(), r.entropy.cpu()
    want, size = _grad64(z, t, lse, ent, gl, ge)
    zd = z.to(dev)
    args = (t.to(dev), r.lse, r.entropy, gl.to(dev), ge.to(dev))
    got = L.token_logprobs_backward(zd, *args)
    assert got.dtype == dtype
    tol = 2 * EPS * size + 1.01 * ROUND[dtype] * want.abs() + torch.finfo(dtype).tiny
    assert bool(((got.double().cpu() - want).abs() <= tol).all())
    # into the logits' own memory, and without either gradient
    assert torch.equal(L.token_logprobs_backward(zd.clone(), *args), got)
    inplace = zd.clone()
    assert L.token_logprobs_backward(inplace, *args, out=inplace) is inplace
    assert torch.equal(inplace, got)
    zero = torch.zeros(m, device=dev)
    for a, b in (((args[3], None), (args[3], zero)), ((None, args[4]), (zero, args[4])), ((None, None), (zero, zero))):
        x = L.token_logprobs_backward(zd, *args[:3], *a)
        assert torch.equal(x, L.token_logprobs_backward(zd, *args[:3], *b))


def test_gradient_against_differences(dev):
    """Central differences of the 64-bit definition along random directions;
    their own error is of the order of the step squared, 1e-8."""
    m, v = 4, 301
    z = _logits(m, v, torch.float32, 9)
    t = torch.tensor([0, 300, 17, -1])
    g = torch.Generator().manual_seed(11)
    gl, ge = torch.randn(m, generator=g), torch.randn(m, generator=g)
    zd = z.to(dev).requires_grad_()
    r = L.token_logprobs(zd, t.to(dev), top=3)
    grad, = torch.autograd.grad((r.logprob * gl.to(dev)).sum() + (r.entropy * ge.to(dev)).sum(), zd)

    def value(x):
        e = [_expect(x[i], int(t[i])) for i in range(m)]
        return sum(float(gl[i]) * e[i][1] + float(ge[i]) * e[i][2] for i in range(m))

    z64 = z.double().numpy()
    for k in range(6):
        d = np.random.default_rng(k).standard_normal((m, v))
        h = 1e-4
        diff = (value(z64 + h * d) - value(z64 - h * d)) / (2 * h)
        dot = float((grad.double().cpu().numpy() * d).sum())
        assert abs(diff - dot) <= 1e-5 * (1 + abs(diff)), (k, diff, dot)


def test_gradient_of_special_rows(dev):
    rows = _special_rows(3001, torch.float32)
    z = torch.stack(list(rows.values())).to(dev)
    t = torch.full((z.shape[0],), 1500, device=dev)
    r = L.token_logprobs(z, t)
    one = torch.ones(z.shape[0], device=dev)
    d = L.token_logprobs_backward(z, t, r.lse, r.entropy, one, one)
    for i, name in enumerate(rows):
        if name == "all -inf":
            assert torch.equal(d[i], torch.zeros_like(d[i])), name
        elif name in ("a NaN", "mostly NaN", "all NaN", "an infinity"):
            assert bool(d[i].isnan().any()), name
        else:
            assert bool(d[i].isfinite().all()), name
            assert abs(float(d[i].double().sum())) < 1e-4, name  # a softmax's gradient sums to zero


def test_no_rows(dev):
    z = torch.empty((0, 100), device=dev)
    t = torch.empty(0, dtype=torch.int64, device=dev)
    r = L.token_logprobs(z, t, top=3)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 3)
    assert L.token_logprobs_backward(z, t, r.lse, r.entropy, r.logprob).shape == (0, 100)


def test_refusals(dev):
    z = torch.zeros((2, 10), device=dev)
    t = torch.zeros(2, dtype=torch.int64, device=dev)
    r = L.token_logprobs(z, t)
    for bad in (lambda: L.token_logprobs(z.cpu(), t), lambda: L.token_logprobs(z, t.cpu()),
                lambda: L.token_logprobs(z, t.int()), lambda: L.token_logprobs(z, t[:1]),
                lambda: L.token_logprobs(z, t, top=11), lambda: L.token_logprobs(z, t, top=-1),
                lambda: L.token_logprobs(z[:, :0], t), lambda: L.token_logprobs(z.new_zeros((2, 100)), t, top=65),
                lambda: L.token_logprobs_backward(z, t, r.lse, None, r.logprob, r.entropy),
                lambda: L.token_logprobs_backward(z, t, None, r.entropy, r.logprob),
                lambda: L.token_logprobs_backward(z, t, r.lse[:1], r.entropy, r.logprob),
                lambda: L.token_logprobs_backward(z, t, r.lse, r.entropy, r.logprob.double()),
                lambda: L.token_logprobs_backward(z, t, r.lse, r.entropy, r.logprob, out=z.half()),
                lambda: L.token_logprobs_backward(z, t, r.lse, r.entropy, r.logprob, out=z[:1].expand(2, 10)),
                lambda: L.token_logprobs(z.clone().requires_grad_(), t, stream=torch.cuda.Stream())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: L.token_logprobs(z.double(), t), lambda: L.token_logprobs(z[0], t)):
        with pytest.raises(TypeError):
            bad()
    t[1] = 10
    with pytest.raises(B.WcError, match="index out of range"):
        L.token_logprobs(z, t)
    with pytest.raises(B.WcError, match="index out of range"):
        L.token_logprobs_backward(z, t, r.lse, r.entropy, r.logprob)
    got = L.token_logprobs(z, t, check=False)
    assert float(got.logprob[0]) == pytest.approx(-math.log(10), rel=1e-6) and math.isnan(float(got.logprob[1]))
    d = L.token_logprobs_backward(z, t, r.lse, r.entropy, torch.ones(2, device=dev), check=False)
    assert torch.equal(d[1], torch.zeros(10, device=dev))

"""Rows of logits of any size.

The kernel subtracts a row's maximum m first, so the statistics do not know
its size.  A term 2^d, d = (z - m) log2 e, has relative error 2^-24 (2 |d| + 3),
|d| weighted by the terms' size stays below 30, and a thread sums V / 256 of
them: ln S and ln 2 W / S are off by at most 2^-24 (V / 256 + 64) (1 + H), so
is the entropy (by the sum of both).  lse = m + ln S is rounded to fp32 once
more, and so is a log probability.
"""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import logprobs as L  # noqa: E402
from test_gpu_logprobs import ROUND, _check, _expect, _grad64, _order, _special_rows  # noqa: E402

EPS = 2.0 ** -24
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


def _strict(z, t, top, r, what):
    zs = z.double().numpy()
    r = [v.cpu().numpy().astype(np.float64) if v is not None and v.dtype == F32 else None if v is None else v.cpu().numpy()
         for v in r]
    for i in range(zs.shape[0]):
        lse, lp, ent = _expect(zs[i], int(t[i]))
        tol = EPS * (zs.shape[1] / 256 + 64)
        at = f"{what} row {i}"
        assert abs(r[2][i] - lse) <= tol + 2 * EPS * abs(lse), f"{at}: lse {r[2][i]} want {lse}"
        assert abs(r[0][i] - lp) <= tol + 2 * EPS * abs(lse) + EPS * abs(lp), f"{at}: logprob {r[0][i]} want {lp}"
        assert abs(r[1][i] - ent) <= 2 * tol * (1 + ent), f"{at}: entropy {r[1][i]} want {ent}"
        assert r[0][i] <= 0, f"{at}: a probability above one"
        if top:
            assert np.array_equal(r[4][i], _order(zs[i], top)), at
            assert (r[3][i] <= 0).all(), at


def _fills(dtype):
    sizes = [6e4, -6e4, -1e4] if dtype == HF else [-1e10, 1e10, -1e11, 1e12, -1e15, 1e15, -1e20, 1e20, 1e30, -1e30, -1e33]
    return [float(torch.tensor(f, dtype=dtype)) for f in sizes]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("v,top", [(3, 3), (3001, 0), (50257, 20), (150001, 5)])
def test_rows_of_one_large_number(dev, dtype, v, top):
    """A mask of a large finite number in a whole row: every token is as likely."""
    fills = _fills(dtype)
    _say(f"[logprobs range] {dtype} {v}: rows of {fills}")
    z = torch.tensor(fills)[:, None].expand(-1, v).to(dtype).contiguous()
    t = torch.arange(len(fills)) % v
    zd, td = z.to(dev), t.to(dev)
    r = L.token_logprobs(zd, td, top=top)
    for i, f in enumerate(fills):
        lse = abs(float(r.lse[i]) - f - math.log(v))
        assert lse <= EPS * (v / 256 + 64) + 2 * EPS * abs(f), f
        assert abs(float(r.entropy[i]) - math.log(v)) <= 2 * EPS * (v / 256 + 64) * (1 + math.log(v)), f
        assert float(r.logprob[i]) <= 0 and math.isfinite(float(r.logprob[i])), f
    if top:
        assert torch.equal(r.top_ids.cpu(), torch.arange(top).expand(len(fills), top))
    # the gradient of logprob: [j = t] - 1 / v, and of the entropy: zero
    one = torch.ones(len(fills), device=dev)
    d = L.token_logprobs_backward(zd, td, r.lse, r.entropy, one).double().cpu()
    want = torch.full((len(fills), v), -1.0 / v, dtype=torch.float64)
    want[torch.arange(len(fills)), t] += 1
    for i, f in enumerate(fills):
        if abs(float(r.lse[i])) >= 65536:  # below, p comes from lse in fp32 as it was given
            # the bound of test_gpu_logprobs.py: p is off by 2^-24 (|log p| + 4) of itself, twice, and one rounding
            tol = 2 * EPS * (want[i].abs() + 1.0 / v) * (math.log(v) + 6) + 1.01 * ROUND[dtype] * want[i].abs()
            assert bool(((d[i] - want[i]).abs() <= tol).all()), f


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("v,top", [(4096, 5), (50257, 0), (140001, 20)])
def test_rows_far_from_zero(dev, dtype, v, top):
    g = torch.Generator().manual_seed(v)
    rows = []
    for f in (0.0, 1e3, -1e4, 5e4) if dtype == HF else (0.0, 1e3, -1e3, 1e4, -5e4, 1e6, -1e6, 3e7):
        base = torch.randn(v, generator=g, dtype=torch.float64) * 2
        rows.append((base + f).to(dtype))
        half = (base + f).to(dtype)
        half[::2] = -math.inf
        rows.append(half)
        if dtype != HF:  # masked by a finite number, or nothing but one token
            half = (base + f).to(dtype)
            half[1::2] = -1e10
            rows.append(half)
            one = torch.full((v,), -1e20, dtype=dtype)
            one[v // 3] = f
            rows.append(one)
    z = torch.stack(rows)
    t = z.argmax(1)
    _say(f"[logprobs range] {dtype} {z.shape[0]} rows of {v}")
    _strict(z, t, top, L.token_logprobs(z.to(dev), t.to(dev), top=top), f"{dtype} {v}")


def test_one_likely_token_of_any_size(dev):
    """All probability at one token: lse is its logit, not the number beside it."""
    m, v = 600, 1000
    z = torch.full((m, v), -1e4)
    t = torch.arange(m) % v
    z[torch.arange(m), t] = torch.linspace(0.5, 40.0, m)
    r = L.token_logprobs(z.to(dev), t.to(dev))
    assert torch.equal(r.lse.cpu(), z[torch.arange(m), t])
    assert bool((r.logprob == 0).all()) and bool((r.entropy == 0).all())


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_special_rows_of_joined_parts(dev, dtype):
    """Vocabularies past 131072 take two blocks a row and a join."""
    v = 131072 + 4099
    z = torch.stack(list(_special_rows(v, dtype).values()))
    for k in (0, v // 2, -1):
        t = torch.full((z.shape[0],), k)
        _say(f"[logprobs range] special rows {dtype} {v} token {k}")
        _check(z, t, 20, L.token_logprobs(z.to(dev), t.to(dev), top=20), f"{dtype} {v} token {k}")


@pytest.mark.parametrize("size", [1.0, 1e9, -1e20, 1e30])
def test_large_gradient_of_the_entropy_at_masked_logits(dev, size):
    """A scaled loss: a masked logit has p = 0 and a gradient of 0, whatever the gradient of the entropy."""
    m, v = 3, 3001
    z = torch.randn((m, v), generator=torch.Generator().manual_seed(5)) * 3
    z[:, ::2] = -math.inf
    z[1, 1::4] = -1e10
    z[2, 1::4] = -300.0
    t = torch.tensor([1, 3, 5])
    r = L.token_logprobs(z.to(dev), t.to(dev))
    ge = torch.tensor([size, -0.5 * size, 0.25 * size])
    want, bound = _grad64(z, t, r.lse.cpu(), r.entropy.cpu(), torch.ones(m), ge)
    got = L.token_logprobs_backward(z.to(dev), t.to(dev), r.lse, r.entropy, torch.ones(m, device=dev), ge.to(dev))
    got = got.double().cpu()
    assert bool((got[:, ::2] == 0).all())
    tol = 2 * EPS * bound + 1.01 * ROUND[F32] * want.abs() + torch.finfo(F32).tiny * max(1.0, abs(size))
    assert bool(((got - want).abs() <= tol).all())

"""The mixture-of-experts layer against its definition in 64 bits.

Tolerance.  A product of n exact terms summed in fp32 is off by at most
(n + 24) 2^-24 times the sum of their sizes.  That holds for the logits (an
error dl of a logit is a relative error of 2 dl of a weight), for gate and up
(silu has a slope below 1.1), and for the second product.  silu's exponential
adds 2^-24 (2 |gate| + 8) of h, and h's two terms leave out 2^-16 of it (BF16)
or 2^-21 and an absolute 2^-28 (FP16).  Then one rounding to the type.
"""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import codec, moe as M  # noqa: E402

EPS = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16
ROUND = {HF: 2.0 ** -11, BF: 2.0 ** -8}
SPLIT = {HF: (2.0 ** -21, 2.0 ** -28), BF: (2.0 ** -16, 0.0)}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _inputs(m, e, h, i, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(dtype)
    return (n(m, h), n(e, h, std=1.5 / h ** 0.5), n(e, i, h, std=h ** -0.5), n(e, i, h, std=h ** -0.5),
            n(e, h, i, std=i ** -0.5))


def _expect(x, router, w1, w3, w2, k, renorm):
    dtype, h, i = x.dtype, x.shape[1], w1.shape[1]
    want, tol = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    for t in range(x.shape[0]):
        v = x[t].double()
        logits = router.double() @ v
        dl = (h + 24) * EPS * float((router.double().abs() @ v.abs()).max())
        best = torch.sort(logits, descending=True, stable=True)
        ids = best.indices[:k]
        if k < logits.numel():
            gap = float(best.values[k - 1] - best.values[k])
            # the choice is sure: either exact logits (whole numbers) or further apart than their error
            assert gap > 2 * dl or bool((logits == logits.round()).all()), f"token {t}: choose another seed"
        p = torch.softmax(logits, 0)[ids]
        p = p / p.sum() if renorm else p
        for w, e in zip(p, ids):
            a, b = w1[e].double(), w3[e].double()
            gate, up = a @ v, b @ v
            dg, du = (h + 24) * EPS * (a.abs() @ v.abs()), (h + 24) * EPS * (b.abs() @ v.abs())
            s = gate / (1 + (-gate).exp())
            hid = s * up
            dh = 1.1 * dg * (up.abs() + du) + (s.abs() + 1.1 * dg) * du
            dh += hid.abs() * (EPS * (2 * gate.abs() + 8) + SPLIT[dtype][0]) + SPLIT[dtype][1]
            c = w2[e].double()
            want[t] += w * (c @ hid)
            tol[t] += w * (c.abs() @ dh + ((2 * i + 24) * EPS + 2 * dl + 16 * EPS) * (c.abs() @ hid.abs()))
    return want, tol + ROUND[dtype] * want.abs() * 1.01 + torch.finfo(dtype).tiny


def _check(args, k, renorm, dev, what):
    _say(f"[moe] {what}")
    want, tol = _expect(*args, k, renorm)
    y = M.moe_layer(*[a.to(dev) for a in args], k, renormalize=renorm)
    assert y.dtype == args[0].dtype and y.shape == args[0].shape
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err / tol).max())} of its tolerance"


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,e,k,h,i", [(1, 1, 1, 8, 8), (1, 8, 2, 64, 40), (3, 5, 5, 72, 24), (16, 64, 8, 256, 128),
                                       (17, 64, 8, 264, 136), (33, 16, 4, 520, 104), (64, 256, 8, 128, 64),
                                       (64, 8, 2, 1032, 264), (5, 300, 16, 64, 32), (2, 1024, 3, 40, 16),
                                       (13, 8, 2, 4096, 1032), (50, 4, 1, 96, 48), (64, 4, 4, 64, 72),
                                       (1, 40, 8, 2056, 520), (31, 2, 1, 5000, 16)])
def test_against_64_bits(dev, dtype, m, e, k, h, i):
    args = _inputs(m, e, h, i, dtype, m + e + h + i)
    for renorm in (True, False):
        _check(args, k, renorm, dev, f"{dtype} {m} tokens, {k} of {e} experts, {h} x {i}, renormalize={renorm}")


@pytest.mark.parametrize("m,e,k", [(4, 8, 3), (40, 70, 5)])
def test_equal_logits_go_to_the_lower_number(dev, m, e, k):
    x, r, w1, w3, w2 = _inputs(m, e, 64, 32, BF, 3)
    g = torch.Generator().manual_seed(8)
    x = torch.randint(-2, 3, x.shape, generator=g).to(BF)
    r = torch.randint(-1, 2, r.shape, generator=g).to(BF)
    r[e // 2:] = r[:e - e // 2]  # pairs of equal experts
    _check((x, r, w1, w3, w2), k, True, dev, "pairs of equal logits")
    _check((x, torch.zeros_like(r), w1, w3, w2), k, False, dev, "all logits equal")
    _check((x, r[:1].expand_as(r).contiguous() * 0 - 1, w1, w3, w2), k, True, dev, "all logits equal, not zero")


def test_every_token_to_the_same_experts(dev):
    x, r, w1, w3, w2 = _inputs(64, 16, 128, 48, BF, 5)
    r = r.double()
    x = x + 1
    r[3] += 1.0
    r[11] += 0.5
    _check((x.to(BF), r.to(BF), w1, w3, w2), 2, True, dev, "64 tokens on two experts")


@pytest.mark.parametrize("m", [5, 40])
def test_nan_stays_with_its_token(dev, m):
    for dtype in (BF, HF):
        args = _inputs(m, 12, 64, 40, dtype, 6)
        want, tol = _expect(*args, 3, True)
        x = args[0].clone()
        x[1, 3] = float("nan")
        x[3, 5] = float("inf")
        y = M.moe_layer(x.to(dev), *[a.to(dev) for a in args[1:]], 3).double().cpu()
        ok = torch.ones(m, dtype=torch.bool)
        ok[[1, 3]] = False
        assert bool(((y - want).abs() <= tol)[ok].all())
        assert bool(y[1].isnan().all()) and not bool(y[3].isfinite().any())
    # an expert of NaN that no token goes to changes nothing
    x, r, w1, w3, w2 = _inputs(5, 12, 64, 40, BF, 6)
    used = {int(e) for row in x.double() @ r.double().T for e in row.topk(3).indices}
    idle = next(e for e in range(12) if e not in used)
    w1[idle] = w3[idle] = w2[idle] = float("nan")
    _check((x, r, w1, w3, w2), 3, True, dev, "an idle expert of NaN")


def test_large_and_small_h_in_half_precision(dev):
    for f in (30.0, 2.0 ** -4):
        x, r, w1, w3, w2 = _inputs(9, 6, 128, 64, HF, 7)
        _check((x, r, (w1 * f).to(HF), (w3 * f * f).to(HF), (w2 / f ** 3 if f > 1 else w2).to(HF)), 2, True, dev,
               f"weights times {f}")


def test_strides_and_out(dev):
    m, e, h, i = 6, 5, 64, 40
    x, r, w1, w3, w2 = [t.to(dev) for t in _inputs(m, e, h, i, BF, 9)]
    want = M.moe_layer(x, r, w1, w3, w2, 2)
    stacked = torch.cat([w1, w3], 1)
    wide = torch.zeros((e, h + 8, i + 16), dtype=BF, device=dev)
    wide[:, :h, :i] = w2
    xs = torch.zeros((m, h + 9), dtype=BF, device=dev)
    xs[:, 1:h + 1] = x
    rs = torch.zeros((e, h + 4), dtype=BF, device=dev)
    rs[:, :h] = r
    out = torch.full((m, h + 3), 7.0, dtype=BF, device=dev)
    y = M.moe_layer(xs[:, 1:h + 1], rs[:, :h], stacked[:, :i], stacked[:, i:], wide[:, :h, :i], 2, out=out[:, 1:h + 1])
    assert torch.equal(y, want) and torch.equal(out[:, 1:h + 1], want)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, h + 1:] == 7).all())


def test_repeats_streams_and_graph(dev):
    for m in (1, 50):
        args = [t.to(dev) for t in _inputs(m, 32, 512, 264, BF, 10)]
        want = M.moe_layer(*args, 4)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        for stream in (None, st, st.cuda_stream):
            y = M.moe_layer(*args, 4, stream=stream)
            torch.cuda.synchronize()  # y was written on another stream than the comparison's
            same = bool(torch.equal(y, want))
            assert same, f"{m} tokens on {stream}"
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = M.moe_layer(*args, 4)
        for k in range(4):
            args[0].copy_(torch.randn(args[0].shape, generator=torch.Generator().manual_seed(k)))
            graph.replay()
            torch.cuda.synchronize()
            same = bool(torch.equal(y, M.moe_layer(*args, 4)))
            assert same, f"replay {k}"


def test_experts_from_a_compressed_set(dev):
    x, r, w1, w3, w2 = [t.to(dev) for t in _inputs(7, 6, 128, 64, BF, 11)]
    want = M.moe_layer(x, r, w1, w3, w2, 2)
    e = codec.encode_batch(list(w1) + list(w3) + list(w2))
    d1, d3, d2 = torch.empty_like(w1), torch.empty_like(w3), torch.empty_like(w2)
    codec.decode_batch(e, outs=list(d1) + list(d3) + list(d2))
    assert torch.equal(M.moe_layer(x, r, d1, d3, d2, 2), want)


def test_offsets_past_32_bits(dev):
    """Experts that lie more than 2^32 bytes behind the first."""
    e, i, h = 3, 64, 1 << 14
    x, r, _, _, _ = _inputs(2, e, h, 8, BF, 12)
    r = torch.zeros_like(r)
    r[2] = x[0].sign()
    r[1] = x[1].sign()
    flat = torch.zeros((1 << 31) + (1 << 26), dtype=BF, device=dev)
    stride = (1 << 30) + 64
    g = torch.Generator().manual_seed(1)
    parts = [(torch.randn((e, i, h), generator=g) / h ** 0.5).to(BF), (torch.randn((e, i, h), generator=g) / h ** 0.5).to(BF),
             (torch.randn((e, h, i), generator=g) / i ** 0.5).to(BF)]
    views, at = [], 0
    for p in parts:
        v = flat[at:].as_strided((e, *p.shape[1:]), (stride, p.shape[2], 1))
        v.copy_(p)
        views.append(v)
        at += p[0].numel() + 64
    assert views[2][2].data_ptr() - flat.data_ptr() > 1 << 32
    want, tol = _expect(x, r, *parts, 1, True)
    y = M.moe_layer(x.to(dev), r.to(dev), *views, 1)
    assert bool(((y.double().cpu() - want).abs() <= tol).all())


def test_no_tokens(dev):
    x, r, w1, w3, w2 = [t.to(dev) for t in _inputs(1, 3, 16, 8, BF, 1)]
    assert M.moe_layer(x[:0], r, w1, w3, w2, 2).shape == (0, 16)


def test_refusals(dev):
    x, r, w1, w3, w2 = [t.to(dev) for t in _inputs(4, 3, 16, 8, BF, 1)]
    big = x.new_zeros((65, 16))
    for args, k in (((x.cpu(), r, w1, w3, w2), 2), ((x, r.cpu(), w1, w3, w2), 2), ((x, r, w1.cpu(), w3, w2), 2),
                    ((x, r, w1, w3, w2), 0), ((x, r, w1, w3, w2), 4), ((big, r, w1, w3, w2), 2),
                    ((x, r[:2], w1, w3, w2), 2), ((x, r, w1, w3[:, :, :8], w2), 2), ((x, r, w1, w3, w1), 2),
                    ((x, r, w1, w3, w2.transpose(1, 2).contiguous().transpose(1, 2)), 2), ((x[0], r, w1, w3, w2), 2),
                    ((x[:, :12], r[:, :12], w1[:, :, :12], w3[:, :, :12], w2[:, :12]), 2),
                    ((x, r, w1, torch.cat([w3, w3], 1)[:, :8], w2), 2)):
        with pytest.raises(ValueError):
            M.moe_layer(*args, k)
    for args in ((x.float(), r, w1, w3, w2), (x, r.half(), w1, w3, w2), (x, r, w1.half(), w3, w2)):
        with pytest.raises(TypeError):
            M.moe_layer(*args, 2)
    with pytest.raises(ValueError):
        M.moe_layer(x, r, w1, w3, w2, 2, out=x.new_zeros((4, 15)))

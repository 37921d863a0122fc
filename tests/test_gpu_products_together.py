"""The products of a training step and of serving as they are used together:
experts and the loss of a large vocabulary with all their gradients, weights
of 4 bits with adapters beside them, in graphs, on given streams, and call by
call through the binding."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import _binding as B  # noqa: E402
from lossless_weight_compression_bf16_amd.adapters import add_adapters  # noqa: E402
from lossless_weight_compression_bf16_amd.fourbit import Weights4, linear4, quantize4  # noqa: E402
from lossless_weight_compression_bf16_amd.grouped import grouped_linear, grouped_linear_backward  # noqa: E402
from lossless_weight_compression_bf16_amd.loss import linear_cross_entropy, linear_cross_entropy_backward  # noqa: E402

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


def _normal(seed, dev, dtype, *shape, scale=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device=dev)).to(dtype)


def _model(dev, dtype, m, cols, inner, vocab, experts, seed=3):
    """A layer of experts with a residual, and a vocabulary: x sorted by expert."""
    cuts = torch.tensor(sorted(((seed * 7919 * (i + 1)) % (m + 1)) for i in range(experts - 1)) + [m], device=dev)
    leaves = [_normal(1, dev, dtype, m, cols), _normal(2, dev, dtype, experts, inner, cols, scale=cols ** -0.5),
              _normal(3, dev, dtype, experts, cols, inner, scale=inner ** -0.5), _normal(4, dev, dtype, vocab, cols, scale=cols ** -0.5)]
    tokens = (torch.arange(m, device=dev) * 31) % vocab
    tokens[::7] = -1
    return leaves, cuts, tokens


def _step(leaves, ends, tokens):
    x, w1, w2, vocab = leaves
    h = grouped_linear(x, w1, ends, check=False)
    y = x + grouped_linear(h * torch.sigmoid(h), w2, ends, check=False)
    r = linear_cross_entropy(y, vocab, tokens, check=False)
    return r.loss.mean() + 1e-3 * (r.lse * r.lse).mean()


def _step64(leaves, ends, tokens):
    x, w1, w2, vocab = leaves
    lo, parts = 0, []
    for e, hi in enumerate(ends.tolist()):
        h = x[lo:hi] @ w1[e].T
        parts.append(x[lo:hi] + (h * torch.sigmoid(h)) @ w2[e].T)
        lo = hi
    z = torch.cat(parts) @ vocab.T
    lse = torch.logsumexp(z, 1)
    loss = torch.where(tokens >= 0, lse - z.gather(1, tokens.clamp(min=0)[:, None])[:, 0], 0)
    return loss.mean() + 1e-3 * (lse * lse).mean()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,cols,inner,vocab,experts", [(5, 64, 40, 300, 4), (200, 256, 136, 1000, 3), (700, 512, 264, 5000, 8)])
def test_a_training_step_against_64_bits(dev, dtype, m, cols, inner, vocab, experts):
    """From the leaves to a gradient there are at most 16 roundings (two products, a sigmoid, a product and a sum of
    16-bit tensors forward, the gradient of the logits, and the gradients of each of these backward).  Each moves
    its tensor by at most eps / 2 of its size in the root mean square, and random terms neither grow nor cancel on the
    way by more than a factor of 2: 16 eps."""
    _say(f"[step] {dtype} {m} rows, {experts} experts of {inner} x {cols}, {vocab} tokens")
    leaves, ends, tokens = _model(dev, dtype, m, cols, inner, vocab, experts)
    ours = [t.clone().requires_grad_() for t in leaves]
    loss = _step(ours, ends, tokens)
    loss.backward()
    exact = [t.double().requires_grad_() for t in leaves]
    want = _step64(exact, ends, tokens)
    want.backward()
    eps = torch.finfo(dtype).eps
    assert abs(float(loss.detach()) - float(want.detach())) <= 16 * eps * abs(float(want.detach()))
    for a, b, what in zip(ours, exact, ("x", "w1", "w2", "vocabulary")):
        assert a.grad.dtype == dtype
        off = float((a.grad.double() - b.grad).norm() / b.grad.norm())
        assert off <= 16 * eps, f"{what}: {off / eps} eps"


def test_weights_of_4_bits_with_adapters(dev):
    """linear4 rounds once, and the adapters' sum is rounded once more and their terms once (a product of A)."""
    m, cols, rows, n, rank = 21, 512, 300, 3, 16
    x, w = _normal(1, dev, BF, m, cols), _normal(2, dev, BF, rows, cols, scale=cols ** -0.5)
    a, b = _normal(3, dev, BF, n, rank, cols, scale=cols ** -0.5), _normal(4, dev, BF, n, rows, rank, scale=rank ** -0.5)
    ids = torch.arange(m, device=dev) % (n + 1) - 1
    q = quantize4(w, group=64, zeros=True)
    y = linear4(x, q)
    base = y.clone()
    got = add_adapters(x, y, a, b, ids)
    assert got.data_ptr() == y.data_ptr()
    values = torch.stack([q.q & 15, q.q >> 4], 2).view(rows, -1, 64).double()
    dense = (q.scales.double()[..., None] * (values - q.zeros.double()[..., None])).view(rows, cols)
    plain = x.double() @ dense.T
    eps = torch.finfo(BF).eps
    size = x.double().abs() @ dense.abs().T
    assert bool(((base.double() - plain).abs() <= eps / 2 * 1.01 * plain.abs() + 2e-4 * size).all())
    none = ids < 0
    assert torch.equal(got[none], base[none])
    for e in range(n):
        r = ids == e
        u = x[r].double() @ a[e].double().T
        want = plain[r] + u @ b[e].double().T
        terms = u.abs() @ b[e].double().abs().T
        tol = 1.01 * (eps / 2 * (plain[r].abs() + want.abs() + terms)) + 1e-3 * (size[r] * 0.2 + terms)
        assert bool(((got[r].double() - want).abs() <= tol).all())


def _serving(x, w1, ends, q, vocab, tokens):
    h = grouped_linear(x, w1, ends, check=False)
    y = linear4(h, q)
    r = linear_cross_entropy(y, vocab, tokens, check=False)
    return h, y, r.loss, r.lse


@pytest.mark.parametrize("m", [1, 30, 300])
def test_two_graphs_that_share_a_pool(dev, m):
    """Their workspaces are the same memory: replayed in turn, with eager work and new inputs between."""
    cols, inner, vocab, experts = 256, 512, 3000, 4
    w1, q = _normal(1, dev, BF, experts, inner, cols, scale=cols ** -0.5), quantize4(_normal(2, dev, BF, cols, inner), group=128)
    v = _normal(3, dev, BF, vocab, cols, scale=cols ** -0.5)
    tokens = torch.arange(m, device=dev)
    ends = torch.tensor([m // 3, m // 3, m - 1, m], device=dev).clamp(min=0)
    xs = [_normal(4 + i, dev, BF, m, cols) for i in range(2)]
    with torch.no_grad():
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for x in xs:
                _serving(x, w1, ends, q, v, tokens)
        torch.cuda.synchronize()
        graphs, outs, pool = [], [], None
        for x in xs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, pool=pool):
                outs.append(_serving(x, w1, ends, q, v, tokens))
            pool = pool or g.pool()
            graphs.append(g)
        for turn in range(4):
            for i in (0, 1, 1, 0):
                _say(f"[graphs] {m} rows, turn {turn}, graph {i}")
                xs[i].copy_(_normal(100 * turn + i, dev, BF, m, cols))
                want = _serving(xs[i], w1, ends, q, v, tokens)
                torch.cuda.synchronize()
                graphs[i].replay()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(outs[i], want))


@pytest.mark.parametrize("m", [3, 90, 700])
def test_captured_gradient_calls(dev, m):
    cols, rows, vocab, experts = 256, 384, 2000, 5
    x, w = _normal(1, dev, HF, m, cols), _normal(2, dev, HF, experts, rows, cols, scale=cols ** -0.5)
    d, v = _normal(3, dev, HF, m, rows), _normal(4, dev, HF, vocab, cols, scale=cols ** -0.5)
    ends = torch.tensor([0, m // 2, m // 2, m - 1, m - 1], device=dev)
    tokens = torch.arange(m, device=dev) - 1
    one = torch.rand(m, device=dev)

    def go():
        lse = linear_cross_entropy(x, v, tokens, check=False).lse
        return (*grouped_linear_backward(x, w, ends, d, check=False),
                *linear_cross_entropy_backward(x, v, tokens, lse, one, one, check=False))
    with torch.cuda.stream(torch.cuda.Stream()):
        go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    for turn in range(4):
        _say(f"[graphs] gradients of {m} rows, turn {turn}")
        x.copy_(_normal(50 + turn, dev, HF, m, cols))
        d.copy_(_normal(60 + turn, dev, HF, m, rows))
        want = go()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_captured_training_step(dev):
    """Captured with nothing of autograd's from before alive."""
    leaves, ends, tokens = _model(dev, BF, 60, 128, 72, 500, 3)
    leaves = [t.requires_grad_() for t in leaves]
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.autograd.grad(_step(leaves, ends, tokens), leaves)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = _step(leaves, ends, tokens)
        grads = torch.autograd.grad(loss, leaves)
    for turn in range(4):
        _say(f"[graphs] training step, turn {turn}")
        with torch.no_grad():
            leaves[0].copy_(_normal(70 + turn, dev, BF, 60, 128))
        plain = [t.detach().clone().requires_grad_() for t in leaves]
        want = _step(plain, ends, tokens)
        found = torch.autograd.grad(want, plain)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want) and all(torch.equal(a, b) for a, b in zip(grads, found))


def test_a_capture_beside_another_graph_of_the_leaves_is_refused(dev):
    m, cols = 8, 64
    x, w = _normal(1, dev, BF, m, cols), _normal(2, dev, BF, 2, 32, cols).requires_grad_()
    v, ends = _normal(3, dev, BF, 100, cols).requires_grad_(), torch.tensor([4, 8], device=dev)
    tokens = torch.arange(m, device=dev)
    calls = (lambda: grouped_linear(x, w, ends, check=False), lambda: linear_cross_entropy(x, v, tokens, check=False).loss)
    for call, leaf in zip(calls, (w, v)):
        for held in (call(), leaf * 1):  # ours, and another's
            _say("[graphs] a leaf of another graph")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                y = x + 1  # noqa: F841
                with pytest.raises(RuntimeError, match="another graph of one of its leaves"):
                    call()
            torch.cuda.synchronize()
            del held, g, y
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):  # and two calls of one capture are fine
            y, z = call(), call()
        g.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            want = call()
        assert torch.equal(y.detach(), want) and torch.equal(z.detach(), want)
        del y, z, g


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


@pytest.mark.parametrize("m", [2, 40, 500])
def test_given_streams(dev, busy, m):
    cols, rows, vocab, experts = 512, 264, 3001, 3
    x, w = _normal(1, dev, BF, m, cols), _normal(2, dev, BF, experts, rows, cols, scale=cols ** -0.5)
    d, v = _normal(3, dev, BF, m, rows), _normal(4, dev, BF, vocab, cols, scale=cols ** -0.5)
    ends, tokens = torch.tensor([m // 2, m // 2, m], device=dev), torch.arange(m, device=dev)
    one = torch.rand(1, device=dev)
    q = quantize4(w[0], group=32, zeros=True)
    xa, da, ea, ta, oa = _apart(x), _apart(d), _apart(ends), _apart(tokens), one.expand(m)
    y = grouped_linear(x, w, ends)
    _on_stream(lambda s: [grouped_linear(xa, w, ea, check=False, stream=s)], [y], busy, "grouped_linear")
    _on_stream(lambda s: [grouped_linear(xa, w, ea, stream=s)], [y], busy, "grouped_linear, checked")
    want = grouped_linear_backward(x, w, ends, d)
    _on_stream(lambda s: grouped_linear_backward(xa, w, ea, da, check=False, stream=s), want, busy, "grouped_linear_backward")
    r = linear_cross_entropy(x, v, tokens)
    _on_stream(lambda s: linear_cross_entropy(xa, v, ta, check=False, stream=s), r, busy, "linear_cross_entropy")
    want = linear_cross_entropy_backward(x, v, tokens, r.lse, oa.contiguous(), oa.contiguous())
    la = _apart(r.lse)
    _on_stream(lambda s: linear_cross_entropy_backward(xa, v, ta, la, oa, oa, check=False, stream=s), want, busy,
               "linear_cross_entropy_backward")
    _on_stream(lambda s: [linear4(xa, q, stream=s)], [linear4(x, q)], busy, "linear4")
    wa = _apart(w[0])
    _on_stream(lambda s: quantize4(wa, 32, True, stream=s)[:3], q[:3], busy, "quantize4")


def test_through_the_binding(dev):
    m, cols, rows, vocab, experts = 300, 256, 136, 700, 4
    x, w = _normal(1, dev, HF, m, cols), _normal(2, dev, HF, experts, rows, cols, scale=cols ** -0.5)
    d, v = _normal(3, dev, HF, m, rows), _normal(4, dev, HF, vocab, cols, scale=cols ** -0.5)
    ends, tokens = torch.tensor([10, 10, 200, m], device=dev), torch.arange(m, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)

    def scratch(n):
        return torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    y = torch.empty((m, rows), dtype=HF, device=dev)
    n = B.wc_grouped_linear_scratch(m, experts, rows, cols)
    B.wc_grouped_linear(B.wc_grouped(x.data_ptr(), cols, w.data_ptr(), rows * cols, cols, ends.data_ptr(), y.data_ptr(), rows, m,
                                     experts, rows, cols, B.WC_T_FP16, 1), scratch(n), n, err)
    assert int(err.item()) == 0 and torch.equal(y, grouped_linear(x, w, ends))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    n = B.wc_grouped_linear_backward_scratch(m, experts, rows, cols)
    B.wc_grouped_linear_backward(B.wc_grouped_grad(x.data_ptr(), cols, w.data_ptr(), rows * cols, cols, ends.data_ptr(),
                                                   d.data_ptr(), rows, dx.data_ptr(), cols, dw.data_ptr(), m, experts, rows, cols,
                                                   B.WC_T_FP16, 1), scratch(n), n, err)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw), grouped_linear_backward(x, w, ends, d)))
    loss, lse = (torch.empty(m, device=dev) for _ in range(2))
    tokens[5] = vocab
    n = B.wc_linear_cross_entropy_scratch(m, vocab, cols)
    B.wc_linear_cross_entropy(B.wc_linear_loss(x.data_ptr(), cols, v.data_ptr(), cols, tokens.data_ptr(), m, vocab, cols,
                                               B.WC_T_FP16, 0, loss.data_ptr(), lse.data_ptr()), scratch(n), n, err)
    assert int(err.item()) == B.EF_BAD_INDEX and bool(loss[5].isnan())
    want = linear_cross_entropy(x, v, tokens, check=False)
    assert torch.equal(lse, want.lse) and torch.equal(loss.nan_to_num(7), want.loss.nan_to_num(7))
    dh, dv, one = torch.empty_like(x), torch.empty_like(v), torch.ones(m, device=dev)
    n = B.wc_linear_cross_entropy_backward_scratch(m, vocab, cols)
    B.wc_linear_cross_entropy_backward(B.wc_linear_loss_grad(x.data_ptr(), cols, v.data_ptr(), cols, tokens.data_ptr(),
                                                             lse.data_ptr(), one.data_ptr(), 0, dh.data_ptr(), cols, dv.data_ptr(),
                                                             m, vocab, cols, B.WC_T_FP16), scratch(n), n, err)
    assert all(torch.equal(a, b) for a, b in zip((dh, dv), linear_cross_entropy_backward(x, v, tokens, lse, one, check=False)))
    q, s, z = (torch.empty(rows, k, dtype=t, device=dev) for k, t in ((cols // 2, torch.uint8), (cols // 64, HF), (cols // 64, HF)))
    B.wc_quantize4(w, cols, rows, cols, 64, B.WC_T_FP16, q, s, z)
    want4 = quantize4(w[0], zeros=True)
    assert all(torch.equal(a, b) for a, b in zip((q, s, z), want4[:3]))
    B.wc_linear4(B.wc_fourbit(x.data_ptr(), cols, q.data_ptr(), s.data_ptr(), z.data_ptr(), y.data_ptr(), rows, m, rows, cols, 64,
                              B.WC_T_FP16))
    assert torch.equal(y, linear4(x, want4))


def test_out_across_the_weights_is_refused(dev):
    x = _normal(1, dev, BF, 4, 64)
    w = _normal(2, dev, BF, 4, 64, 64)
    ends = torch.tensor([1, 2, 3, 4], device=dev)
    with pytest.raises(ValueError, match="memory in common"):
        grouped_linear(x, w, ends, out=w[1][:4])
    q = quantize4(w[0])
    held = torch.zeros(64 * 64, dtype=BF, device=dev)
    scales = held[:64].view(64, 1)
    with pytest.raises(ValueError, match="memory in common"):
        linear4(x, Weights4(q.q, scales, None, 64), out=held[:256].view(4, 64))

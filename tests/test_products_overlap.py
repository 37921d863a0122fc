"""Results in the memory of inputs, or of each other, that are still to be read:
refused at the C boundary before anything is launched.  What is side by side in
rows of one pitch passes, and gives what it gives apart."""
import pytest

import lossless_weight_compression_bf16_amd as wc
from lossless_weight_compression_bf16_amd import _binding as B

torch = pytest.importorskip("torch")

BIG = 1 << 50
M, E, N, K = 1000, 4, 512, 1024


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: only where nothing can be launched on them")
    return wc.lib()


def _across(at, size, other):
    """Places of `other` bytes that have some of the `size` bytes from `at` on, all of them 256-byte aligned."""
    last = (size - 1) // 256 * 256
    return [at, at + last, at - (other - 1) // 256 * 256, at + (size // 2) // 256 * 256]


def _grouped(**kw):
    s = B.wc_grouped(0x10000000, K, 0x20000000, N * K, K, 0x30000000, 0x40000000, N, M, E, N, K, B.WC_T_BF16, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _grouped_grad(**kw):
    s = B.wc_grouped_grad(0x10000000, K, 0x20000000, N * K, K, 0x30000000, 0x40000000, N, 0x50000000, K, 0x60000000, M, E, N, K,
                          B.WC_T_BF16, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


X, W, Y, ENDS = 2 * M * K, 2 * E * N * K, 2 * M * N, 8 * E


def test_grouped(L):
    for size, at in ((W, 0x20000000), (ENDS, 0x30000000), (X, 0x10000000)):
        for y in _across(at, size, Y):
            assert L.wc_grouped_linear(_grouped(y=y), 0x8000000, BIG, None, None) == B.WC_ERR_ARG, (hex(at), hex(y))
    # experts further apart than their rows take: y in the gap between two
    far = dict(w_expert=4 * N * K, w=0x20000000)
    assert L.wc_grouped_linear(_grouped(**far, y=0x20000000 + 4 * 4 * N * K), 0x8000000, BIG, None, None) == B.WC_ERR_ARG
    # the last element of the last expert
    assert L.wc_grouped_linear(_grouped(**far, y=0x20000000 + 2 * (3 * 4 * N * K + N * K - 8)), 0x8000000, BIG, None, None) == B.WC_ERR_ARG


def test_grouped_gradient(L):
    def call(**kw):
        return L.wc_grouped_linear_backward(_grouped_grad(**kw), 0x8000000, BIG, None, None)
    for size, at in ((X, 0x10000000), (W, 0x20000000), (ENDS, 0x30000000), (Y, 0x40000000), (W, 0x60000000)):
        for dx in _across(at, size, X):
            assert call(grad_x=dx) == B.WC_ERR_ARG, (hex(at), hex(dx))
    for size, at in ((X, 0x10000000), (ENDS, 0x30000000), (Y, 0x40000000), (X, 0x50000000)):
        for dw in _across(at, size, W):
            assert call(grad_w=dw) == B.WC_ERR_ARG, (hex(at), hex(dw))
    assert call(grad_x=0, grad_w=0x30000000) == B.WC_ERR_ARG and call(grad_w=0, grad_x=0x20000000) == B.WC_ERR_ARG
    assert call(m=0, grad_w=0x30000000) == B.WC_ERR_ARG


V = 5000


def _loss(**kw):
    s = B.wc_linear_loss(0x10000000, K, 0x20000000, K, 0x30000000, M, V, K, B.WC_T_BF16, 0, 0x40000000, 0x50000000)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _loss_grad(**kw):
    s = B.wc_linear_loss_grad(0x10000000, K, 0x20000000, K, 0x30000000, 0x40000000, 0x50000000, 0x60000000, 0x70000000, K, 0x80000000,
                              M, V, K, B.WC_T_BF16)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_loss(L):
    for size, at in ((X, 0x10000000), (2 * V * K, 0x20000000), (8 * M, 0x30000000)):
        for to in _across(at, size, 4 * M):
            for name in ("loss", "lse"):
                assert L.wc_linear_cross_entropy(_loss(**{name: to}), 0x8000000, BIG, None, None) == B.WC_ERR_ARG, (name, hex(to))
    for to in _across(0x50000000, 4 * M, 4 * M):
        assert L.wc_linear_cross_entropy(_loss(loss=to), 0x8000000, BIG, None, None) == B.WC_ERR_ARG, hex(to)


def test_loss_gradient(L):
    def call(**kw):
        return L.wc_linear_cross_entropy_backward(_loss_grad(**kw), 0x8000000, BIG, None, None)
    inputs = ((X, 0x10000000), (2 * V * K, 0x20000000), (8 * M, 0x30000000), (4 * M, 0x40000000), (4 * M, 0x50000000),
              (4 * M, 0x60000000))
    for size, at in inputs + ((2 * V * K, 0x80000000),):
        for to in _across(at, size, X):
            assert call(grad_hidden=to) == B.WC_ERR_ARG, (hex(at), hex(to))
    for size, at in inputs + ((X, 0x70000000),):
        for to in _across(at, size, 2 * V * K):
            assert call(grad_weight=to) == B.WC_ERR_ARG, (hex(at), hex(to))


def test_4_bits(L):
    m, rows, cols, group = 7, 512, 1024, 64
    for size, at, name in ((rows * cols // 2, 0x20000000, "q"), (2 * rows * cols // group, 0x30000000, "scales"),
                           (2 * rows * cols // group, 0x40000000, "zeros")):
        for y in _across(at, size, 2 * m * rows):
            s = B.wc_fourbit(0x10000000, cols, 0x20000000, 0x30000000, 0x40000000, y, rows, m, rows, cols, group, B.WC_T_BF16)
            assert L.wc_linear4(s, None) == B.WC_ERR_ARG, (name, hex(y))
    sizes = {"w": 2 * rows * cols, "q": rows * cols // 2, "scales": 2 * rows * cols // group, "zeros": 2 * rows * cols // group}
    places = {"w": 0x10000000, "q": 0x20000000, "scales": 0x30000000, "zeros": 0x40000000}
    for a in places:
        for b in places:
            if a == b:
                continue
            for to in _across(places[a], sizes[a], sizes[b]):
                p = {**places, b: to}
                assert L.wc_quantize4(p["w"], cols, rows, cols, group, B.WC_T_BF16, p["q"], p["scales"], p["zeros"],
                                      None) == B.WC_ERR_ARG, (a, b, hex(to))


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 70, 600])
def test_side_by_side_passes(dev, m):
    """y and x, y and the weights, and gradients and inputs in the columns of one buffer."""
    g = torch.Generator(device=dev).manual_seed(m)
    n, k, e = 64, 128, 2
    print(f"[overlap] side by side, {m} rows", flush=True)
    r = max(m, e * n)
    buf = torch.randn((r, 3 * k), generator=g, device=dev).bfloat16()
    x, w, y = buf[:m, :k], buf[:e * n, k:2 * k].unflatten(0, (e, n)), buf[:m, 2 * k:2 * k + n]
    ends = torch.tensor([m // 3, m], device=dev)
    want = wc.grouped_linear(x.contiguous(), w.contiguous(), ends)
    d = torch.randn((m, n), generator=g, device=dev).bfloat16()
    dx, dw = wc.grouped_linear_backward(x.contiguous(), w.contiguous(), ends, d)
    before = buf.clone()
    row = 3 * k
    scratch = torch.empty(max(B.wc_grouped_linear_scratch(m, e, n, k), B.wc_grouped_linear_backward_scratch(m, e, n, k), 256),
                          dtype=torch.uint8, device=dev)
    B.wc_grouped_linear(B.wc_grouped(x.data_ptr(), row, w.data_ptr(), n * row, row, ends.data_ptr(), y.data_ptr(), row, m, e, n, k,
                                     B.WC_T_BF16, 1), scratch, scratch.numel())
    before[:m, 2 * k:2 * k + n] = want
    assert torch.equal(buf, before)
    # the gradient of x where y was, that of w behind all
    to = torch.empty_like(dw)
    B.wc_grouped_linear_backward(B.wc_grouped_grad(x.data_ptr(), row, w.data_ptr(), n * row, row, ends.data_ptr(), d.data_ptr(), n,
                                                   buf[:, 2 * k:].data_ptr(), row, to.data_ptr(), m, e, n, k, B.WC_T_BF16, 1),
                                 scratch, scratch.numel())
    assert torch.equal(buf[:m, 2 * k:], dx) and torch.equal(to, dw) and torch.equal(buf[:, :2 * k], before[:, :2 * k])
    # and in x's own place, where x is not read
    B.wc_grouped_linear_backward(B.wc_grouped_grad(0, 0, w.data_ptr(), n * row, row, ends.data_ptr(), d.data_ptr(), n,
                                                   x.data_ptr(), row, 0, m, e, n, k, B.WC_T_BF16, 1), scratch, scratch.numel())
    assert torch.equal(buf[:m, :k], dx)

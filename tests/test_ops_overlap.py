"""Outputs in the memory of inputs: refused at the C boundary before anything
is launched, except where every element is read before its place is written."""
import pytest

import lossless_weight_compression_bf16_amd as wc
from lossless_weight_compression_bf16_amd import _binding as B

torch = pytest.importorskip("torch")

BF = torch.bfloat16


def test_adapters_refuse_y_across_x():
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: only where nothing can be launched on them")
    lib, base = wc.lib(), 0x100000
    for y_type, size in ((B.WC_T_BF16, 2), (B.WC_T_FP32, 4)):
        for m in (1, 5, 64, 600):
            need = lib.wc_add_adapters_scratch(m, 16, 64, 64)
            for at, stride in ((0, 64), (2 * 63, 64), (-size * 63, 64), (0, 200), (2 * 64 * (m - 1), 64)):
                s = B.wc_adapters(base, 64, base + at, stride, 0x800000, 0x900000, 0xA00000, 0, m, 4, 16, 64, 64,
                                  B.WC_T_BF16, y_type)
                assert lib.wc_add_adapters(s, 0x10000000, need, None, None) == B.WC_ERR_ARG, (y_type, m, at, stride)
            # side by side, one element short of room
            s = B.wc_adapters(base, 64 + 32 * size, base + 2 * 64, (64 + 32 * size) * 2 // size, 0x8000000, 0x9000000,
                              0xA000000, 0, m, 4, 16, 64, 65, B.WC_T_BF16, y_type)
            if m > 1:
                assert lib.wc_add_adapters(s, 0x10000000, 1 << 30, None, None) == B.WC_ERR_ARG, (y_type, m)


def test_gradient_refuses_out_across_logits():
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: only where nothing can be launched on them")
    lib, base = wc.lib(), 0x100000
    for m, at, stride in ((1, 4, 100), (1, -4 * 99, 100), (3, 400, 100), (3, -800, 100), (3, 4, 100), (3, 0, 101),
                          (2, 4 * 199, 100)):
        s = B.wc_logprobs_grad(base, 100, base + at, stride, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, m, 100, B.WC_T_FP32)
        assert lib.wc_token_logprobs_backward(s, None, None) == B.WC_ERR_ARG, (m, at, stride)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 3, 61, 600])
def test_adapters_into_their_own_input(dev, m):
    from lossless_weight_compression_bf16_amd.adapters import add_adapters
    n, rank, c = 3, 16, 512
    g = torch.Generator().manual_seed(m)

    def normal(*shape):
        return torch.randn(shape, generator=g).to(BF).to(dev)
    a, b, ids = normal(n, rank, c), normal(n, c, rank), (torch.arange(m) % n).to(dev)
    for x_at, y_at, width in ((0, 0, c), (8, 0, c + 8), (0, 3, c + 8), (0, c, 2 * c), (c, 0, 2 * c), (0, 8, c + 64)):
        print(f"[overlap] adapters, {m} tokens, x at {x_at}, y at {y_at} of rows of {width}", flush=True)
        buf = normal(m, width)
        x, y = buf[:, x_at:x_at + c], buf[:, y_at:y_at + c]
        want = buf.clone()
        want[:, y_at:y_at + c] = add_adapters(x.clone(), y.clone(), a, b, ids)
        assert add_adapters(x, y, a, b, ids) is y
        assert torch.equal(buf, want)


@pytest.mark.gpu
def test_gradient_across_the_logits(dev):
    from lossless_weight_compression_bf16_amd import logprobs as L
    m, v = 5, 9001
    for rows, cols in ((0, 0), (1, 0), (0, 3), (2, 5)):
        print(f"[overlap] gradient, out {rows} rows and {cols} columns behind the logits", flush=True)
        buf = torch.randn((m + 2, v + 8), generator=torch.Generator().manual_seed(rows + cols)).to(dev)
        z, out = buf[:m, :v], buf[rows:rows + m, cols:cols + v]
        t = torch.arange(m, device=dev)
        r = L.token_logprobs(z, t)
        one = torch.ones(m, device=dev)
        want = buf.clone()
        want[rows:rows + m, cols:cols + v] = L.token_logprobs_backward(z, t, r.lse, r.entropy, one, one)
        assert L.token_logprobs_backward(z, t, r.lse, r.entropy, one, one, out=out) is out
        assert torch.equal(buf, want)

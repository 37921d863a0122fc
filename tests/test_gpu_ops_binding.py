"""The operators through the binding, call by call as in the C header: a
caller's own buffers and scratch, the same results as the tensor-level calls."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import _binding as B, adapters as A, logprobs as L, moe as M  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


def _scratch(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def test_log_probabilities(dev):
    m, v, top = 3, 140001, 5
    z, t = torch.randn((m, v), device=dev), torch.tensor([0, -1, v], device=dev)
    lp, ent, lse = (torch.empty(m, device=dev) for _ in range(3))
    best, ids = torch.empty((m, top), device=dev), torch.empty((m, top), dtype=torch.int64, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    n = B.wc_token_logprobs_scratch(m, v, top)
    B.wc_token_logprobs(B.wc_logprobs(z.data_ptr(), v, t.data_ptr(), m, v, top, B.WC_T_FP32, 0, lp.data_ptr(), ent.data_ptr(),
                                      lse.data_ptr(), best.data_ptr(), ids.data_ptr()), _scratch(n, dev), n, err)
    want = L.token_logprobs(z, t, top=top, check=False)
    assert int(err.item()) == B.EF_BAD_INDEX
    assert torch.equal(lp[:2], want.logprob[:2]) and bool(lp[2].isnan())
    assert all(torch.equal(a, b) for a, b in zip((ent, lse, best, ids), want[1:]))
    err.zero_()
    out, g = torch.empty_like(z), torch.ones(m, device=dev)
    B.wc_token_logprobs_backward(B.wc_logprobs_grad(z.data_ptr(), v, out.data_ptr(), v, t.data_ptr(), lse.data_ptr(),
                                                    ent.data_ptr(), g.data_ptr(), g.data_ptr(), m, v, B.WC_T_FP32), err)
    assert int(err.item()) == B.EF_BAD_INDEX
    assert torch.equal(out, L.token_logprobs_backward(z, t, lse, ent, g, g, check=False))


def test_adapters(dev):
    m, n, rank, cols, rows = 70, 3, 20, 520, 300
    x, a, b = (torch.randn(s, device=dev).to(BF) for s in ((m, cols), (n, rank, cols), (n, rows, rank)))
    y, ids = torch.randn((m, rows), device=dev), torch.arange(m, device=dev) % n
    want = A.add_adapters(x, y.clone(), a, b, ids)
    size = B.wc_add_adapters_scratch(m, rank, cols, rows)
    B.wc_add_adapters(B.wc_adapters(x.data_ptr(), cols, y.data_ptr(), rows, a.data_ptr(), b.data_ptr(), ids.data_ptr(), 0, m,
                                    n, rank, cols, rows, B.WC_T_BF16, B.WC_T_FP32), _scratch(size, dev), size)
    assert torch.equal(y, want)


def test_experts(dev):
    m, e, h, i = 5, 6, 64, 40
    x, r, w1, w3, w2 = (torch.randn(s, device=dev).to(BF) / 8 for s in ((m, h), (e, h), (e, i, h), (e, i, h), (e, h, i)))
    out = torch.empty_like(x)
    size = B.wc_moe_layer_scratch(m, e, 2, h, i)
    B.wc_moe_layer(B.wc_moe(x.data_ptr(), h, r.data_ptr(), w1.data_ptr(), w3.data_ptr(), w2.data_ptr(), i * h, h, h * i, i,
                            out.data_ptr(), h, m, e, 2, h, i, B.WC_T_BF16, 1), _scratch(size, dev), size)
    assert torch.equal(out, M.moe_layer(x, r, w1, w3, w2, 2))


def test_refusals_raise(dev):
    with pytest.raises(B.WcError, match="wc_moe_layer"):
        B.wc_moe_layer(B.wc_moe(), None, 0)
    with pytest.raises(B.WcError, match="wc_add_adapters"):
        B.wc_add_adapters(B.wc_adapters(), None, 0)
    with pytest.raises(B.WcError, match="wc_token_logprobs"):
        B.wc_token_logprobs(B.wc_logprobs(), None, 0)
    with pytest.raises(B.WcError, match="wc_token_logprobs_backward"):
        B.wc_token_logprobs_backward(B.wc_logprobs_grad())

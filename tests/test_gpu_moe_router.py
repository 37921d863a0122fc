"""A token with a NaN among its router's logits: softmax over all experts makes
all of its weights NaN, whether or not they are divided by the chosen ones'
sum, and whether or not the expert in question is chosen."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import lossless_weight_compression_bf16_amd as wc  # noqa: E402
from lossless_weight_compression_bf16_amd import moe as M  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    wc.lib()
    return torch.device("cuda:0")


# the router in one launch (small), and in parts
@pytest.mark.parametrize("m,experts,cols", [(1, 6, 64), (5, 6, 64), (20, 70, 64), (1, 70, 1024), (40, 300, 256)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_one_nan_logit(dev, m, experts, cols, renormalize):
    print(f"[moe router] {m} tokens, {experts} experts, {cols} columns, renormalize={renormalize}", flush=True)
    inner = 24
    g = torch.Generator().manual_seed(m + cols)
    x, r, w1, w3, w2 = (torch.randn(s, generator=g) for s in ((m, cols), (experts, cols), (experts, inner, cols),
                                                              (experts, inner, cols), (experts, cols, inner)))
    # expert 2's logit is inf - inf for the last token and as ever for the others; nothing else sees its two numbers
    for t in (x, r, w1, w3):
        t[..., :2] = 0.0
    args = [t.to(torch.bfloat16).to(dev) for t in (x, r, w1, w3, w2)]
    want = M.moe_layer(*args, 2, renormalize=renormalize)
    assert bool(want.isfinite().all())
    args[0][-1, :2] = 3e38
    args[1][2, 0], args[1][2, 1] = 3e38, -3e38
    assert math.isnan(float(args[0][-1, :2].float() @ args[1][2, :2].float()))
    got = M.moe_layer(*args, 2, renormalize=renormalize)
    assert torch.equal(got[:-1], want[:-1])
    assert bool(got[-1].isnan().all())

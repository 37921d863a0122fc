"""4-bit weights at the edges of what the types hold, and what cannot be followed by autograd.

Tolerances: as in test_gpu_fourbit.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from lossless_weight_compression_bf16_amd import fourbit as F  # noqa: E402
from test_gpu_fourbit import BF, HF, _check, _inputs, _say, dev  # noqa: E402, F401


@pytest.mark.parametrize("zeros", [False, True])
def test_making_them_has_no_gradient_and_says_so(dev, zeros):  # noqa: F811
    w = torch.randn((16, 128), generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(BF)
    want = F.quantize4(w, 64, zeros)
    p = torch.nn.Parameter(w.clone())
    for t in (p, 2 * p):
        with pytest.raises(RuntimeError, match="quantize4 has no backward pass"):
            F.quantize4(t, 64, zeros)
    with torch.no_grad():
        got = F.quantize4(p, 64, zeros)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    assert all(a is None or torch.equal(a, b) for a, b in zip(F.quantize4(p.detach(), 64, zeros)[:3], want[:3]))
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(RuntimeError, match="forward-mode"):
            F.quantize4(forward_ad.make_dual(w, w), 64, zeros)
        assert torch.equal(F.quantize4(w, 64, zeros).q, want.q)

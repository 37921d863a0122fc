"""Sizes past what a call takes, refused at the C boundary (and scratch sizes
of 0) before anything is launched."""
import pytest

import lossless_weight_compression_bf16_amd as wc
from lossless_weight_compression_bf16_amd import _binding as B

torch = pytest.importorskip("torch")


def test_scratch_of_sizes_past_the_limits():
    lib = wc.lib()
    assert lib.wc_token_logprobs_scratch((1 << 31) - 1, 131073, 0) == ((1 << 31) - 1) * 2 * 16
    assert lib.wc_token_logprobs_scratch(1 << 31, 131073, 0) == 0
    # experts with tokens times rows of 16: below 2^24
    assert lib.wc_moe_layer_scratch(64, 1024, 16, 8, (1 << 18) - 16) > 0
    assert lib.wc_moe_layer_scratch(64, 1024, 16, 8, 1 << 18) == 0
    assert lib.wc_moe_layer_scratch(8, 1024, 16, 8, 1 << 20) > 0
    # adapters: several sets of launches share the scratch of one
    assert lib.wc_add_adapters_scratch(1 << 31, 8, 64, 48) == lib.wc_add_adapters_scratch(1 << 24, 8, 64, 48) > 0


def test_refusals_past_the_limits():
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: only where nothing can be launched on them")
    lib = wc.lib()
    z = B.wc_logprobs(0x1000, 10, 0x2000, 1 << 31, 10, 0, B.WC_T_BF16, 0, 0x3000, 0x4000, 0x5000, 0, 0)
    assert lib.wc_token_logprobs(z, None, 0, None, None) == B.WC_ERR_ARG
    d = B.wc_logprobs_grad(0x1000, 10, 0x1000, 10, 0x2000, 0x3000, 0, 0, 0, 1 << 31, 10, B.WC_T_BF16)
    assert lib.wc_token_logprobs_backward(d, None, None) == B.WC_ERR_ARG
    e = B.wc_moe(0x10000, 8, 0x20000, 0x30000, 0x40000, 0x50000, 1 << 21, 8, 1 << 21, 1 << 18, 0x60000, 8, 64, 1024, 16, 8,
                 1 << 18, B.WC_T_BF16, 1)
    assert lib.wc_moe_layer(e, 0x100000, 1 << 50, None) == B.WC_ERR_ARG


def test_adapters_in_one_launch_need_no_scratch():
    """One launch where a block reads at most 256 KiB of A, and all of them 16 MiB."""
    lib = wc.lib()
    for m, rank, cols, rows, one in ((1, 16, 4096, 4096, True), (1, 32, 4096, 4096, True), (1, 33, 4096, 4096, False),
                                     (1, 64, 2048, 4096, True), (1, 64, 2056, 4096, False), (64, 16, 4096, 4096, True),
                                     (64, 16, 4096, 14336, False), (65, 16, 64, 64, False), (1, 65, 64, 64, False)):
        assert (lib.wc_add_adapters_scratch(m, rank, cols, rows) == 0) == one, (m, rank, cols, rows)


@pytest.mark.gpu
def test_experts_past_the_limit():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    from lossless_weight_compression_bf16_amd.moe import moe_layer
    bf, inner = torch.bfloat16, 1 << 18
    x, r = torch.zeros((64, 8), dtype=bf, device="cuda"), torch.zeros((1024, 8), dtype=bf, device="cuda")
    up = torch.zeros((1, inner, 8), dtype=bf, device="cuda").expand(1024, inner, 8)
    down = torch.zeros((1, 8, inner), dtype=bf, device="cuda").expand(1024, 8, inner)
    with pytest.raises(ValueError, match="below 2\\^28"):
        moe_layer(x, r, up, up, down, 16)
    assert moe_layer(x, r, up[:, :1024], up[:, :1024], down[:, :, :1024], 2).shape == x.shape

"""The C ABI of the products grouped by expert, the cross entropy from hidden
states and the products with weights of 4 bits, without a GPU: scratch sizes,
limits and every refusal, before anything is launched."""
import ctypes
import os

import pytest

import lossless_weight_compression_bf16_amd as wc
from lossless_weight_compression_bf16_amd import _binding as B

torch = pytest.importorskip("torch")

BIG = 1 << 50  # bytes of scratch: never too few


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: only where nothing can be launched on them")
    if not os.path.exists(B.LIB_PATH):
        from lossless_weight_compression_bf16_amd import build
        build.build()
    return wc.lib()


def _with(s, **kw):
    c = type(s).from_buffer_copy(s)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_struct_sizes():
    """The ctypes mirrors follow the C structs' natural alignment."""
    assert ctypes.sizeof(B.wc_grouped) == 96
    assert ctypes.sizeof(B.wc_grouped_grad) == 120
    assert ctypes.sizeof(B.wc_linear_loss) == 80
    assert ctypes.sizeof(B.wc_linear_loss_grad) == 112
    assert ctypes.sizeof(B.wc_fourbit) == 80


GROUPED = B.wc_grouped(0x100000, 64, 0x200000, 64 * 48, 64, 0x300000, 0x400000, 48, 600, 4, 48, 64, B.WC_T_BF16, 0)


def test_grouped_refusals(L):
    def call(s, scratch=0x8000000, nbytes=BIG, err=None):
        return L.wc_grouped_linear(s, scratch, nbytes, err, None)
    assert L.wc_grouped_linear(None, None, 0, None, None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"type": 7}, {"experts": 0}, {"experts": 1025}, {"rows": 0}, {"rows": 44},
               {"rows": (1 << 20) + 8}, {"cols": 0}, {"cols": 60}, {"cols": (1 << 20) + 8}, {"x": 0}, {"x": 0x100008},
               {"x_stride": 56}, {"x_stride": 68}, {"x_stride": 1 << 22}, {"w": 0}, {"w": 0x200002}, {"w_row": 56},
               {"w_row": 65}, {"w_row": 1 << 22}, {"w_expert": 64 * 48 + 4}, {"ends": 0}, {"ends": 0x300004}, {"y": 0},
               {"y": 0x400004}, {"y_stride": 40}, {"y_stride": 50}, {"y_stride": 1 << 22}, {"m": 1 << 31},
               {"y": 0x100000}, {"y": 0x100000 + 2 * 64 * 599}, {"y": 0x100000 - 2 * 48 * 599}):
        assert call(_with(GROUPED, **kw)) == B.WC_ERR_ARG, kw
    assert call(GROUPED, err=0x9002) == B.WC_ERR_ARG
    assert call(_with(GROUPED, m=0)) == B.WC_OK  # nothing to do


def test_grouped_scratch(L):
    # no last round to be split: few rows of each expert, or a short k
    assert L.wc_grouped_linear_scratch(2, 8, 1024, 2048) == 0
    assert L.wc_grouped_linear_scratch(600, 4, 48, 64) == 0
    for bad in ((0, 4, 48, 64), (600, 0, 48, 64), (600, 1025, 48, 64), (600, 4, 44, 64), (600, 4, 48, 60), (1 << 31, 4, 48, 64),
                (1000, 4, (1 << 20) + 8, 64)):
        assert L.wc_grouped_linear_scratch(*bad) == 0 and L.wc_grouped_linear_backward_scratch(*bad) == 0, bad
    size = (1000, 8, 4096, 4096)
    need = L.wc_grouped_linear_scratch(*size)
    assert need > 0 and need % 16 == 0
    s = _with(GROUPED, m=1000, experts=8, rows=4096, cols=4096, x_stride=4096, w_row=4096, w_expert=4096 * 4096, y_stride=4096,
              y=0x10000000)
    assert L.wc_grouped_linear(s, 0x8000000, need - 1, None, None) == B.WC_ERR_CAPACITY
    assert L.wc_grouped_linear(s, None, need, None, None) == B.WC_ERR_ARG
    assert L.wc_grouped_linear(s, 0x8000008, need, None, None) == B.WC_ERR_ARG


def test_grouped_limits(L):
    """So many tiles that a launch could not hold them."""
    wide = {"rows": 1 << 20, "y_stride": 1 << 20, "experts": 128, "y": 1 << 40}
    assert L.wc_grouped_linear(_with(GROUPED, **wide), 0x8000000, BIG, None, None) == B.WC_ERR_ARG
    assert L.wc_grouped_linear(_with(GROUPED, m=(1 << 31) - 1, rows=1 << 16, y_stride=1 << 16, y=1 << 40), 0x8000000, BIG, None,
                               None) == B.WC_ERR_ARG
    # where the few rows take their own kernel too
    assert L.wc_grouped_linear(_with(GROUPED, **wide, m=4), 0x8000000, BIG, None, None) == B.WC_ERR_ARG


GROUPED_GRAD = B.wc_grouped_grad(0x100000, 64, 0x200000, 64 * 48, 64, 0x300000, 0x400000, 48, 0x500000, 64, 0x600000, 600, 4, 48,
                                 64, B.WC_T_FP16, 0)


def test_grouped_gradient_refusals(L):
    def call(s, scratch=0x8000000, nbytes=BIG, err=None):
        return L.wc_grouped_linear_backward(s, scratch, nbytes, err, None)
    assert call(None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"experts": 0}, {"experts": 1025}, {"rows": 44}, {"cols": 60}, {"x": 0}, {"x": 0x100008},
               {"x_stride": 56}, {"x_stride": 68}, {"w": 0}, {"w": 0x200002}, {"w_row": 56}, {"w_expert": 4}, {"ends": 0},
               {"ends": 0x300004}, {"grad": 0}, {"grad": 0x400004}, {"grad_stride": 40}, {"grad_stride": 52},
               {"grad_x": 0x500008}, {"grad_x_stride": 56}, {"grad_x_stride": 66}, {"grad_w": 0x600008}, {"m": 1 << 31},
               {"grad_x": 0x400000}, {"grad_x": 0x400000 + 2 * 48 * 599}):
        assert call(_with(GROUPED_GRAD, **kw)) == B.WC_ERR_ARG, kw
    assert call(GROUPED_GRAD, err=0x9002) == B.WC_ERR_ARG
    # neither asked for
    assert call(_with(GROUPED_GRAD, grad_x=0, grad_w=0)) == B.WC_OK
    # what only the other one needs
    assert call(_with(GROUPED_GRAD, grad_w=0, x=0, m=0)) == B.WC_OK
    size = (1000, 8, 4096, 4096)
    need = L.wc_grouped_linear_backward_scratch(*size)
    assert need > 0
    s = _with(GROUPED_GRAD, m=1000, experts=8, rows=4096, cols=4096, x_stride=4096, w_row=4096, w_expert=4096 * 4096,
              grad_stride=4096, grad_x_stride=4096, grad_x=0x10000000)
    assert call(s, nbytes=need - 1) == B.WC_ERR_CAPACITY
    assert call(s, scratch=0) == B.WC_ERR_ARG and call(s, scratch=0x8000008) == B.WC_ERR_ARG


LOSS = B.wc_linear_loss(0x100000, 64, 0x200000, 64, 0x300000, 100, 1000, 64, B.WC_T_BF16, 0, 0x400000, 0x500000)


def test_loss_refusals(L):
    need = L.wc_linear_cross_entropy_scratch(100, 1000, 64)

    def call(s, scratch=0x8000000, nbytes=BIG, err=None):
        return L.wc_linear_cross_entropy(s, scratch, nbytes, err, None)
    assert need > 0 and call(None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"vocab": 0}, {"vocab": (1 << 22) + 1}, {"cols": 0}, {"cols": 60}, {"cols": (1 << 20) + 8},
               {"hidden": 0}, {"hidden": 0x100008}, {"hidden_stride": 56}, {"hidden_stride": 68}, {"hidden_stride": 1 << 22},
               {"weight": 0}, {"weight": 0x200002}, {"weight_stride": 56}, {"weight_stride": 65}, {"tokens": 0},
               {"tokens": 0x300004}, {"loss": 0}, {"loss": 0x400002}, {"lse": 0}, {"lse": 0x500001}, {"m": (1 << 19) + 1}):
        assert call(_with(LOSS, **kw)) == B.WC_ERR_ARG, kw
    assert call(LOSS, err=0x9002) == B.WC_ERR_ARG
    assert call(LOSS, nbytes=need - 1) == B.WC_ERR_CAPACITY
    assert call(LOSS, scratch=0) == B.WC_ERR_ARG and call(LOSS, scratch=0x8000010) == B.WC_ERR_ARG
    assert call(_with(LOSS, m=0)) == B.WC_OK  # nothing to do


LOSS_GRAD = B.wc_linear_loss_grad(0x100000, 64, 0x200000, 64, 0x300000, 0x400000, 0x500000, 0x600000, 0x700000, 64, 0x800000, 100,
                                  1000, 64, B.WC_T_BF16)


def test_loss_gradient_refusals(L):
    need = L.wc_linear_cross_entropy_backward_scratch(100, 1000, 64)

    def call(s, scratch=0x8000000, nbytes=BIG, err=None):
        return L.wc_linear_cross_entropy_backward(s, scratch, nbytes, err, None)
    assert need > 0 and call(None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"vocab": 0}, {"vocab": (1 << 22) + 1}, {"cols": 60}, {"hidden": 0}, {"hidden": 0x100008},
               {"hidden_stride": 56}, {"weight": 0}, {"weight": 0x200004}, {"weight_stride": 60}, {"tokens": 0},
               {"tokens": 0x300004}, {"lse": 0}, {"lse": 0x400002}, {"grad_loss": 0x500002}, {"grad_lse": 0x600001},
               {"grad_hidden": 0x700008}, {"grad_hidden_stride": 56}, {"grad_hidden_stride": 66}, {"grad_weight": 0x800008},
               {"m": 0}, {"m": (1 << 19) + 1}):
        assert call(_with(LOSS_GRAD, **kw)) == B.WC_ERR_ARG, kw
    assert call(LOSS_GRAD, err=0x9002) == B.WC_ERR_ARG
    assert call(LOSS_GRAD, nbytes=need - 1) == B.WC_ERR_CAPACITY
    assert call(LOSS_GRAD, scratch=0) == B.WC_ERR_ARG and call(LOSS_GRAD, scratch=0x8000010) == B.WC_ERR_ARG
    assert call(_with(LOSS_GRAD, grad_hidden=0, grad_weight=0)) == B.WC_OK  # neither asked for
    for bad in ((0, 1000, 64), (100, 0, 64), (100, 1000, 60), ((1 << 19) + 1, 1000, 64), (100, (1 << 22) + 1, 64)):
        assert L.wc_linear_cross_entropy_backward_scratch(*bad) == 0, bad
        assert L.wc_linear_cross_entropy_scratch(*bad) == 0, bad


def test_loss_scratch_does_not_grow_with_the_logits(L):
    """A piece of the vocabulary at a time: 2^27 numbers of 16 bits, and what the rows need."""
    small, large = (L.wc_linear_cross_entropy_backward_scratch(4096, v, 4096) for v in (1 << 17, 1 << 22))
    rows = 4096 * 4096 * 2 + 4096 * 64
    assert small < 2 * (1 << 27) + rows + (1 << 24) + 4 * 4096 * 4096 * 16
    assert large < small + (1 << 20)
    assert L.wc_linear_cross_entropy_scratch(1 << 19, 1 << 22, 64) < 1 << 36


FOURBIT = B.wc_fourbit(0x100000, 256, 0x200000, 0x300000, 0x400000, 0x500000, 100, 7, 100, 256, 64, B.WC_T_BF16)


def test_fourbit_refusals(L):
    def call(s):
        return L.wc_linear4(s, None)
    assert call(None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"rows": 0}, {"rows": (1 << 24) + 1}, {"cols": 0}, {"cols": 96}, {"cols": 2 << 20},
               {"group": 0}, {"group": 16}, {"group": 48}, {"group": 256}, {"x": 0}, {"x": 0x100008}, {"x_stride": 248},
               {"x_stride": 260}, {"q": 0}, {"q": 0x200008}, {"scales": 0}, {"scales": 0x300001}, {"zeros": 0x400001}, {"y": 0},
               {"y": 0x500001}, {"y_stride": 99}, {"m": 1 << 31}, {"y": 0x100000}, {"y": 0x100000 + 2 * 256 * 6},
               {"m": (1 << 31) - 1, "rows": 1 << 24, "y_stride": 1 << 24, "y": 1 << 50},
               {"m": 2100, "rows": 1 << 24, "y_stride": 1 << 24, "y": 1 << 50}):
        assert call(_with(FOURBIT, **kw)) == B.WC_ERR_ARG, kw
    assert call(_with(FOURBIT, m=0)) == B.WC_OK  # nothing to do


def test_quantize_refusals(L):
    ok = dict(w=0x100000, w_stride=256, rows=10, cols=256, group=64, type=B.WC_T_BF16, q=0x200000, scales=0x300000, zeros=0x400000)

    def call(**kw):
        return L.wc_quantize4(*{**ok, **kw}.values(), None)
    for kw in ({"w": None}, {"w": 0x100001}, {"w_stride": 255}, {"rows": 0}, {"rows": (1 << 24) + 1}, {"cols": 0}, {"cols": 96},
               {"group": 16}, {"type": B.WC_T_FP32}, {"q": None}, {"q": 0x200008}, {"scales": None}, {"scales": 0x300001},
               {"zeros": 0x400001}):
        assert call(**kw) == B.WC_ERR_ARG, kw

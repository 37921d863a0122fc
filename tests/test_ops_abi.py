"""The C ABI of the operators beside the weights, without a GPU: scratch
sizes and every refusal, before anything is launched."""
import ctypes
import os

import pytest

import lossless_weight_compression_bf16_amd as wc
from lossless_weight_compression_bf16_amd import _binding as B


@pytest.fixture(scope="module")
def L():
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
    assert ctypes.sizeof(B.wc_logprobs) == 88
    assert ctypes.sizeof(B.wc_logprobs_grad) == 88
    assert ctypes.sizeof(B.wc_adapters) == 96
    assert ctypes.sizeof(B.wc_moe) == 128


def test_logprobs_refusals(L):
    # 2^17 + 1 logits: two blocks a row, whose parts need scratch
    assert L.wc_token_logprobs_scratch(3, 131073, 5) == 3 * 2 * (16 + 8 * 5)
    assert L.wc_token_logprobs_scratch(3, 131072, 5) == 0
    assert L.wc_token_logprobs_scratch(0, 100, 5) == 0 and L.wc_token_logprobs_scratch(1, 1 << 23, 0) == 0
    ok = B.wc_logprobs(0x1000, 131073, 0x2000, 3, 131073, 5, B.WC_T_BF16, 0, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000)
    need = L.wc_token_logprobs_scratch(3, 131073, 5)

    def call(s, scratch=0x100000, nbytes=need, err=None):
        return L.wc_token_logprobs(s, scratch, nbytes, err, None)
    assert L.wc_token_logprobs(None, None, 0, None, None) == B.WC_ERR_ARG
    for kw in ({"type": 3}, {"vocab": 0}, {"vocab": (1 << 22) + 1}, {"top": 65}, {"vocab": 4}, {"stride": 131072},
               {"logits": 0}, {"logits": 0x1001}, {"tokens": 0}, {"tokens": 0x2004}, {"logprob": 0}, {"entropy": 0},
               {"lse": 0}, {"lse": 0x5002}, {"top_logprobs": 0}, {"top_ids": 0}, {"top_ids": 0x7004},
               {"m": 1 << 31}):
        assert call(_with(ok, **kw)) == B.WC_ERR_ARG, kw
    assert call(ok, nbytes=need - 1) == B.WC_ERR_CAPACITY
    assert call(ok, scratch=0) == B.WC_ERR_ARG and call(ok, scratch=0x100008) == B.WC_ERR_ARG
    assert call(ok, err=0x9002) == B.WC_ERR_ARG
    assert call(_with(ok, m=0)) == B.WC_OK  # nothing to do


def test_logprobs_gradient_refusals(L):
    ok = B.wc_logprobs_grad(0x1000, 100, 0x9000, 100, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 3, 100, B.WC_T_FP32)

    def call(s, err=None):
        return L.wc_token_logprobs_backward(s, err, None)
    assert call(None) == B.WC_ERR_ARG
    for kw in ({"type": 3}, {"vocab": 0}, {"stride": 99}, {"out_stride": 99}, {"logits": 0}, {"out": 0},
               {"out": 0x9002}, {"tokens": 0}, {"lse": 0}, {"lse": 0x3002}, {"entropy": 0}, {"grad_logprob": 0x5001},
               {"grad_entropy": 0x6002}, {"out": 0x1000, "out_stride": 104}, {"m": 1 << 40}):
        assert call(_with(ok, **kw)) == B.WC_ERR_ARG, kw
    assert call(ok, err=0x9002) == B.WC_ERR_ARG
    assert call(_with(ok, m=0)) == B.WC_OK


def test_adapters_refusals(L):
    ok = B.wc_adapters(0x10000, 64, 0x20000, 48, 0x30000, 0x40000, 0x50000, 0x60000, 600, 4, 8, 64, 48, B.WC_T_BF16,
                       B.WC_T_FP32)
    need = L.wc_add_adapters_scratch(600, 8, 64, 48)
    assert need >= 600 * 32 * 2 * 3 + 600 * 4
    assert L.wc_add_adapters_scratch(1, 16, 4096, 4096) == 0  # few tokens: no scratch
    for bad in ((0, 8, 64, 48), (600, 0, 64, 48), (600, 257, 64, 48), (600, 8, 60, 48), (600, 8, 64, 0),
                (600, 8, 64, 1 << 28), ((1 << 31) + 1, 8, 64, 48)):
        assert L.wc_add_adapters_scratch(*bad) == 0, bad

    def call(s, scratch=0x100000, nbytes=need, err=None):
        return L.wc_add_adapters(s, scratch, nbytes, err, None)
    assert call(None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"y_type": B.WC_T_FP16}, {"rank": 0}, {"rank": 257}, {"cols": 60}, {"cols": 0},
               {"rows": 0}, {"x": 0}, {"x": 0x10008}, {"x_stride": 56}, {"x_stride": 68}, {"y": 0}, {"y": 0x20002},
               {"y_stride": 47}, {"a": 0}, {"a": 0x30008}, {"b": 0}, {"b": 0x40001}, {"ids": 0}, {"ids": 0x50004},
               {"scales": 0x60002}, {"n": 1 << 31}):
        assert call(_with(ok, **kw)) == B.WC_ERR_ARG, kw
    assert call(ok, nbytes=need - 1) == B.WC_ERR_CAPACITY
    assert call(ok, scratch=0) == B.WC_ERR_ARG and call(ok, scratch=0x100008) == B.WC_ERR_ARG
    assert call(ok, err=0x9002) == B.WC_ERR_ARG
    assert call(_with(ok, m=0)) == B.WC_OK


def test_moe_refusals(L):
    ok = B.wc_moe(0x10000, 64, 0x20000, 0x30000, 0x40000, 0x50000, 32 * 64, 64, 64 * 32, 32, 0x60000, 64, 5, 8, 2, 64,
                  32, B.WC_T_BF16, 1)
    need = L.wc_moe_layer_scratch(5, 8, 2, 64, 32)
    assert need >= 5 * 2 * (4 + 4 + 4 * 32 + 4 * 64)
    for bad in ((0, 8, 2, 64, 32), (65, 8, 2, 64, 32), (5, 0, 2, 64, 32), (5, 1025, 2, 64, 32), (5, 8, 0, 64, 32),
                (5, 8, 9, 64, 32), (5, 20, 17, 64, 32), (5, 8, 2, 60, 32), (5, 8, 2, 64, 0), (5, 8, 2, 64, 1 << 21)):
        assert L.wc_moe_layer_scratch(*bad) == 0, bad

    def call(s, scratch=0x100000, nbytes=need):
        return L.wc_moe_layer(s, scratch, nbytes, None)
    assert call(None) == B.WC_ERR_ARG
    for kw in ({"type": B.WC_T_FP32}, {"m": 65}, {"experts": 0}, {"experts": 1025}, {"top_k": 0}, {"top_k": 9},
               {"cols": 60}, {"inner": 30}, {"x": 0}, {"x": 0x10008}, {"x_stride": 56}, {"x_stride": 68}, {"router": 0},
               {"router": 0x20008}, {"w1": 0}, {"w3": 0x40002}, {"w2": 0x50008}, {"up_row": 56}, {"up_row": 68},
               {"up_expert": 4}, {"down_row": 24}, {"down_row": 36}, {"down_row": 1 << 27}, {"down_expert": 4},
               {"out": 0}, {"out": 0x60001}, {"out_stride": 63}):
        assert call(_with(ok, **kw)) == B.WC_ERR_ARG, kw
    assert call(ok, nbytes=need - 1) == B.WC_ERR_CAPACITY
    assert call(ok, scratch=0) == B.WC_ERR_ARG and call(ok, scratch=0x100080) == B.WC_ERR_ARG
    assert call(_with(ok, m=0)) == B.WC_OK


def test_error_bit_has_a_name():
    assert B.error_names(B.EF_BAD_INDEX) == ["index out of range"]

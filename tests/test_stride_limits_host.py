"""Outputs that coincide are refused at the largest strides and sizes too, without a GPU: no call here
gets past the host checks."""
import ctypes

import pytest

from mla_latent_kv_absorb_gb300 import binding, build

P = ctypes.c_void_p
FAR = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return binding.lib()


@pytest.mark.parametrize("tokens,heads,token_stride,head_stride", [
    ((1 << 23) + 1, 2, FAR, FAR),            # (tokens - 1) * token_stride = 2^63
    (2, (1 << 23) + 1, FAR, FAR),
    ((1 << 24) + 1, 2, FAR, FAR),            # 2^64
    (3, (1 << 29) - 1, FAR, FAR // 2),
])
def test_rope_outputs_that_coincide_far_apart(L, tokens, heads, token_stride, head_stride):
    r = binding.Rope(64)
    st = L.mla_rope(ctypes.byref(r.config), 0, tokens, heads, 64, 0, P(0x100000), 64, 64, P(0x800000), token_stride,
                    head_stride, None, 0, 0, P(0x700000), None)
    assert st == binding.MLA_ERR_INVALID_ARG


def test_product_outputs_that_coincide_far_apart(L):
    w = binding.W4Struct(0, 2, 128, 128, 32, 0, 1.0, 0x200000)
    for rows in ((1 << 21) + 1, (1 << 23) + 1):   # inside 2^63 and past it
        assert L.mla_linear_w4(rows, P(0x100000), 256, 128, ctypes.byref(w), P(0x800000), FAR, FAR, None) == \
            binding.MLA_ERR_INVALID_ARG

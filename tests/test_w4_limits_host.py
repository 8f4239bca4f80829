"""The largest sizes of the 4-bit products, without a GPU: what is past them is refused by the host
checks, and no call here gets past those."""
import ctypes

import pytest

from mla_latent_kv_absorb_gb300 import binding, build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return binding.lib()


def _weight(n, k, group=32, heads=1, fmt=0):
    return binding.W4Struct(fmt, heads, n, k, group, 0, 1.0, 0x200000)


def _product(L, rows, n, k, **kw):
    w = _weight(n, k, **kw)
    heads = w.heads
    return L.mla_linear_w4(rows, P(0x1000000), heads * k, k, ctypes.byref(w), P(0x800000), heads * n, n, None)


@pytest.mark.parametrize("group,fmt", [(32, 0), (64, 0), (128, 0), (16, 1)])
def test_rows_past_the_grid_are_refused(L, group, fmt):
    """Four warps over k (few outputs, long k) take 32 rows a thread block, other weights 64, and a grid
    has 65,535 blocks of rows."""
    kw = dict(group=group, fmt=fmt)
    for rows in (65535 * 32 + 1, 65535 * 48, 65535 * 64):
        assert _product(L, rows, 128, 1024, **kw) == binding.MLA_ERR_UNSUPPORTED
    for n, k in ((128, 1024), (128, 128), (8192, 1024)):
        assert _product(L, 65535 * 64 + 1, n, k, **kw) == binding.MLA_ERR_UNSUPPORTED
        assert _product(L, 2 ** 31 - 1, n, k, **kw) == binding.MLA_ERR_UNSUPPORTED


def test_outputs_that_do_not_fit_32_bits_when_filled_up_are_refused(L):
    """The kernels round the outputs up to 4, 8 or 256 at a time in 32 bits."""
    most = 2 ** 31 - 256
    for n in (most + 1, 2 ** 31 - 4, 2 ** 31 - 1):
        w = _weight(n, 32)
        assert L.mla_w4_packed_bytes(ctypes.byref(w)) == 0
        assert _product(L, 1, n, 32) == binding.MLA_ERR_UNSUPPORTED
        assert L.mla_w4_pack(ctypes.byref(w), P(0x100000), P(0x200000), None, P(0x300000), None) == binding.MLA_ERR_UNSUPPORTED
    assert L.mla_w4_packed_bytes(ctypes.byref(_weight(most // 2 + 1, 32, heads=2))) == 0
    # 32 outputs x 128 k a block: 2,048 bytes of codes and 32 x 4 scales
    assert L.mla_w4_packed_bytes(ctypes.byref(_weight(most, 32))) == most // 32 * (2048 + 256)
    assert L.mla_w4_packed_bytes(ctypes.byref(_weight(most // 2, 32, heads=2))) == most // 32 * (2048 + 256)

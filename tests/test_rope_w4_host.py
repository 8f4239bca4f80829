"""Rotary positions, the rotated append and the 4-bit products without a GPU: the rotation's
constants against their formulas, and every refusal of the C ABI and of the binding.  No call here
gets past the host checks, so nothing is launched even where a GPU is present.
"""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from mla_latent_kv_absorb_gb300 import binding, build

P = ctypes.c_void_p
INV, ALIGN, UNSUP = binding.MLA_ERR_INVALID_ARG, binding.MLA_ERR_ALIGNMENT, binding.MLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return binding.lib()


def _steps(rope):
    return [int(v) for v in rope.config.step[: rope.dim // 2]]


def _freqs(dim, base=10000.0):
    return [base ** (-2.0 * i / dim) for i in range(dim // 2)]


def _assert_steps(rope, freqs):
    """step = inv_freq / 2 pi turns: the quotient is rounded in 64 bits (1 / 2 pi and the quotient, two
    half steps of 2^-53, and pow's own last place), whole turns dropped."""
    for s, f in zip(_steps(rope), freqs):
        turns = Fraction(f) / Fraction(2 * math.pi)
        off = abs(Fraction(s, 2 ** 64) - (turns - math.floor(turns)))
        off = min(off, 1 - off)
        assert off <= turns * Fraction(1, 2 ** 50) + Fraction(1, 2 ** 64)


@pytest.mark.parametrize("dim", [2, 32, 64, 128, 256])
def test_plain_frequencies(L, dim):
    r = binding.Rope(dim)
    assert (r.config.dim, r.config.layout, r.magnitude) == (dim, 0, 1.0)
    _assert_steps(r, _freqs(dim))
    _assert_steps(binding.Rope(dim, base=500000.0, layout="half"), _freqs(dim, 500000.0))


def test_linear_and_own_frequencies(L):
    _assert_steps(binding.Rope(64, scaling="linear", factor=4.0), [f / 4 for f in _freqs(64)])
    own = [0.0, 1.0, 7.25, 1e-9]
    r = binding.Rope(8, inv_freq=own, magnitude=0.5)
    _assert_steps(r, own)
    assert r.magnitude == 0.5 and _steps(r)[0] == 0


def test_yarn_frequencies(L):
    """The ends of the ramp by hand for dim 64, base 10,000, 4,096 positions: pair(32) = 32 ln(4096 /
    64 pi) / ln 10000 = 10.47 and pair(1) = 22.51, so the ramp runs from 10 to 23."""
    r = binding.Rope(64, scaling="yarn", factor=40.0, original_len=4096)
    want = []
    for i, f in enumerate(_freqs(64)):
        t = min(max((i - 10) / 13, 0.0), 1.0)
        want.append(f * (1 - t) + f / 40 * t)
    _assert_steps(r, want)
    assert r.magnitude == np.float32(0.1 * math.log(40.0) + 1.0)
    assert binding.Rope(64, scaling="yarn", factor=1.0, original_len=4096).magnitude == 1.0
    assert binding.Rope(64, scaling="yarn", factor=40.0, original_len=4096, magnitude=1.0).magnitude == 1.0


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=7), dict(dim=258), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
    dict(scaling="linear", factor=0.0), dict(scaling="linear", factor=float("nan")),
    dict(scaling="yarn", factor=0.5, original_len=4096), dict(scaling="yarn", factor=2.0),
    dict(scaling="yarn", factor=2.0, original_len=4096, beta_fast=1.0, beta_slow=2.0),
    dict(magnitude=-1.0), dict(magnitude=float("inf")), dict(magnitude=1e-60),
    dict(dim=4, inv_freq=[1.0, -1.0]), dict(dim=4, inv_freq=[1.0, float("inf")]),
    dict(dim=4, inv_freq=[1.0, 0.5], scaling="linear", factor=2.0)])
def test_rope_init_refuses(L, kw):
    with pytest.raises(binding.MlaError) as e:
        binding.Rope(**{"dim": 64, **kw})
    assert e.value.status == INV


def test_rope_names_are_checked(L):
    for kw in (dict(layout="pairs"), dict(scaling="ntk"), dict(dim=8, inv_freq=[1.0])):
        with pytest.raises(ValueError):
            binding.Rope(**{"dim": 64, **kw})
    assert L.mla_rope_init(None, None) == INV


def _rope(L, r=None, dtype=0, tokens=4, heads=8, head_dim=192, off=128, x=0x100000, xs=(1536, 192), out=0x800000,
          os_=(512, 64), rest=0x900000, rs=(1024, 128), pos=0xA00000):
    r = binding.Rope(64) if r is None else r
    return L.mla_rope(ctypes.byref(r.config), dtype, tokens, heads, head_dim, off, P(x), xs[0], xs[1], P(out), os_[0],
                      os_[1], P(rest) if rest else None, rs[0], rs[1], P(pos), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INV), (dict(tokens=-1), INV), (dict(heads=0), INV), (dict(off=-8), INV), (dict(off=129), INV),
    (dict(head_dim=32, off=0), INV), (dict(x=0), INV), (dict(out=0), INV), (dict(pos=0), INV),
    (dict(xs=(-1, 192)), INV), (dict(xs=(1 << 41, 192)), INV), (dict(rs=(-8, 128)), INV),
    (dict(out=0x100000), INV),                                   # in place with rest
    (dict(out=0x100000, rest=0, os_=(1536, 200)), INV),          # in place with other strides
    (dict(rest=0x100000), INV), (dict(rest=0x800000), INV),
    (dict(os_=(0, 64)), INV), (dict(os_=(512, 0)), INV), (dict(os_=(512, 32)), INV),   # elements of out coincide
    (dict(os_=(448, 64)), INV), (dict(rest=0), INV), (dict(rs=(512, 128)), INV),
    (dict(head_dim=64, off=0, xs=(512, 64)), INV),               # rest, and nothing to put there
    (dict(x=0x100001), ALIGN), (dict(out=0x800001), ALIGN), (dict(rest=0x900001), ALIGN), (dict(pos=0xA00002), ALIGN),
    (dict(dtype=2, x=0x100002), ALIGN),
    (dict(tokens=1 << 24, heads=128, os_=(8192, 64), rs=(1 << 14, 128)), UNSUP),
    (dict(head_dim=65538, os_=(512, 64), rs=(1 << 30, 1 << 20)), UNSUP)])
def test_rope_refuses(L, kw, status):
    assert _rope(L, **kw) == status


def test_rope_of_no_tokens_and_of_a_spoilt_config(L):
    assert _rope(L, tokens=0, x=0, out=0, pos=0) == binding.MLA_OK
    for field, value in (("dim", 63), ("dim", 0), ("dim", 300), ("layout", 2), ("magnitude", float("nan")),
                         ("magnitude", 0.0)):
        r = binding.Rope(64)
        setattr(r.config, field, value)
        assert _rope(L, r) == INV
    assert L.mla_rope(None, 0, 1, 1, 64, 0, P(16), 64, 64, P(4096), 64, 64, None, 0, 0, P(16), None) == INV


def _append(L, r=None, n=4, c=0x100000, cs=576, k=0x100400, ks=576, pos=0x200000, slots=0x201000, dtype=0, pages=8,
            pool=0x300000, scale=None, kr=None, q=None, qs=(24576, 192), qc=None, qr=None, err=0x400000):
    r = binding.Rope(64) if r is None else r
    f = lambda v: P(v) if v else None  # noqa: E731
    return L.mla_rope_append_kv(ctypes.byref(r.config), n, f(c), cs, f(k), ks, f(pos), f(slots), dtype, pages, f(pool),
                                f(scale), f(kr), f(q), qs[0], qs[1], f(qc), f(qr), f(err), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INV), (dict(pages=0), INV), (dict(dtype=3), INV), (dict(c=0), INV), (dict(k=0), INV),
    (dict(pos=0), INV), (dict(slots=0), INV), (dict(pool=0), INV), (dict(err=0), INV), (dict(cs=-8), INV),
    (dict(ks=1 << 41), INV), (dict(dtype=1), INV), (dict(dtype=2, scale=0x500000), INV),
    (dict(q=0x600000), INV), (dict(q=0x600000, qc=0x700000), INV),
    (dict(q=0x600000, qc=0x700000, qr=0x800000, qs=(-8, 192)), INV),
    (dict(c=0x100008), ALIGN), (dict(k=0x100408), ALIGN), (dict(cs=577), ALIGN), (dict(ks=580), ALIGN),
    (dict(pool=0x300008), ALIGN), (dict(slots=0x201002), ALIGN), (dict(pos=0x200001), ALIGN),
    (dict(err=0x400002), ALIGN), (dict(dtype=1, scale=0x500002, kr=0x600000), ALIGN),
    (dict(dtype=2, scale=0x500000, kr=0x600008), ALIGN),
    (dict(q=0x600008, qc=0x700000, qr=0x800000), ALIGN), (dict(q=0x600000, qc=0x700008, qr=0x800000), ALIGN),
    (dict(q=0x600000, qc=0x700000, qr=0x800008), ALIGN),
    (dict(q=0x600000, qc=0x700000, qr=0x800000, qs=(24576, 196)), ALIGN),
    (dict(q=0x600000, qc=0x700000, qr=0x800000, qs=(24577, 192)), ALIGN),
    (dict(q=0x600000, qc=0x600000, qr=0x800000), INV), (dict(q=0x600000, qc=0x700000, qr=0x600000), INV),
    (dict(q=0x600000, qc=0x700000, qr=0x700000), INV),           # queries over themselves
    (dict(n=(1 << 23) + 1), UNSUP)])
def test_rope_append_refuses(L, kw, status):
    assert _append(L, **kw) == status


def test_rope_append_of_nothing_and_of_another_dim(L):
    assert _append(L, n=0, c=0, k=0, slots=0) == binding.MLA_OK
    assert _append(L, binding.Rope(128)) == INV


def _weight(**kw):
    f = dict(format=0, heads=1, n=512, k=128, group=32, has_zero=0, tensor_scale=1.0, packed=0x200000)
    f.update(kw)
    return binding.W4Struct(*[f[n] for n, _ in binding.W4Struct._fields_])


def _w4(L, rows=4, x=0x100000, xs=(128, 128), out=0x800000, os_=(512, 512), **kw):
    w = _weight(**kw)
    return L.mla_linear_w4(rows, P(x) if x else None, xs[0], xs[1], ctypes.byref(w), P(out) if out else None, os_[0],
                           os_[1], None)


SHAPES = [(dict(format=2), INV), (dict(heads=0), INV), (dict(n=0), INV), (dict(k=0), INV), (dict(group=16), INV),
          (dict(group=48), INV), (dict(k=144), INV), (dict(k=96, group=64), INV), (dict(format=1), INV),
          (dict(format=1, group=16, has_zero=1), INV), (dict(format=1, group=16, k=48), INV), (dict(has_zero=2), INV),
          (dict(tensor_scale=float("nan")), INV), (dict(tensor_scale=float("inf")), INV), (dict(heads=65536), UNSUP),
          (dict(heads=65535, n=40000), UNSUP), (dict(k=(1 << 30) + 128), UNSUP), (dict(n=1 << 30, k=1 << 14), UNSUP)]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(rows=-1), INV), (dict(x=0), INV), (dict(out=0), INV), (dict(packed=None), INV), (dict(out=0x100000), INV),
    (dict(xs=(-8, 128)), INV), (dict(os_=(-8, 512)), INV), (dict(os_=(256, 512)), INV), (dict(os_=(0, 512)), INV),
    (dict(heads=2, os_=(512, 512)), INV), (dict(heads=2, os_=(1024, 256)), INV), (dict(xs=(1 << 41, 128)), INV),
    (dict(x=0x100008), ALIGN), (dict(packed=0x200008), ALIGN), (dict(out=0x800001), ALIGN),
    (dict(xs=(132, 128)), ALIGN), (dict(heads=2, xs=(256, 132), os_=(1024, 512)), ALIGN)])
def test_w4_refuses(L, kw, status):
    assert _w4(L, **kw) == status


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(codes=0), INV), (dict(scale=0), INV), (dict(to=0), INV), (dict(zero=0x400000), INV), (dict(has_zero=1), INV),
    (dict(codes=0x200008), ALIGN), (dict(scale=0x300001), ALIGN), (dict(to=0x500008), ALIGN)])
def test_w4_pack_refuses(L, kw, status):
    p = dict(codes=0x200000, scale=0x300000, zero=0, to=0x500000)
    p.update({k: v for k, v in kw.items() if k in p})
    w = _weight(**{k: v for k, v in kw.items() if k not in p})
    f = lambda v: P(v) if v else None  # noqa: E731
    assert L.mla_w4_pack(ctypes.byref(w), f(p["codes"]), f(p["scale"]), f(p["zero"]), f(p["to"]), None) == status


def test_w4_packed_bytes(L):
    """Steps of four blocks of 32 n x 128 k: 2,048 bytes of codes, and 32 scales and zeros per group of
    k; the four side by side over n (128 outputs) or, for few outputs, over k."""
    size = lambda **kw: L.mla_w4_packed_bytes(ctypes.byref(_weight(**kw)))  # noqa: E731
    assert size(n=512, k=128, group=128) == 16 * (2048 + 64)
    assert size(n=33, k=160, group=32, has_zero=1, heads=3) == 3 * 2 * 4 * (2048 + 256 + 128)
    assert size(n=1, k=64, group=64, has_zero=1) == 4 * (2048 + 128 + 64)
    assert size(n=32, k=128, group=16, format=1) == 4 * (2048 + 256)
    assert size(n=64, k=16384, group=128) == 2 * 128 * (2048 + 64)
    assert all(size(**kw) == 0 for kw, _ in SHAPES)
    assert L.mla_w4_packed_bytes(None) == 0


def test_w4_of_no_rows_and_head_shapes(L):
    assert _w4(L, rows=0, x=0, out=0) == binding.MLA_OK
    assert L.mla_linear_w4(1, P(16), 8, 8, None, P(4096), 8, 8, None) == INV
    w = _weight(heads=128)
    for fn, bad in ((L.mla_absorb_q_w4, dict(heads=128, n=128, k=512)), (L.mla_out_proj_w4, dict(heads=128)),
                    (L.mla_absorb_q_w4, {})):
        v = _weight(**bad)
        assert fn(P(0x100000), ctypes.byref(v), P(0x800000), 1, None) == INV
        assert fn(P(0x100000), None, P(0x800000), 1, None) == INV
    assert L.mla_absorb_q_w4(P(0x100000), ctypes.byref(w), P(0x800000), 0, None) == INV
    assert L.mla_absorb_q_w4(P(0x100008), ctypes.byref(w), P(0x800000), 1, None) == ALIGN


def test_w4_weight_checks():
    """Shapes and types are refused before anything is asked of a GPU."""
    codes = torch.zeros(2, 3, 32, dtype=torch.uint8)
    ones = torch.ones(2, 3, 2, dtype=torch.bfloat16)
    for args, kw in (((codes, ones), dict(group=64)),
                     ((codes, torch.ones(2, 3, 3, dtype=torch.bfloat16)), {}),     # 3 groups of k = 64
                     ((codes, torch.ones(2, 3, 4, dtype=torch.bfloat16)), {}),     # int4 in groups of 16
                     ((codes, ones[0]), {}),                                       # another number of dimensions
                     ((codes[:, :, :24], torch.zeros(2, 3, 3, dtype=torch.uint8)), {}),   # k = 48
                     ((codes, torch.zeros(2, 3, 4, dtype=torch.uint8)), dict(zero=torch.zeros(2, 3, 4, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            binding.W4Weight(*args, **kw)
    for args, kw in (((codes, ones.float()), {}), ((codes, None), {}), ((codes, ones), dict(zero=7))):
        with pytest.raises(TypeError):
            binding.W4Weight(*args, **kw)

"""GPU parity of the rotary positions with so many rows that a thread takes four heads (from 155,648
threads' worth on): every type, layout and path against the formulas in 64 bits, with the tolerances
derived in test_gpu_rope.py, and a check that it is that kernel which ran."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from launch_util import launches_of  # noqa: E402
from test_gpu_rope import DEV, _assert_rotated, _cache, _freqs, _nvfp4_rows, _positions, _tokens  # noqa: E402

from mla_latent_kv_absorb_gb300 import binding  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {torch.bfloat16: "13__nv_bfloat16", torch.float16: "6__half", torch.float32: "f"}


def _four_heads(dtype, vector, layout):
    """The start of the template arguments of the kernel that takes four heads a thread."""
    pieces = (4 if dtype == torch.float32 else 8) if vector else 1
    return f"rope_kernelI{TYPES[dtype]}Li{pieces}ELb{int(layout == 'half')}ELi4EE"


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H,D,dim,off,vector,kind", [
    (1301, 128, 192, 64, 128, True, "near"),   # a prompt's queries
    (1301, 128, 192, 64, 64, True, "far"),     # the rotated part in the middle
    (20011, 8, 64, 64, 0, True, "near"),       # the whole head: nothing copied
    (4101, 12, 77, 26, 13, False, "far"),      # no 16-byte pieces
    (1201, 4, 600, 256, 301, False, "near"),   # more pieces than threads
])
def test_rope_of_many_rows(layout, dtype, T, H, D, dim, off, vector, kind):
    g = torch.Generator().manual_seed(T + D)
    x = torch.randn(T, H, D, generator=g).to(dtype).to(DEV)
    pos = _positions(T, kind, g)
    rope, name = binding.Rope(dim, layout=layout), _four_heads(dtype, vector, layout)
    kept = x.clone()
    others = torch.cat([x[..., :off], x[..., off + dim:]], -1)
    out = torch.full_like(x, float("nan"))                                    # copied along
    call = lambda: binding.mla_rope(rope, x, pos, out, rot_offset=off)  # noqa: E731
    assert [name in k.name for k in launches_of(call)] == [True]
    call()
    _assert_rotated(out[..., off:off + dim], x[..., off:off + dim], pos, _freqs(dim), 1.0, layout)
    assert torch.equal(torch.cat([out[..., :off], out[..., off + dim:]], -1), others) and torch.equal(x, kept)
    if D > dim:                                                               # split
        rot = torch.full((T, H, dim), float("nan"), dtype=dtype, device=DEV)
        rest = torch.full((T, H, D - dim), float("nan"), dtype=dtype, device=DEV)
        call = lambda: binding.mla_rope(rope, x, pos, rot, rest=rest, rot_offset=off)  # noqa: E731
        assert [name in k.name for k in launches_of(call)] == [True]
        call()
        assert torch.equal(rot, out[..., off:off + dim]) and torch.equal(rest, others)
    binding.mla_rope(rope, x, pos, rot_offset=off)                            # in place
    assert torch.equal(x, out)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_of_many_rows_in_place_takes_four_heads(layout):
    x = torch.randn(1301, 128, 192, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    pos = _positions(1301, "near", torch.Generator().manual_seed(2))
    call = lambda: binding.mla_rope(binding.Rope(64, layout=layout), x, pos, rot_offset=128)  # noqa: E731
    assert [_four_heads(torch.bfloat16, True, layout) in k.name for k in launches_of(call)] == [True]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_of_many_rows_strides(layout):
    """Columns of wider rows, heads outside tokens, one head for all, outputs of odd strides: the
    contiguous call's bits, and nothing around them touched."""
    T, g = 2601, torch.Generator().manual_seed(5)
    rope, pos = binding.Rope(64, layout=layout), _positions(T, "near", g)
    wide = torch.randn(T, 16 * 192 + 24, generator=g).bfloat16().to(DEV)
    x = wide[:, 24:].unflatten(1, (16, 192))
    ref = torch.empty(T, 16, 192, dtype=torch.bfloat16, device=DEV)
    binding.mla_rope(rope, x.contiguous(), pos, ref, rot_offset=128)
    heads_outside = torch.empty(16, T, 192, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    odd = torch.full((T * 16 * 193 + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    odd_out = odd[1:].view(T, 16, 193)[:, :, :192]
    for view in (x, x.transpose(0, 1).contiguous().transpose(0, 1)):
        for out, vector in ((heads_outside, True), (odd_out, False)):
            call = lambda: binding.mla_rope(rope, view, pos, out, rot_offset=128)  # noqa: E731
            assert [_four_heads(torch.bfloat16, vector, layout) in k.name for k in launches_of(call)] == [True]
            call()
            assert torch.equal(out, ref)
            out.zero_()
    assert (odd[1:].view(T, 16, 193)[:, :, 192] == 7.0).all() and odd[0] == 7.0
    out = torch.empty_like(ref)
    binding.mla_rope(rope, x[:, :1].expand(T, 16, 192), pos, out, rot_offset=128)
    assert torch.equal(out, ref[:, :1].expand(T, 16, 192))
    inside = wide.clone()
    binding.mla_rope(rope, inside[:, 24:].unflatten(1, (16, 192)), pos, rot_offset=128)
    assert torch.equal(inside[:, 24:].unflatten(1, (16, 192)), ref) and torch.equal(inside[:, :24], wide[:, :24])


@pytest.mark.parametrize("layout,units", [("interleaved", 8 + 16), ("half", 4 + 16)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
def test_rope_append_of_many_queries(layout, units, kind):
    """300 tokens with their queries, four heads a thread (the grid shows it: one thread a unit and
    four heads): queries against the formula, pools the bits of mla_rope and mla_append_kv."""
    n, heads = 300, 128
    c_kv, k_r, pos, slots, q = _tokens(n, 77)
    rope = binding.Rope(64, layout=layout)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = _cache(kind), _cache(kind)
    k = torch.empty(n, 1, 64, dtype=torch.bfloat16, device=DEV)
    binding.mla_rope(rope, k_r.unsqueeze(1), pos, k)
    binding.mla_append_kv(c_kv.contiguous(), k[:, 0].contiguous(), slots, dev_error=err, **a)
    if kind == "nvfp4":
        live = slots >= 0
        rows, sigma = _nvfp4_rows(c_kv[live])
        a["kv_pool"].view(-1, binding.NVFP4_ROW)[slots[live].long()] = rows
        a["kv_scale"].view(-1)[slots[live].long()] = sigma
    q_c = torch.full((n, heads, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    q_r = torch.full((n, heads, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    call = lambda: binding.mla_rope_append_kv(rope, c_kv, k_r, pos, slots, dev_error=err, q=q, q_c=q_c, q_r=q_r,  # noqa: E731
                                              **b)
    lanes = 256 // units
    blocks = (n + 7) // 8 + (n * heads // 4 + lanes - 1) // lanes
    assert [x.grid for x in launches_of(call)] == [(blocks, 1, 1)]
    call()
    assert binding.mla_read_device_error(err) == 0
    _assert_rotated(q_r, q[..., 128:], pos, _freqs(64), 1.0, layout)
    assert torch.equal(q_c, q[..., :128])
    for name in a:
        assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name

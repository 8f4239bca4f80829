"""GPU parity of the products with 4-bit weights (mla_linear_w4, and as the decode step's absorb and
value projection) against the formula in 64 bits.

Tolerance, counted: the weights' values have at most 13 significant bits and x has 8, so that each
product is exact in fp32.  An output is the sum of chains of at most k / 16 additions of tensor-core
or fp32 partial sums and 16 more to join them and to apply the scales, each off by at most 2^-22 of
the partial sum (the tensor core may truncate), so by at most 2^-22 (k / 16 + 16) sum |x| |W|; then
half a bf16 step, 2^-8 of the value.  Over all outputs the partial sums are no larger than the
outputs in the mean (terms of random sign), which bounds the relative L2 error by
2^-8 + 2^-22 (k / 16 + 16).
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from parity_util import SCALE, TOL_BF16, assert_close  # noqa: E402

from mla_latent_kv_absorb_gb300 import binding, synth  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _weight(heads, n, k, fmt, group, zero, seed, change=None):
    """(W4Weight, its values in 64 bits [heads, n, k])."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (heads, n, k // 2), generator=g, dtype=torch.uint8)
    both = torch.stack([codes & 15, codes >> 4], -1).view(heads, n, k // group, group)
    z = None
    if fmt == "int4":
        scale = (torch.randn(heads, n, k // group, generator=g) * 2 / k ** 0.5).bfloat16()
        scale[0, 0, 0] = 0.0
        if change is not None:
            change(scale)
        if zero:
            z = torch.randint(0, 16, (heads, n, k // group), generator=g, dtype=torch.uint8)
        value = (both.double() - (8.0 if z is None else z.double()[..., None])) * scale.double()[..., None]
        t = 1.0
    else:
        scale = torch.randint(0, 0x7F, (heads, n, k // group), generator=g, dtype=torch.uint8)  # subnormals and 0 too
        scale |= torch.randint(0, 2, scale.shape, generator=g, dtype=torch.uint8) << 7
        value = E2M1[both.long()] * scale.view(torch.float8_e4m3fn).double()[..., None]
        t = 0.75 / 256
    w = binding.W4Weight(codes.to(DEV), scale.to(DEV), zero=None if z is None else z.to(DEV), group=group, tensor_scale=t)
    return w, (value.view(heads, n, k) * t).to(DEV)


def _assert_product(out, x, value):
    """out [rows, heads, n] against x [rows, heads, k] and value [heads, n, k]."""
    x = x.double()
    ref = torch.einsum("rhk,hnk->rhn", x, value)
    size = torch.einsum("rhk,hnk->rhn", x.abs(), value.abs())
    chain = 2.0 ** -22 * (x.shape[-1] / 16 + 16)
    far = (out.double() - ref).abs()
    tol = chain * size
    bad = far > tol + 2.0 ** -8 * (ref.abs() + tol) + 1e-38
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} past the tolerance, first at {bad.nonzero()[0].tolist()}"
    norm = float(ref.norm())
    assert norm == 0 or float(far.norm()) / norm <= 2.0 ** -8 + chain


FORMATS = [("int4", 32, False), ("int4", 64, True), ("int4", 128, True), ("int4", 128, False), ("nvfp4", 16, False)]


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130])
def test_linear_rows(fmt, group, zero, rows):
    w, value = _weight(1, 200, 640, fmt, group, zero, rows)
    x = torch.randn(rows, 640, generator=torch.Generator().manual_seed(rows)).bfloat16().to(DEV)
    out = torch.full((rows, 200), float("nan"), dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out[:, None], x[:, None], value)


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("heads,n,k", [(1, 1, 128), (1, 16, 16384), (3, 15, 256), (1, 17, 384), (2, 129, 1152),
                                       (1, 1000, 128), (1, 4099, 2048), (5, 64, 4224)])
def test_linear_sizes(fmt, group, zero, heads, n, k):
    for rows in (1, 11):
        w, value = _weight(heads, n, k, fmt, group, zero, n + k)
        x = torch.randn(rows, heads, k, generator=torch.Generator().manual_seed(k)).bfloat16().to(DEV)
        out = torch.full((rows, heads, n), float("nan"), dtype=torch.bfloat16, device=DEV)
        binding.mla_linear_w4(x, w, out)
        _assert_product(out, x, value)


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("heads,n,k,rows", [
    (1, 20000, 512, 17),
    (1, 8200, 1312, 33),      # k ends inside a step, two thread blocks of a cluster
    (1, 8192, 2560, 64),      # clusters of four
    (5, 1400, 2048, 65),      # heads, a second block of rows with one row
    (1, 20100, 640, 130),
])
def test_linear_many_rows(fmt, group, zero, heads, n, k, rows):
    """More rows and outputs than the cases above: all warps of a thread block over the outputs."""
    k -= k % max(group, 32)
    w, value = _weight(heads, n, k, fmt, group, zero, n + rows)
    x = torch.randn(rows, heads, k, generator=torch.Generator().manual_seed(rows)).bfloat16().to(DEV)
    out = torch.full((rows, heads, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out, x, value)


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("heads,n,k,rows", [
    (1, 16500, 2112, 57),     # outputs and k end inside a tile and a step, an odd number of steps
    (1, 8200, 4096, 64),      # clusters of four, four of 256 outputs are there
    (1, 4096, 4096, 192),     # two warps over k in the packed layout, three blocks of rows
    (1, 2048, 8192, 250),     # four warps over k
    (128, 512, 128, 30),      # two pairs of tiles in turn, one step each
    (64, 384, 192, 60),       # half a pair
    (3, 3000, 1024, 100),
    (1, 40000, 64, 64),       # less than a step
    (1, 65000, 320, 49),
])
def test_linear_rows_in_tensor_memory(fmt, group, zero, heads, n, k, rows):
    """Sizes where the rows are the columns of tensor memory."""
    k = max(k - k % max(group, 32), group)
    w, value = _weight(heads, n, k, fmt, group, zero, n + rows)
    x = torch.randn(rows, heads, k, generator=torch.Generator().manual_seed(rows)).bfloat16().to(DEV)
    out = torch.full((rows, heads, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out, x, value)


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("rows", [41, 48, 49, 64, 90])
def test_linear_many_rows_of_few_outputs(fmt, group, zero, rows):
    """Four warps over k: x of so many rows is more than a thread block's shared memory holds."""
    w, value = _weight(1, 576, 8192, fmt, group, zero, rows)
    x = torch.randn(rows, 1, 8192, generator=torch.Generator().manual_seed(rows)).bfloat16().to(DEV)
    out = torch.full((rows, 1, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out, x, value)


def test_many_rows_in_a_chain_in_graphs_and_on_streams():
    """The step's two products for 40 rows, one reading what the other wrote: in one stream, captured and
    replayed, and on three streams at once, the same bits as calls waited for one by one."""
    uk, _ = _weight(128, 512, 128, "int4", 32, False, 31)
    uv, _ = _weight(128, 128, 512, "nvfp4", 16, False, 32)
    for w in (uk, uv):
        w.struct.tensor_scale *= 0.02
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 128, 128, generator=g).bfloat16().to(DEV)

    def buffers():
        return torch.empty(40, 128, 512, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)

    def chain(first, bufs, stream=None, wait=False):
        q, (lat, back) = first, bufs
        for _ in range(3):
            for fn, a, w, b in ((binding.mla_absorb_q_w4, q, uk, lat), (binding.mla_out_proj_w4, lat, uv, back)):
                fn(a, w, b, stream)
                if wait:
                    torch.cuda.synchronize()
            q = back
        return back

    want = chain(x, buffers(), wait=True).clone()
    assert want.isfinite().all()
    assert torch.equal(chain(x, buffers()), want)
    torch.cuda.synchronize()
    streams, sets = [torch.cuda.Stream() for _ in range(3)], [buffers() for _ in range(3)]
    torch.cuda.synchronize()
    for s, b in zip(streams, sets):
        chain(x, b, s)
    torch.cuda.synchronize()
    assert all(torch.equal(b[1], want) for b in sets)
    static, bufs, graph = torch.zeros_like(x), buffers(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(static, bufs)
    static.copy_(x)
    for _ in range(2):
        graph.replay()
    assert torch.equal(bufs[1], want)


@pytest.mark.parametrize("rows", [40, 60])
def test_linear_many_rows_strides(rows):
    """Rows of a wider tensor, one row for all heads, odd strides of the outputs, not-finite rows."""
    w, value = _weight(6, 1400, 2048, "int4", 64, True, 5)
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(rows, 6 * 2048 + 8, generator=g).bfloat16().to(DEV)
    x = wide[:, 8:].unflatten(1, (6, 2048))
    want = torch.empty(rows, 6, 1400, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x.contiguous(), w, want)
    _assert_product(want, x, value)
    buf = torch.full((rows * 6 * 1401 + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[1:].view(rows, 6, 1401)[:, :, :1400]
    binding.mla_linear_w4(x, w, out)
    assert torch.equal(out, want) and (buf[1:].view(rows, 6, 1401)[:, :, 1400] == 7.0).all() and buf[0] == 7.0
    swapped = torch.empty(6, rows, 1400, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x.transpose(0, 1).contiguous().transpose(0, 1), w, swapped.transpose(0, 1))
    assert torch.equal(swapped.transpose(0, 1), want)
    out = torch.empty_like(want)
    shared = x[:, :1].expand(rows, 6, 2048)
    binding.mla_linear_w4(shared, w, out)
    _assert_product(out, shared, value)
    binding.mla_linear_w4(x[:1].expand(rows, 6, 2048), w, out)     # one row for all: every row the same bits
    assert torch.equal(out, out[:1].expand(rows, 6, 1400))
    _assert_product(out, x[:1].expand(rows, 6, 2048), value)
    y = x.clone()
    y[3, 2, 100], y[rows - 1, 5, 2047] = float("nan"), float("inf")
    binding.mla_linear_w4(y, w, out)
    keep = torch.ones(rows, 6, dtype=torch.bool, device=DEV)
    keep[3, 2], keep[rows - 1, 5] = False, False
    assert torch.equal(out[keep], want[keep]) and out[3, 2].isnan().all() and not out[rows - 1, 5].isfinite().all()


@pytest.mark.parametrize("k", [32, 64, 96, 160, 2016])
def test_linear_groups_of_32_at_any_multiple(k):
    w, value = _weight(1, 40, k, "int4", 32, True, k)
    x = torch.randn(5, 1, k, generator=torch.Generator().manual_seed(k)).bfloat16().to(DEV)
    out = torch.empty(5, 1, 40, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out, x, value)


def test_nvfp4_k_of_32():
    w, value = _weight(2, 40, 32, "nvfp4", 16, False, 3)
    x = torch.randn(3, 2, 32, generator=torch.Generator().manual_seed(4)).bfloat16().to(DEV)
    out = torch.empty(3, 2, 40, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out, x, value)


@pytest.mark.parametrize("rows", [1, 16, 130])
@pytest.mark.parametrize("fmt,group,zero", FORMATS)
def test_step_products(rows, fmt, group, zero):
    g = torch.Generator().manual_seed(rows)
    for fn, n, k in ((binding.mla_absorb_q_w4, 512, 128), (binding.mla_out_proj_w4, 128, 512)):
        w, value = _weight(128, n, k, fmt, group, zero, n)
        x = torch.randn(rows, 128, k, generator=g).bfloat16().to(DEV)
        out = torch.full((rows, 128, n), float("nan"), dtype=torch.bfloat16, device=DEV)
        fn(x, w, out)
        _assert_product(out, x, value)
        again = torch.empty_like(out)
        binding.mla_linear_w4(x, w, again)
        assert torch.equal(again, out)


@pytest.mark.parametrize("rows", [3, 40])
def test_linear_strides(rows):
    """Columns of wider rows, one row for all heads, outputs with odd strides: the contiguous call's
    bits, and nothing around them touched."""
    w, value = _weight(4, 100, 256, "int4", 64, True, 5)
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(rows, 4 * 256 + 8, generator=g).bfloat16().to(DEV)
    x = wide[:, 8:].unflatten(1, (4, 256))
    want = torch.empty(rows, 4, 100, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x.contiguous(), w, want)
    _assert_product(want, x, value)
    buf = torch.full((rows * 4 * 101 + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[1:].view(rows, 4, 101)[:, :, :100]
    binding.mla_linear_w4(x, w, out)
    assert torch.equal(out, want) and (buf[1:].view(rows, 4, 101)[:, :, 100] == 7.0).all() and buf[0] == 7.0
    swapped = torch.empty(4, rows, 100, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, swapped.transpose(0, 1))
    assert torch.equal(swapped.transpose(0, 1), want)
    shared = x[:, :1].expand(rows, 4, 256)
    out = torch.empty_like(want)
    binding.mla_linear_w4(shared, w, out)
    _assert_product(out, shared, value)
    same_row = x[:1].expand(rows, 4, 256)
    binding.mla_linear_w4(same_row, w, out)
    assert torch.equal(out, want[:1].expand(rows, 4, 100))


def test_linear_special_values():
    """Zeros give zeros, a NaN or an infinity in one row of x stays in that row, infinite scales (int4)
    reach the outputs of their own column only."""
    w, _ = _weight(1, 50, 256, "int4", 64, False, 9)
    x = torch.randn(12, 256, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    clean = torch.empty(12, 50, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, clean)
    y = x.clone()
    y[3, 100], y[9, 7] = float("nan"), float("inf")
    out = torch.empty_like(clean)
    binding.mla_linear_w4(y, w, out)
    keep = [r for r in range(12) if r not in (3, 9)]
    assert torch.equal(out[keep], clean[keep]) and out[3].isnan().all() and not out[9].isfinite().all()
    binding.mla_linear_w4(torch.zeros_like(x), w, out)
    assert (out == 0).all()

    def infinite(scale):
        scale[0, 20, 1] = float("inf")

    w, _ = _weight(1, 50, 256, "int4", 64, False, 9, infinite)
    binding.mla_linear_w4(x, w, out)
    keep = [c for c in range(50) if c != 20]
    assert torch.equal(out[:, keep], clean[:, keep]) and not out[:, 20].isfinite().any()


def test_linear_is_repeatable_and_runs_on_any_stream():
    w, value = _weight(1, 2048, 4096, "int4", 128, True, 12)
    x = torch.randn(4, 1, 4096, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    out = torch.empty(4, 1, 2048, dtype=torch.bfloat16, device=DEV)
    binding.mla_linear_w4(x, w, out)
    _assert_product(out, x, value)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [torch.empty_like(out) for _ in streams]
    for s, o in zip(streams, outs):   # at once on three streams
        for _ in range(5):
            binding.mla_linear_w4(x, w, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(x)
    mid = torch.empty_like(out)
    with torch.cuda.graph(graph):   # its output is the next call's input
        binding.mla_linear_w4(static, w, mid)
        binding.mla_linear_w4(static, w, out)
    static.copy_(x)
    graph.replay()
    assert torch.equal(mid, outs[0]) and torch.equal(out, outs[0])


def test_linear_chain_sees_the_previous_call():
    """A product of a product, many times over in one stream: each call reads what the one before it
    wrote."""
    w, value = _weight(1, 256, 256, "int4", 32, False, 21)
    x = torch.randn(2, 1, 256, generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    bufs = [x.clone(), torch.empty_like(x)]
    want = x
    for _ in range(6):
        out = torch.empty_like(x)
        binding.mla_linear_w4(want, w, out)
        torch.cuda.synchronize()
        want = out
    for i in range(6):
        binding.mla_linear_w4(bufs[i % 2], w, bufs[(i + 1) % 2])
    assert torch.equal(bufs[0], want)


def test_linear_empty_and_refusals():
    w, _ = _weight(1, 50, 256, "int4", 64, False, 9)
    binding.mla_linear_w4(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV), w,
                          torch.empty(0, 50, dtype=torch.bfloat16, device=DEV))
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(4, 50, dtype=torch.bfloat16, device=DEV)
    for bad_x, bad_out in ((x[:, :128], out), (x, out[:, :49]), (x[:3], out), (x.t().contiguous().t(), out),
                           (x.cpu(), out), (x, out.cpu())):
        with pytest.raises(ValueError):
            binding.mla_linear_w4(bad_x, w, bad_out)
    for bad_x, bad_out in ((x.float(), out), (x, out.half())):
        with pytest.raises(TypeError):
            binding.mla_linear_w4(bad_x, w, bad_out)
    with pytest.raises(binding.MlaError):
        binding.mla_linear_w4(x, w, out[:1].expand(4, 50))
    with pytest.raises(ValueError):
        binding.mla_absorb_q_w4(torch.zeros(1, 128, 128, dtype=torch.bfloat16, device=DEV), w,
                                torch.zeros(1, 128, 512, dtype=torch.bfloat16, device=DEV))
    codes = torch.zeros(2, 3, 32, dtype=torch.uint8, device=DEV)
    ones = torch.ones(2, 3, 2, dtype=torch.bfloat16, device=DEV)
    for args, kw in (((codes.cpu(), ones), {}), ((codes, ones.cpu()), {}), ((codes[:, :, ::2], ones[:, :, :1]), {}),
                     ((codes, ones[:, :2]), {}), ((codes, ones), dict(zero=codes[:, :, :2]))):
        with pytest.raises(ValueError):
            binding.W4Weight(*args, **kw)
    with pytest.raises(TypeError):
        binding.W4Weight(codes.int(), ones)


def _attention(inp, q_c, q_r, k_val, v_val):
    """The step in 64 bits: out [rows, 128, 128] for one query row per sequence."""
    outs = []
    pool = inp.pool.double().reshape(-1, 576).to(DEV)
    for b, S in enumerate(inp.seq_lens):
        idx = torch.tensor([int(inp.block_table[b, p // 64]) * 64 + p % 64 for p in range(int(S))], device=DEV)
        c, kr = pool[idx, :512], pool[idx, 512:]
        q_lat = torch.einsum("hd,hcd->hc", q_c[b].double(), k_val)
        p = ((q_lat @ c.t() + q_r[b].double() @ kr.t()) * SCALE).softmax(-1)
        outs.append(torch.einsum("hc,hdc->hd", p @ c, v_val))
    return torch.stack(outs)


@pytest.mark.parametrize("fmt,group,zero", FORMATS[:1] + FORMATS[2:3] + FORMATS[4:])
def test_step_with_4_bit_weights(fmt, group, zero):
    inp = synth.make_inputs([300, 1, 700], seed=71)
    q_c, q_r, w_uk, w_uv, kv, bt = binding.inputs_to_device(inp, DEV)
    uk, k_val = _weight(128, 512, 128, fmt, group, zero, 1)
    uv, v_val = _weight(128, 128, 512, fmt, group, zero, 2)
    # absolute bounds of the step's tolerance are for outputs of about 1: weights of unit rows
    for w, v in ((uk, k_val), (uv, v_val)):
        s = 1.0 / float(v.square().sum(-1).mean().sqrt()) * (0.5 if w is uk else 1.0)
        w.struct.tensor_scale = s * w.tensor_scale   # a float of the struct, read at each call
        v *= w.struct.tensor_scale / w.tensor_scale
    step = binding.DecodeStep(inp.seq_lens, w_uk=uk, w_uv=uv, block_table=bt, min_pages_per_split=2, **kv)
    out = step.run(q_c, q_r).clone()
    assert step.device_error() == 0
    assert_close(out, _attention(inp, q_c, q_r, k_val, v_val), TOL_BF16, "out")
    graph = step.capture(q_c, q_r)
    step.out.zero_()
    graph.replay()
    assert torch.equal(step.out, out)
    if step.graph_kernel_nodes is not None:
        assert step.graph_kernel_nodes == step.launches_per_step
    # one product in 4 bits, the other in bf16
    mixed = binding.DecodeStep(inp.seq_lens, w_uk=uk, w_uv=w_uv, block_table=bt, fused_tail=True, **kv)
    got = mixed.run(q_c, q_r)
    assert_close(got, _attention(inp, q_c, q_r, k_val, w_uv.double()), TOL_BF16, "out (bf16 projection)")


def test_step_with_4_bit_weights_and_many_sequences():
    """48 sequences: the step's kernels one behind the other against calls waited for one by one."""
    lens = [1 + (37 * i) % 300 for i in range(48)]
    inp = synth.make_inputs(lens, seed=73)
    q_c, q_r, _, _, kv, bt = binding.inputs_to_device(inp, DEV)
    uk, _ = _weight(128, 512, 128, "int4", 128, True, 3)
    uv, _ = _weight(128, 128, 512, "int4", 64, False, 4)
    uk.struct.tensor_scale *= 0.05
    step = binding.DecodeStep(inp.seq_lens, w_uk=uk, w_uv=uv, block_table=bt, **kv)
    out = step.run(q_c, q_r).clone()
    assert step.device_error() == 0
    q_abs, proj = torch.empty_like(step.q_abs), torch.empty_like(out)
    binding.mla_absorb_q_w4(q_c, uk, q_abs)
    torch.cuda.synchronize()
    assert torch.equal(q_abs, step.q_abs)
    binding.mla_out_proj_w4(step.o_lat, uv, proj)
    assert torch.equal(proj, out) and out.isfinite().all()
    graph = step.capture(q_c, q_r)
    for _ in range(3):
        step.out.zero_()
        graph.replay()
        assert torch.equal(step.out, out)


def test_4_bit_step_refusals():
    inp = synth.make_inputs([300], seed=72)
    q_c, q_r, w_uk, w_uv, kv, bt = binding.inputs_to_device(inp, DEV)
    uk, _ = _weight(128, 512, 128, "int4", 32, False, 1)
    uv, _ = _weight(128, 128, 512, "int4", 32, False, 2)
    for kw in (dict(w_uk=uk, w_uv=w_uv, fused_absorb=True), dict(w_uk=w_uk, w_uv=uv, fused_tail=True)):
        with pytest.raises(ValueError):
            binding.DecodeStep(inp.seq_lens, block_table=bt, **kv, **kw)
    step = binding.DecodeStep(inp.seq_lens, w_uk=uk, w_uv=uv, block_table=bt, **kv)
    with pytest.raises(ValueError):
        step.run_host(inp.q_c, inp.q_r)
    with pytest.raises(ValueError):
        binding.prefill_chunk(300, torch.zeros(260, 128, 128, dtype=torch.bfloat16, device=DEV),
                              torch.zeros(260, 128, 64, dtype=torch.bfloat16, device=DEV), w_uk=uk, w_uv=uv,
                              kv_pool=kv["kv_pool"], block_table_row=bt[0])
    out, err = binding.prefill_chunk(300, q_c, q_r, w_uk=uk, w_uv=uv, kv_pool=kv["kv_pool"], block_table_row=bt[0])
    assert torch.equal(out, step.run(q_c, q_r))

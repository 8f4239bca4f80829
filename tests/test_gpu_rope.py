"""GPU parity of the rotary positions (mla_rope) and of the append that applies them on the way
(mla_rope_append_kv) against the formulas in 64 bits.

Tolerance of one rotated element, y = m (x0 cos a -+ x1 sin a), counted from the roundings of the
path: the angle's rest r, at most a quarter of a half turn, in fp32 and in radians (r (2 * 6.0e-8 +
2.8e-8) < 1.2e-7 rad, against sines and cosines that are 0.71 where r is that large: 8.3e-8), sine
and cosine (series 2e-9, one ulp and a part: 7e-8), m and its product (2 * 6.0e-8), two products and
their sum (2 * 6.0e-8 against |x0| + |x1|): less than 4e-7 m (|x0| + |x1|); the frequency's own
roundings (pow, 1 / 2 pi, their quotient: 2^-51 of the angle, for the kernel and the
reference together); then the output type's half step.  Copied elements are equal.
"""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from mla_latent_kv_absorb_gb300 import binding, synth  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _freqs(dim, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / dim) for i in range(dim // 2)], dtype=torch.float64)


def _reference(x, positions, freq, m, layout):
    """(rotated rows in 64 bits, their tolerance) of x [T, H, dim]."""
    x = x.double()
    d = x.shape[-1]
    angle = positions.double()[:, None, None] * freq.to(x.device)
    c, s = angle.cos() * m, angle.sin() * m
    a, b = (x[..., : d // 2], x[..., d // 2:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    y0, y1 = a * c - b * s, a * s + b * c
    tol = m * (a.abs() + b.abs()) * (4e-7 + angle.abs() * 2.0 ** -51)
    if layout == "half":
        return torch.cat([y0, y1], -1), torch.cat([tol, tol], -1)
    return torch.stack([y0, y1], -1).flatten(-2), torch.stack([tol, tol], -1).flatten(-2)


def _assert_rotated(got, x, positions, freq, m, layout):
    ref, tol = _reference(x, positions, freq, m, layout)
    tol = tol + HALF_STEP[got.dtype] * (ref.abs() + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} past the tolerance, first at {bad.nonzero()[0].tolist()}"


def _positions(T, kind, g):
    if kind == "far":
        p = torch.randint(-(2 ** 31), 2 ** 31 - 1, (T,), generator=g, dtype=torch.int64)
        p[:1] = 2 ** 31 - 1
        p[-1:] = -(2 ** 31) if T > 1 else p[-1:]
        return p.to(torch.int32).to(DEV)
    p = torch.randint(-100, 200000, (T,), generator=g, dtype=torch.int32)
    p[0] = 0
    return p.to(DEV)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D,dim,off,kind", [
    (1, 128, 192, 64, 128, "near"),       # one token's query
    (3, 5, 192, 64, 128, "far"),          # heads not in fours
    (700, 16, 128, 32, 0, "near"),        # rotated part first
    (33, 128, 192, 64, 64, "near"),       # rotated part in the middle
    (2500, 1, 64, 64, 0, "far"),          # one head, all of it rotated
    (7, 3, 2, 2, 0, "near"),              # the smallest head
    (5, 4, 77, 26, 13, "near"),           # no 16-byte pieces
    (2, 8, 600, 256, 300, "near"),        # the widest rotation, more pieces than threads without vectors
    (4097, 4, 72, 64, 8, "near"),
])
def test_rope_matches_formula(layout, dtype, T, H, D, dim, off, kind):
    g = torch.Generator().manual_seed(T * 31 + D)
    x = torch.randn(T, H, D, generator=g).to(dtype).to(DEV)
    pos = _positions(T, kind, g)
    rope = binding.Rope(dim, layout=layout)
    kept = x.clone()
    others = torch.cat([x[..., :off], x[..., off + dim:]], -1)
    # copied along
    out = torch.full_like(x, float("nan"))
    assert binding.mla_rope(rope, x, pos, out, rot_offset=off) is out
    _assert_rotated(out[..., off:off + dim], x[..., off:off + dim], pos, _freqs(dim), 1.0, layout)
    assert torch.equal(torch.cat([out[..., :off], out[..., off + dim:]], -1), others)
    assert torch.equal(x, kept)
    # split
    if D > dim:
        rot = torch.full((T, H, dim), float("nan"), dtype=dtype, device=DEV)
        rest = torch.full((T, H, D - dim), float("nan"), dtype=dtype, device=DEV)
        binding.mla_rope(rope, x, pos, rot, rest=rest, rot_offset=off)
        assert torch.equal(rot, out[..., off:off + dim]) and torch.equal(rest, others)
    # in place
    assert binding.mla_rope(rope, x, pos, rot_offset=off) is x
    assert torch.equal(x, out)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_strides(layout):
    """Columns of wider rows, tokens inside heads, one head row expanded over the heads, a base that is
    not 16-byte aligned: each equals the contiguous call's bits, and nothing around it is touched."""
    g = torch.Generator().manual_seed(5)
    rope = binding.Rope(64, layout=layout)
    pos = _positions(37, "near", g)
    wide = torch.randn(37, 8 * 192 + 24, generator=g).bfloat16().to(DEV)
    x = wide[:, 24:].unflatten(1, (8, 192))
    ref = torch.empty(37, 8, 192, dtype=torch.bfloat16, device=DEV)
    binding.mla_rope(rope, x.contiguous(), pos, ref, rot_offset=128)
    for view in (x, x.transpose(0, 1).contiguous().transpose(0, 1)):
        out = torch.empty_like(ref)
        binding.mla_rope(rope, view, pos, out, rot_offset=128)
        assert torch.equal(out, ref)
    odd = torch.full((37 * 8 * 193 + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = odd[1:].view(37, 8, 193)[:, :, :192]                  # 2-byte aligned, odd strides
    binding.mla_rope(rope, x, pos, out, rot_offset=128)
    assert torch.equal(out, ref) and (odd[1:].view(37, 8, 193)[:, :, 192] == 7.0).all() and odd[0] == 7.0
    heads_outside = torch.empty(8, 37, 192, dtype=torch.bfloat16, device=DEV)
    binding.mla_rope(rope, x, pos, heads_outside.transpose(0, 1), rot_offset=128)
    assert torch.equal(heads_outside.transpose(0, 1), ref)
    one = x[:, :1].expand(37, 8, 192)
    out = torch.empty_like(ref)
    binding.mla_rope(rope, one, pos, out, rot_offset=128)
    assert torch.equal(out, ref[:, :1].expand(37, 8, 192))
    inside = wide.clone()
    binding.mla_rope(rope, inside[:, 24:].unflatten(1, (8, 192)), pos, rot_offset=128)   # in place in a wider row
    assert torch.equal(inside[:, 24:].unflatten(1, (8, 192)), ref) and torch.equal(inside[:, :24], wide[:, :24])


@pytest.mark.parametrize("kw,freq,m", [
    (dict(scaling="linear", factor=8.0), _freqs(64) / 8, 1.0),
    (dict(inv_freq=[0.5 ** i for i in range(32)], magnitude=1.25), torch.tensor([0.5 ** i for i in range(32)]).double(), 1.25),
    (dict(base=500000.0), _freqs(64, 500000.0), 1.0)])
def test_rope_scalings(kw, freq, m):
    g = torch.Generator().manual_seed(8)
    x = torch.randn(50, 4, 64, generator=g).to(DEV)
    pos = _positions(50, "near", g)
    out = torch.empty_like(x)
    binding.mla_rope(binding.Rope(64, **kw), x, pos, out)
    _assert_rotated(out, x, pos, freq, m, "interleaved")


def test_rope_yarn_follows_its_constants():
    """The rows of a YaRN rotation turn by the struct's own steps (which the host test holds to the
    formula) and have its magnitude."""
    rope = binding.Rope(64, scaling="yarn", factor=40.0, original_len=4096, layout="half")
    steps = torch.tensor([int(v) / 2.0 ** 64 for v in rope.config.step[:32]], dtype=torch.float64)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(300, 128, 64, generator=g).bfloat16().to(DEV)
    pos = _positions(300, "near", g)
    out = torch.empty_like(x)
    binding.mla_rope(rope, x, pos, out)
    _assert_rotated(out, x, pos, steps * 2 * np.pi, rope.magnitude, "half")


def test_rope_backwards_is_the_gradient():
    """Negative positions give the transposed map, which is the rotation's gradient: against central
    differences of sum(w * rope(x)) in fp32.  The map is linear, so a difference over a step of 1 has
    no error but rounding: 2 y's of |y| <= |x0| + |x1| + 2 with 6e-7 each, against w of about 1."""
    rope = binding.Rope(64, layout="interleaved")
    g = torch.Generator().manual_seed(10)
    x = torch.randn(6, 2, 64, generator=g).to(DEV)
    w = torch.randn(6, 2, 64, generator=g).to(DEV)
    pos = torch.tensor([0, 1, 17, 4095, 100000, 2 ** 30], dtype=torch.int32, device=DEV)
    grad = torch.empty_like(w)
    binding.mla_rope(rope, w, -pos, grad)
    for i in range(64):
        y = []
        for step in (0.5, -0.5):
            xs = x.clone()
            xs[..., i] += step
            out = torch.empty_like(xs)
            binding.mla_rope(rope, xs, pos, out)
            y.append((out.double() * w.double()).sum(-1))
        scale = (x.abs().double().amax() + 2) * 2 * w.abs().double().sum(-1) * 6e-7 * 2
        assert ((y[0] - y[1] - grad[..., i].double()).abs() <= scale).all()


def test_rope_nan_and_infinity_stay_in_their_pair():
    rope = binding.Rope(64)
    x = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    x[0, 1, 6], x[0, 2, 9] = float("nan"), float("inf")
    out = torch.empty_like(x)
    binding.mla_rope(rope, x, torch.tensor([3], dtype=torch.int32, device=DEV), out)
    fine = torch.ones(1, 4, 64, dtype=torch.bool, device=DEV)
    fine[0, 1, 6:8], fine[0, 2, 8:10] = False, False
    assert torch.isfinite(out)[fine].all() and not torch.isfinite(out)[~fine].any()


def test_rope_empty_and_refusals():
    rope = binding.Rope(64)
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    binding.mla_rope(rope, x, torch.empty(0, dtype=torch.int32, device=DEV))
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        binding.mla_rope(rope, x, pos.long())
    with pytest.raises(TypeError):
        binding.mla_rope(rope, x, pos, torch.empty(4, 4, 64, device=DEV))
    with pytest.raises(TypeError):
        binding.mla_rope(rope, x.double(), pos)
    with pytest.raises(ValueError):
        binding.mla_rope(rope, x, pos[:3])
    with pytest.raises(ValueError):
        binding.mla_rope(rope, x.transpose(1, 2), pos)
    with pytest.raises(ValueError):
        binding.mla_rope(rope, x.cpu(), pos)
    with pytest.raises(ValueError):
        binding.mla_rope(rope, x[..., ::2].expand(4, 4, 32), pos)
    with pytest.raises(binding.MlaError):
        binding.mla_rope(rope, x, pos, x[:1].expand(4, 4, 64))                # rows of out coincide
    with pytest.raises(binding.MlaError):
        binding.mla_rope(rope, x, pos, rot_offset=1)


# ---------------------------------------------------------------------------------- the append

PAGES = 8


def _cache(kind, pages=PAGES):
    g = torch.Generator().manual_seed(3)
    if kind == "bf16":
        return {"kv_pool": torch.randn(pages, 64, 576, generator=g).bfloat16().to(DEV)}
    width = 512 if kind == "fp8" else binding.NVFP4_ROW
    return {"kv_pool": torch.randint(0, 256, (pages, 64, width), generator=g, dtype=torch.uint8).to(DEV),
            "kv_scale": torch.rand(pages, 64, generator=g).to(DEV),
            "kr_pool": torch.randn(pages, 64, 64, generator=g).bfloat16().to(DEV)}


def _tokens(n, seed, pitch=576):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(n, pitch, generator=g) * torch.exp2(torch.empty(n, 1).uniform_(-12, 8, generator=g))
    rows = rows.bfloat16().to(DEV)[:, pitch - 576:]
    slots = torch.from_numpy(np.random.default_rng(seed).permutation(PAGES * 64)[:n].astype(np.int32))
    if n > 8:
        slots[5], slots[n - 2] = -1, -7
    pos = torch.randint(0, 200000, (n,), generator=g, dtype=torch.int32).to(DEV)
    q = torch.randn(n, 128, 192, generator=g).bfloat16().to(DEV)
    return rows[:, :512], rows[:, 512:], pos, slots.to(DEV), q


def _nvfp4_rows(c):
    """The NVFP4 rows and scales of latents c [n, 512] by the rule of the rotated append, in fp32 on the
    host: products with the reciprocals of 2688 and 6, the other quotients as they are."""
    c = c.float().cpu().numpy()
    top = np.abs(c).max(1)
    sigma = np.where(top > 0, top * (np.float32(1) / np.float32(2688)), np.float32(1)).astype(np.float32)
    blocks = c.reshape(-1, 32, 16)
    unit = (np.abs(blocks).max(2) / sigma[:, None]) * (np.float32(1) / np.float32(6))
    s8 = torch.from_numpy(unit).to(torch.float8_e4m3fn)
    den = sigma[:, None, None] * s8.float().numpy()[:, :, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(den == 0, blocks * np.float32(0), blocks / den)
    a = np.abs(v)
    code = np.zeros(v.shape, np.uint8)
    for border, even_above in ((.25, False), (.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if even_above else (a > border)   # a tie goes to the even code
    code = (code + 8 * np.signbit(v)).reshape(-1, 512).astype(np.uint8)
    rows = np.concatenate([code[:, 0::2] | code[:, 1::2] << 4, s8.view(torch.uint8).numpy()], 1)
    return torch.from_numpy(rows).to(DEV), torch.from_numpy(sigma).to(DEV)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("n,pitch,query", [(1, 576, True), (13, 2112, True), (300, 584, False), (65, 576, True)])
def test_rope_append_is_rope_then_append(layout, kind, n, pitch, query):
    """The pools (untouched slots too) and the queries equal, bit for bit, those of mla_rope and
    mla_append_kv one after the other, which have their own parity tests; an NVFP4 row has its own
    rule's bytes."""
    c_kv, k_r, pos, slots, q = _tokens(n, 40 + n, pitch)
    if n > 8:
        c_kv[3] = 0.0             # an all-zero row
        c_kv[4, 16:32] *= 1e-9    # a block whose scale rounds to zero
        c_kv[6, :16] = -0.0
    rope = binding.Rope(64, layout=layout, scaling="yarn", factor=8.0, original_len=4096)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, b = _cache(kind), _cache(kind)
    rot = torch.empty(n, 1, 64, dtype=torch.bfloat16, device=DEV)
    binding.mla_rope(rope, k_r.unsqueeze(1), pos, rot)
    binding.mla_append_kv(c_kv.contiguous(), rot[:, 0].contiguous(), slots, dev_error=err, **a)
    if kind == "nvfp4":
        live = slots >= 0
        rows, sigma = _nvfp4_rows(c_kv[live])
        a["kv_pool"].view(-1, binding.NVFP4_ROW)[slots[live].long()] = rows
        a["kv_scale"].view(-1)[slots[live].long()] = sigma
    outs = {}
    if query:
        outs = {"q": q, "q_c": torch.full((n, 128, 128), 9.0, dtype=torch.bfloat16, device=DEV),
                "q_r": torch.full((n, 128, 64), 9.0, dtype=torch.bfloat16, device=DEV)}
    binding.mla_rope_append_kv(rope, c_kv, k_r, pos, slots, dev_error=err, **b, **outs)
    assert binding.mla_read_device_error(err) == 0
    for name in a:
        assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name
    if query:
        q_r = torch.empty(n, 128, 64, dtype=torch.bfloat16, device=DEV)
        binding.mla_rope(rope, q[..., 128:], pos, q_r)
        assert torch.equal(outs["q_c"], q[..., :128]) and torch.equal(outs["q_r"], q_r)


def test_rope_append_slot_past_pool_is_reported_and_skipped():
    c_kv, k_r, pos, slots, q = _tokens(4, 7)
    slots = torch.tensor([3, PAGES * 64, 2 ** 31 - 1, -1], dtype=torch.int32, device=DEV)
    for kind in ("bf16", "fp8", "nvfp4"):
        cache, before = _cache(kind), _cache(kind)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        q_c = torch.empty(4, 128, 128, dtype=torch.bfloat16, device=DEV)
        q_r = torch.full((4, 128, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
        binding.mla_rope_append_kv(binding.Rope(), c_kv, k_r, pos, slots, dev_error=err, q=q, q_c=q_c, q_r=q_r, **cache)
        assert binding.mla_read_device_error(err) == 16  # MLA_DEVERR_BAD_SLOT, and nothing else
        assert torch.isfinite(q_r).all() and torch.equal(q_c, q[..., :128])
        for name in cache:
            same = (cache[name].view(torch.uint8) == before[name].view(torch.uint8)).flatten(2).all(-1) \
                if cache[name].dim() == 3 else cache[name] == before[name]
            assert not same[0, 3] and int(same.sum()) == PAGES * 64 - 1, name


def test_rope_append_query_strides():
    c_kv, k_r, pos, slots, q = _tokens(9, 11)
    rope, err = binding.Rope(layout="half"), torch.zeros(1, dtype=torch.int32, device=DEV)
    want = [torch.empty(9, 128, d, dtype=torch.bfloat16, device=DEV) for d in (128, 64)]
    binding.mla_rope_append_kv(rope, c_kv, k_r, pos, slots, dev_error=err, q=q, q_c=want[0], q_r=want[1], **_cache("bf16"))
    wide = torch.zeros(9, 128, 200, dtype=torch.bfloat16, device=DEV)
    wide[..., 8:] = q
    for view in (wide[..., 8:], q.transpose(0, 1).contiguous().transpose(0, 1)):
        got = [torch.empty_like(t) for t in want]
        binding.mla_rope_append_kv(rope, c_kv, k_r, pos, slots, dev_error=err, q=view, q_c=got[0], q_r=got[1],
                                   **_cache("bf16"))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(binding.MlaError) as e:   # a query row that does not start on 16 bytes
        binding.mla_rope_append_kv(rope, c_kv, k_r, pos, slots, dev_error=err, q=wide[..., 4:196], q_c=want[0],
                                   q_r=want[1], **_cache("bf16"))
    assert e.value.status == binding.MLA_ERR_ALIGNMENT
    with pytest.raises(ValueError):
        binding.mla_rope_append_kv(rope, c_kv, k_r, pos, slots, dev_error=err, q_c=want[0], **_cache("bf16"))
    with pytest.raises(ValueError):
        binding.mla_rope_append_kv(rope, c_kv, k_r, pos[:4], slots, dev_error=err, **_cache("bf16"))


# ---------------------------------------------------------------------------------- in the step

@pytest.mark.parametrize("kind,lens,q", [("bf16", [300, 64, 129], 1), ("fp8_e4m3", [200, 65], 1), ("bf16", [130, 70], 3)])
def test_run_tokens_is_the_step_on_rotated_inputs(kind, lens, q):
    """run_tokens against rotating, appending and run done one by one: the same bits; then the same
    through a captured graph replayed on new tokens, and on another stream."""
    inp = synth.make_inputs(lens, seed=61, kv_dtype=kind, queries_per_seq=q)
    rope = binding.Rope(64, scaling="yarn", factor=40.0, original_len=4096)
    rows = len(lens) * q
    places = [(b, S - q + t) for b, S in enumerate(lens) for t in range(q)]
    pos = torch.tensor([p for _, p in places], dtype=torch.int32, device=DEV)
    slots = torch.tensor([int(inp.block_table[b, p // 64]) * 64 + p % 64 for b, p in places], dtype=torch.int32, device=DEV)

    def new(seed):
        c_kv, k_r, _, _, qq = _tokens(rows, seed)
        return qq, (c_kv / c_kv.float().abs().amax(1, keepdim=True)).bfloat16().contiguous(), k_r.contiguous()

    def parts(step, qq, c_kv, k_r):
        q_c, q_r = qq[..., :128].contiguous(), torch.empty(rows, 128, 64, dtype=torch.bfloat16, device=DEV)
        k = torch.empty(rows, 1, 64, dtype=torch.bfloat16, device=DEV)
        binding.mla_rope(rope, qq[..., 128:], pos, q_r)
        binding.mla_rope(rope, k_r.unsqueeze(1), pos, k)
        kv = {n: getattr(step, n) for n in ("kv_pool", "kv_scale", "kr_pool")}
        binding.mla_append_kv(c_kv, k[:, 0].contiguous(), slots, dev_error=step.dev_error, **kv)
        return step.run(q_c, q_r).clone()

    def make(**kw):
        _, _, w_uk, w_uv, kv, bt = binding.inputs_to_device(inp, DEV)
        return binding.DecodeStep(inp.seq_lens, w_uk=w_uk, w_uv=w_uv, block_table=bt, queries_per_seq=q,
                                  min_pages_per_split=2, **kv, **kw)

    one, two = make(), make(rope=rope)
    first, second = new(1), new(2)
    wants = [parts(one, *first), parts(one, *second)]
    assert torch.equal(two.run_tokens(*first, pos, slots), wants[0])
    static = [t.clone() for t in first]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        two.run_tokens(*static, pos, slots)
    for s, t in zip(static, second):
        s.copy_(t)
    graph.replay()
    assert torch.equal(two.out, wants[1])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    two.run_tokens(*first, pos, slots, stream=stream)
    stream.synchronize()
    assert torch.equal(two.out, wants[0])
    assert one.device_error() == 0 and two.device_error() == 0


def test_one_token_of_any_token_stride():
    """The stride from token to token of a single token is never used, so it may be anything."""
    rope, err = binding.Rope(64), torch.zeros(1, dtype=torch.int32, device=DEV)
    c_kv, k_r, pos, slots, q = _tokens(1, 8)
    pools = [_cache("bf16") for _ in range(2)]
    outs = [[torch.zeros(1, 128, d, dtype=torch.bfloat16, device=DEV) for d in (128, 64)] for _ in range(2)]
    odd = [c_kv.as_strided(c_kv.shape, (577, 1)), k_r.as_strided(k_r.shape, (1, 1)),
           q.as_strided(q.shape, (3, q.stride(1), 1))]
    for (c, k, qq), kv, (q_c, q_r) in zip(([c_kv, k_r, q], odd), pools, outs):
        kv["kv_pool"].zero_()
        binding.mla_rope_append_kv(rope, c, k, pos, slots, dev_error=err, q=qq, q_c=q_c, q_r=q_r, **kv)
    assert torch.equal(pools[0]["kv_pool"], pools[1]["kv_pool"]) and int(err) == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_run_tokens_refusals():
    inp = synth.make_inputs([100], seed=1)
    _, _, w_uk, w_uv, kv, bt = binding.inputs_to_device(inp, DEV)
    make = lambda **kw: binding.DecodeStep(inp.seq_lens, w_uk=w_uk, w_uv=w_uv, block_table=bt, **kv, **kw)  # noqa: E731
    c_kv, k_r, pos, slots, q = _tokens(2, 3)
    with pytest.raises(ValueError):
        make().run_tokens(q[:1], c_kv[:1], k_r[:1], pos[:1], slots[:1])
    with pytest.raises(ValueError):
        make(rope=binding.Rope(64)).run_tokens(q, c_kv, k_r, pos, slots)
    with pytest.raises(ValueError):
        make(rope=binding.Rope(64)).run_tokens(None, c_kv[:1], k_r[:1], pos[:1], slots[:1])
    with pytest.raises(ValueError):
        make(rope=binding.Rope(128))

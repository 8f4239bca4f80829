"""The decode step under a sliding window with sinks, and behind a shared prefix, in 64 bits."""
import math

import pytest
import torch

import attend_util as au
from mla_latent_kv_absorb_gb300 import binding
from parity_util import TOL_BF16, TOL_FP8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def visible(L, W, n):
    """The positions that a row with L tokens sees."""
    return [j for j in range(L) if W == 0 or j >= L - W or j < n]


def draw(lens, q, W, n, kind="bf16", seed=0, poison=True):
    """A batch whose cache holds the pages that some row sees, everything else in them NaN; other table entries are -1."""
    gen = au.generator(seed)
    rows = [[visible(S - q + 1 + t, W, n) for t in range(q)] for S in lens]
    tokens = [sorted(set().union(*r)) for r in rows]
    pages = [sorted({j // 64 for j in t}) for t in tokens]
    total = sum(map(len, pages))
    kv = au.make_cache(gen, total + 3, kind)
    table = torch.full((len(lens), (max(lens) + 63) // 64), -1, dtype=torch.int32)
    perm, at = torch.randperm(total + 3, generator=gen, device="cuda").tolist(), 0
    live = torch.zeros((total + 3) * 64, dtype=torch.bool)
    for b, held in enumerate(pages):
        for p in held:
            table[b, p] = perm[at]
            at += 1
        idx = torch.tensor(tokens[b])
        live[table[b, idx // 64].long() * 64 + idx % 64] = True
    if poison:
        dead = ~live.cuda()
        if kind == "bf16":
            kv["kv_pool"].flatten(0, 1)[dead] = float("nan")
        else:
            kv["kv_pool"].flatten(0, 1)[dead] = 0x7F
            kv["kv_scale"].flatten(0, 1)[dead] = float("nan")
            kv["kr_pool"].flatten(0, 1)[dead] = float("nan")
    R = len(lens) * q
    return dict(kv=kv, table=table.cuda(), rows=[r for s in rows for r in s], q=q,
                w_uk=au.normal(gen, 128, 128, 512, std=512 ** -0.5), w_uv=au.normal(gen, 128, 128, 512, std=512 ** -0.5),
                q_c=au.normal(gen, R, 128, 128), q_r=au.normal(gen, R, 128, 64))


def reference(x, r):
    """Row r: out [128, 128] and lse [128]."""
    at = torch.tensor(x["rows"][r], device="cuda")
    c, kr = au.cache_values(x["kv"], x["table"][r // x["q"]].long()[at // 64] * 64 + at % 64)
    folded = torch.einsum("hd,hdc->hc", x["q_c"][r].double(), x["w_uk"].double())
    s = (folded @ c.T + x["q_r"][r].double() @ kr.T) * au.SCALE
    return torch.einsum("hc,hdc->hd", torch.softmax(s, dim=1) @ c, x["w_uv"].double()), torch.logsumexp(s, dim=1)


def compare(step, out, x, tol, rows=None):
    """The library's tolerances of the step, beside half a step of bf16 where an output is large."""
    for r in range(len(x["rows"])) if rows is None else rows:
        want, lse = reference(x, r)
        err = (out[r].double() - want).abs()
        assert torch.isfinite(out[r].float()).all(), f"row {r}"
        assert float((err - au.U * want.abs()).max()) <= tol["max_abs"], f"row {r}: {float(err.max())}"
        assert float(err.norm() / want.norm()) <= tol["rel_l2"], f"row {r}: {float(err.norm() / want.norm())}"
        assert float((step.lse[r].double() - lse).abs().max()) <= tol["max_abs"], f"row {r}: lse"
    assert step.device_error() == 0


def make(x, lens, W, n, **kw):
    return binding.DecodeStep(lens, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table=x["table"], queries_per_seq=x["q"], window=W,
                              sinks=n, **x["kv"], **kw)


CASES = [([1], 1, 1, 0), ([64, 65, 63], 1, 1, 0), ([300], 1, 64, 0), ([300, 7, 1000], 1, 65, 1), ([130], 1, 40, 100),
         ([129], 1, 20, 100), ([700, 701], 1, 128, 64), ([4000], 1, 1, 129), ([2000, 64], 1, 5000, 3),
         ([6000], 1, 1500, 70), ([100, 250, 1000], 4, 33, 5), ([64, 300], 3, 64, 0), ([513], 7, 2, 2),
         ([1000, 2000, 3000, 1, 77, 640], 1, 200, 10)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,q,W,n", CASES)
def test_window(lens, q, W, n, kind):
    lens = [max(S, q) for S in lens]
    x = draw(lens, q, W, n, kind, seed=sum(lens) + W + n)
    step = make(x, lens, W, n)
    compare(step, step.run(x["q_c"], x["q_r"]), x, TOL_BF16 if kind == "bf16" else TOL_FP8)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_window_splits(kind):
    """Items that begin and end everywhere: the sinks' page, the window's first page, inside it."""
    lens = [1000, 333, 2100]
    x = draw(lens, 1, 700, 130, kind, seed=2)
    for pages, clusters in ((1, 0), (1, 7), (2, 11), (3, 3)):
        step = make(x, lens, 700, 130, min_pages_per_split=pages, max_clusters=clusters)
        compare(step, step.run(x["q_c"], x["q_r"]), x, TOL_BF16 if kind == "bf16" else TOL_FP8)


def test_many_sequences():
    lens = [1 + (37 * i) % 900 for i in range(200)]
    x = draw(lens, 1, 150, 9, seed=5)
    step = make(x, lens, 150, 9)
    compare(step, step.run(x["q_c"], x["q_r"]), x, TOL_BF16, rows=range(0, 200, 7))


def test_window_past_the_length_is_no_window():
    lens = [70, 500, 1]
    x = draw(lens, 1, 0, 0, seed=6)
    want = make(x, lens, 0, 0).run(x["q_c"], x["q_r"])
    for W in (500, 5000, 2 ** 31 - 1):
        assert torch.equal(make(x, lens, W, 0).run(x["q_c"], x["q_r"]), want)
        assert torch.equal(make(x, lens, W, 2 ** 31 - 1).run(x["q_c"], x["q_r"]), want)


@pytest.mark.parametrize("W,n", [(100, 0), (64, 3)])
def test_fused_and_static_and_graph_and_host(W, n):
    lens = [900, 130, 64]
    x = draw(lens, 1, W, n, seed=7)
    step = make(x, lens, W, n)
    want, lse = step.run(x["q_c"], x["q_r"]).clone(), step.lse.clone()
    compare(step, want, x, TOL_BF16)
    for kw in (dict(fused_absorb=True), dict(fused_tail=True)):
        other = make(x, lens, W, n, **kw)
        assert torch.equal(other.run(x["q_c"], x["q_r"]), want) and torch.equal(other.lse, lse)
    graph = step.capture(x["q_c"], x["q_r"])
    step.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, want)
    o_lat, l2 = torch.empty_like(step.o_lat), torch.empty_like(step.lse)
    binding.mla_decode_paged_static_ws(step.info, step.plan_dev, step.q_abs, x["q_r"], block_table=x["table"], o_lat=o_lat,
                                       lse=l2, dev_error=step.dev_error, **x["kv"])
    assert torch.equal(o_lat, step.o_lat) and torch.equal(l2, lse)
    host = [t.cpu().pin_memory() for t in (x["q_c"], x["q_r"], torch.empty_like(want))]
    assert torch.equal(step.run_host(host[0], host[1]).cuda(), want)
    assert torch.equal(step.run_host(host[0], host[1], out=host[2]).cuda(), want)


def test_prefill_chunk_dispatch():
    """Chunks on both sides of the threshold, under a window, against each other's formula."""
    S, W, n = 700, 90, 5
    for T in (3, 300):
        x = draw([S], T, W, n, seed=T)
        out, err = binding.prefill_chunk(S, x["q_c"], x["q_r"], w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["table"][0],
                                         window=W, sinks=n, **x["kv"])
        assert binding.mla_read_device_error(err) == 0
        for r in (0, 1, T - 1):
            want, _ = reference(x, r)
            d = (out[r].double() - want).abs()
            assert float((d - au.U * want.abs()).max()) <= 2e-2 and float(d.norm() / want.norm()) <= 1e-2


def test_window_moves_with_run_tokens():
    """A few tokens one after the other: rotated, appended, attended under the window; pages behind it are given back."""
    gen = au.generator(11)
    W, n, S0 = 100, 3, 250
    kv = au.make_cache(gen, 8, "bf16")
    table = torch.tensor([[5, 2, 7, 0, 3]], dtype=torch.int32, device="cuda")
    w = [au.normal(gen, 128, 128, 512, std=512 ** -0.5) for _ in range(2)]
    rope = binding.Rope(64)
    for step_no in range(3):
        S = S0 + step_no + 1
        gone = [p for p in range(5) if (p + 1) * 64 <= S - W and p * 64 >= n]
        t = table.clone()
        t[0, gone] = 10 ** 9
        step = binding.DecodeStep([S], w_uk=w[0], w_uv=w[1], block_table=t, window=W, sinks=n, rope=rope, **kv)
        q, row = au.normal(gen, 1, 128, 192), au.normal(gen, 1, 576)
        pos = torch.tensor([S - 1], dtype=torch.int32, device="cuda")
        slot = (table[0, (S - 1) // 64] * 64 + (S - 1) % 64).reshape(1).int()
        out = step.run_tokens(q, row[:, :512], row[:, 512:], pos, slot)
        x = dict(kv=kv, table=table, rows=[visible(S, W, n)], q=1, w_uk=w[0], w_uv=w[1], q_c=step.q_c, q_r=step.q_r)
        compare(step, out, x, TOL_BF16)


# ---------------------------------------------------------------------------- behind a shared prefix

def own_and_whole(lens, P, kind="bf16", q=1, seed=0):
    """A batch of sequences behind a prefix of P tokens: own tables, the prefix's table, the rows' own tokens."""
    gen = au.generator(seed)
    x = draw(lens, q, 0, 0, kind, seed=seed + 1)
    pages = (P + 63) // 64
    pre = au.make_cache(gen, pages, kind)
    base = x["kv"]["kv_pool"].shape[0]
    x["kv"] = {k: torch.cat([x["kv"][k], pre[k]]) for k in pre}
    x["pre"] = (base + torch.randperm(pages, generator=gen, device="cuda")).int()
    return x


def joined(x, r, P):
    at = torch.tensor(x["rows"][r], device="cuda")
    pre = torch.arange(P, device="cuda")
    slots = torch.cat([x["pre"].long()[pre // 64] * 64 + pre % 64, x["table"][r // x["q"]].long()[at // 64] * 64 + at % 64])
    c, kr = au.cache_values(x["kv"], slots)
    folded = torch.einsum("hd,hdc->hc", x["q_c"][r].double(), x["w_uk"].double())
    s = (folded @ c.T + x["q_r"][r].double() @ kr.T) * au.SCALE
    return torch.einsum("hc,hdc->hd", torch.softmax(s, dim=1) @ c, x["w_uv"].double()), torch.logsumexp(s, dim=1)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,P,q", [([1], 1, 1), ([64, 1, 300], 130, 1), ([10, 90], 1000, 3), ([5] * 70, 333, 2)])
def test_step_behind_prefix(lens, P, q, kind):
    lens = [max(S, q) for S in lens]
    x = own_and_whole(lens, P, kind, q, seed=P)
    prefix = binding.SharedPrefix(P, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["pre"], **x["kv"])
    step = binding.DecodeStep(lens, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table=x["table"], queries_per_seq=q, prefix=prefix,
                              **x["kv"])
    tol = TOL_BF16 if kind == "bf16" else TOL_FP8

    def look(out, rows):
        for r in rows:
            want, lse = joined(x, r, P)
            err = (out[r].double() - want).abs()
            assert float((err - au.U * want.abs()).max()) <= tol["max_abs"] and float(err.norm() / want.norm()) <= tol["rel_l2"]
            assert float((step.lse[r].double() - lse).abs().max()) <= tol["max_abs"]

    rows = range(0, len(lens) * q, 1 + len(lens) * q // 8)
    out = step.run(x["q_c"], x["q_r"])
    look(out, rows)
    want = out.clone()
    graph = step.capture(x["q_c"], x["q_r"])
    step.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, want) and step.device_error() == 0
    assert step.graph_kernel_nodes in (None, step.launches_per_step)


def test_prefix_with_run_tokens_and_4_bit_weights():
    """The whole chain: rotate and append, the step in 4 bits over the own tokens, the prefix, the merge."""
    P, lens = 200, [70, 3]
    x = own_and_whole(lens, P, seed=9)
    gen = au.generator(77)
    packed = []
    for shape in ((128, 512, 128), (128, 128, 512)):
        codes = torch.randint(0, 256, shape[:2] + (shape[2] // 2,), generator=gen, device="cuda", dtype=torch.uint8)
        scale = ((torch.rand(*shape[:2], shape[2] // 32, generator=gen, device="cuda") + 0.5) / (4 * math.sqrt(512))).bfloat16()
        both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8
        packed.append((binding.W4Weight(codes, scale), (both * scale.float().repeat_interleave(32, dim=-1))))
    (uk, uk_f), (uv, uv_f) = packed
    # the prefix is made with the same weights in bf16: a product of a 4-bit code and a bf16 scale rounds once
    x["w_uk"], x["w_uv"] = uk_f.transpose(1, 2).bfloat16().contiguous(), uv_f.bfloat16()
    prefix = binding.SharedPrefix(P, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["pre"], **x["kv"])
    step = binding.DecodeStep(lens, w_uk=uk, w_uv=uv, block_table=x["table"], prefix=prefix, rope=binding.Rope(64), **x["kv"])
    q, row = au.normal(gen, 2, 128, 192), au.normal(gen, 2, 576)
    pos = torch.tensor([P + S - 1 for S in lens], dtype=torch.int32, device="cuda")
    slots = torch.stack([x["table"][b, (S - 1) // 64] * 64 + (S - 1) % 64 for b, S in enumerate(lens)]).int()
    out = step.run_tokens(q, row[:, :512], row[:, 512:], pos, slots)
    x["q_c"], x["q_r"] = step.q_c, step.q_r
    for r in range(2):
        want, _ = joined(x, r, P)
        err = (out[r].double() - want).abs()
        assert float((err - au.U * want.abs()).max()) <= 2e-2 and float(err.norm() / want.norm()) <= 1e-2
    assert step.device_error() == 0


def test_prefix_refusals():
    x = own_and_whole([10], 70, seed=1)
    prefix = binding.SharedPrefix(70, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["pre"], **x["kv"])
    kw = dict(w_uk=x["w_uk"], w_uv=x["w_uv"], block_table=x["table"], prefix=prefix, **x["kv"])
    with pytest.raises(ValueError):
        binding.DecodeStep([10], window=5, **kw)
    step = binding.DecodeStep([10], **kw)
    with pytest.raises(ValueError):
        step.run_host(x["q_c"].cpu(), x["q_r"].cpu())
    with pytest.raises(ValueError):
        binding.SharedPrefix(0, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["pre"], **x["kv"])
    with pytest.raises(ValueError):
        binding.SharedPrefix(129, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["pre"][:2], **x["kv"])
    out = torch.empty_like(x["q_c"])
    good = dict(out=out, own_out=out, own_lse=step.lse)
    for bad in (dict(own_lse=None), dict(own_out=out.float()), dict(out=out[:, :64]), dict(own_lse=step.lse[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            binding.mla_prefix_attend(prefix, x["q_c"], x["q_r"], **{**good, **bad})
    with pytest.raises(binding.MlaError) as e:
        binding.mla_prefix_attend(prefix, x["q_c"], x["q_r"], **good, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == binding.MLA_ERR_WORKSPACE
    with pytest.raises((ValueError, TypeError)):
        binding.SharedPrefix.of(prefix.k, prefix.v[:, :5], prefix.k_r)

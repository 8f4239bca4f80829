"""Shared prefixes: mla_prefix_open, mla_prefix_attend against the formulas in 64 bits."""
import math

import pytest
import torch

import attend_util as au
from mla_latent_kv_absorb_gb300 import binding

pytestmark = pytest.mark.gpu
W_STD = 512 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def draw(R, P, seed, std=1.0):
    gen = au.generator(seed)
    return dict(q_c=au.normal(gen, R, 128, 128, std=std), q_r=au.normal(gen, R, 128, 64, std=std),
                k=au.normal(gen, 128, P, 128), v=au.normal(gen, 128, P, 128), k_r=au.normal(gen, P, 576)[:, 512:],
                own_out=au.normal(gen, R, 128, 128), own_lse=torch.randn(R, 128, generator=gen, device="cuda") + math.log(P + 1))


def reference(x, own=True, scale=au.SCALE):
    ref = au.attend64(x["q_c"], x["q_r"], x["k"], x["v"], x["k_r"], scale=scale)
    if not own:
        return ref
    o = x["own_out"].double()
    return au.merge64([ref, (o, x["own_lse"].double(), o.abs(), torch.zeros_like(ref[3]))])


def attend(x, **kw):
    prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
    out, lse = torch.full_like(x["q_c"], float("nan")), torch.full(x["q_c"].shape[:2], float("nan"), device="cuda")
    own = {} if kw.pop("own", True) is False else dict(own_out=x["own_out"], own_lse=x["own_lse"])
    binding.mla_prefix_attend(prefix, x["q_c"], x["q_r"], out, lse=lse, **own, **kw)
    assert binding.mla_read_device_error(prefix.dev_error) == 0
    return out, lse


@pytest.mark.parametrize("R,P", [(1, 1), (1, 64), (2, 127), (3, 128), (2, 129), (1, 257), (5, 513), (32, 65), (33, 300),
                                 (64, 1000), (97, 2001), (128, 640), (128, 129), (129, 1), (129, 300), (200, 129),
                                 (256, 770), (257, 200), (300, 513), (600, 130)])
def test_attend(R, P):
    x = draw(R, P, 100 * R + P)
    out, lse = attend(x)
    ref = reference(x)
    au.check(out, ref, keys=P, what=f"{R} rows, {P} tokens")
    au.check_lse(lse, ref, keys=P)


@pytest.mark.parametrize("R,P", [(1, 130), (40, 333), (150, 257)])
def test_prefix_alone(R, P):
    x = draw(R, P, R + P)
    out, lse = attend(x, own=False)
    ref = reference(x, own=False)
    au.check(out, ref, keys=P)
    au.check_lse(lse, ref, keys=P)


@pytest.mark.parametrize("R", [17, 140])
def test_sharp_scores_move_the_maximum(R):
    # scores of some 40 nats: the running maximum moves and earlier tiles are rescaled
    P = 900
    x = draw(R, P, R, std=24.0)
    x["k"][:, -1] *= 4
    out, lse = attend(x)
    ref = reference(x)
    au.check(out, ref, keys=P)
    au.check_lse(lse, ref, keys=P)


def test_other_scale():
    x = draw(9, 200, 5)
    out, lse = attend(x, softmax_scale=0.31)
    ref = reference(x, scale=0.31)
    au.check(out, ref, keys=200)
    au.check_lse(lse, ref, keys=200)


@pytest.mark.parametrize("R", [37, 131])
def test_rows_without_own_tokens(R):
    x = draw(R, 300, R)
    x["own_lse"][::3] = -math.inf
    x["own_out"][::3] = float("nan")
    x["own_lse"][1::3] += 60.0  # and rows that are nearly all own
    out, lse = attend(x)
    ref = reference(x)
    au.check(out, ref, keys=300)
    au.check_lse(lse, ref, keys=300)


@pytest.mark.parametrize("R", [20, 160])
def test_in_place_and_rows_behind_untouched(R):
    x = draw(R, 257, R)
    want, want_lse = attend(x)
    whole = torch.cat([x["own_out"], torch.full_like(x["own_out"][:3], 7.0)])
    lses = torch.cat([x["own_lse"], torch.full_like(x["own_lse"][:3], 7.0)])
    prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
    ws = torch.full((prefix.workspace_bytes(R) + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN, and a guard behind it
    binding.mla_prefix_attend(prefix, x["q_c"], x["q_r"], whole[:R], lse=lses[:R], own_out=whole[:R], own_lse=lses[:R],
                              workspace=ws[:-64])
    assert torch.equal(whole[:R], want) and torch.equal(lses[:R], want_lse)
    assert (whole[R:] == 7).all() and (lses[R:] == 7).all() and (ws[-64:] == 255).all()


def test_graph_and_other_stream():
    x = draw(70, 500, 3)
    want, want_lse = attend(x)
    prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
    out, lse, ws = torch.empty_like(want), torch.empty_like(want_lse), prefix.workspace(70)
    side = torch.cuda.Stream()
    call = lambda: binding.mla_prefix_attend(prefix, x["q_c"], x["q_r"], out, lse=lse, own_out=x["own_out"],  # noqa: E731
                                             own_lse=x["own_lse"], workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_no_rows():
    x = draw(1, 70, 1)
    prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
    out = torch.empty(0, 128, 128, dtype=torch.bfloat16, device="cuda")
    binding.mla_prefix_attend(prefix, out, torch.empty(0, 128, 64, dtype=torch.bfloat16, device="cuda"), out)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("P", [1, 64, 65, 300, 1001])
def test_open(kind, P):
    gen = au.generator(P)
    pages = (P + 63) // 64
    kv = au.make_cache(gen, pages + 3, kind)
    table = torch.randperm(pages + 3, generator=gen, device="cuda").int()
    w_uk, w_uv = au.normal(gen, 128, 128, 512, std=W_STD), au.normal(gen, 128, 128, 512, std=W_STD)
    p = binding.SharedPrefix(P, w_uk=w_uk, w_uv=w_uv, block_table_row=table, **kv)
    assert binding.mla_read_device_error(p.dev_error) == 0
    at = torch.arange(P, device="cuda")
    slots = table.long()[at // 64] * 64 + at % 64
    c, kr = au.cache_values(kv, slots)
    c = c.float().bfloat16().double()  # the cache's values as mla_gather_kv gives them: bf16
    assert torch.equal(p.k_r.double(), kr)
    for got, w in ((p.k, w_uk), (p.v, w_uv)):
        want, size = torch.einsum("pc,hdc->hpd", c, w.double()), torch.einsum("pc,hdc->hpd", c.abs(), w.double().abs())
        # exact products, a sum of 512 in fp32, one rounding
        tol = au.U * want.abs() + 512 * 2.0 ** -23 * size
        assert ((got.double() - want).abs() <= tol).all()


def test_open_bad_page():
    gen = au.generator(1)
    kv = au.make_cache(gen, 3, "bf16")
    w = au.normal(gen, 128, 128, 512)
    p = binding.SharedPrefix(130, w_uk=w, w_uv=w, block_table_row=torch.tensor([0, 9, 1], dtype=torch.int32, device="cuda"), **kv)
    assert binding.mla_read_device_error(p.dev_error) == binding.MLA_DEVERR_BAD_PAGE


def test_workspace_is_the_streams(monkeypatch):
    """A workspace that the call makes belongs to the stream that the call is sent to."""
    x = draw(40, 300, 12)
    want = attend(x)
    prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
    side, seen, empty = torch.cuda.Stream(), [], torch.empty
    out = torch.empty_like(x["q_c"])
    torch.cuda.synchronize()

    def spy(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    for stream in (side, side.cuda_stream):
        monkeypatch.setattr(torch, "empty", spy)
        binding.mla_prefix_attend(prefix, x["q_c"], x["q_r"], out, own_out=x["own_out"], own_lse=x["own_lse"], stream=stream)
        monkeypatch.undo()
        side.synchronize()
        assert seen == [side.cuda_stream] and torch.equal(out, want[0])
        seen.clear()


def test_long_prefix():
    """140,001 tokens: the last heads' keys and values lie behind 2^31 elements."""
    P, heads = 140001, [0, 127]
    gen = au.generator(21)
    kv = au.make_cache(gen, (P + 63) // 64, "bf16")
    table = torch.randperm((P + 63) // 64, generator=gen, device="cuda").int()
    w_uk, w_uv = (au.normal(gen, 128, 128, 512, std=W_STD) for _ in range(2))
    prefix = binding.SharedPrefix(P, w_uk=w_uk, w_uv=w_uv, block_table_row=table, **kv)
    at = torch.tensor([0, 70000, P - 2, P - 1], device="cuda")
    c, kr = au.cache_values(kv, table.long()[at // 64] * 64 + at % 64)
    assert torch.equal(prefix.k_r[at].double(), kr)
    for got, w in ((prefix.k, w_uk), (prefix.v, w_uv)):
        want = torch.einsum("pc,hdc->hpd", c, w[heads].double())
        size = torch.einsum("pc,hdc->hpd", c.abs(), w[heads].double().abs())
        assert ((got[heads][:, at].double() - want).abs() <= au.U * want.abs() + 512 * 2.0 ** -23 * size).all()
    for R in (3, 130):
        q_c, q_r = au.normal(gen, R, 128, 128), au.normal(gen, R, 128, 64)
        out, lse = torch.empty_like(q_c), torch.empty(R, 128, device="cuda")
        binding.mla_prefix_attend(prefix, q_c, q_r, out, lse=lse)
        assert binding.mla_read_device_error(prefix.dev_error) == 0
        ref = au.attend64(q_c[:, heads], q_r[:, heads], prefix.k[heads], prefix.v[heads], prefix.k_r)
        au.check(out[:, heads], ref, keys=P)
        au.check_lse(lse[:, heads], ref, keys=P)


def test_two_calls_at_once():
    """Two streams with a workspace each share a prefix."""
    x, y = draw(40, 700, 5), draw(150, 700, 6)
    prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
    y.update(k=x["k"], v=x["v"], k_r=x["k_r"])
    want = attend(x)[0], attend(y)[0]
    got = [torch.empty_like(w) for w in want]
    streams, ws = [torch.cuda.Stream() for _ in got], [prefix.workspace(w.shape[0]) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w, z in zip(streams, got, ws, (x, y)):
            binding.mla_prefix_attend(prefix, z["q_c"], z["q_r"], o, own_out=z["own_out"], own_lse=z["own_lse"], workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

"""mla_prefill_window against attention over the visible tokens in 64 bits."""
import pytest
import torch

import attend_util as au
from mla_latent_kv_absorb_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def visible(S, T, W, n):
    pos, at = torch.arange(S - T, S, device="cuda")[:, None], torch.arange(S, device="cuda")
    return (at <= pos) & ((at > pos - W) | (at < n))


def draw(S, T, W, n, kind="bf16", seed=0, heads_std=1.0):
    """A sequence whose pages outside every query's window are not there: their entries are -1, and the rows of
    held pages that no query sees are NaN."""
    gen = au.generator(seed)
    seen = visible(S, T, W, n)
    token = seen.any(dim=0)
    pages = (S + 63) // 64
    held = torch.nn.functional.pad(token, (0, pages * 64 - S)).view(pages, 64).any(dim=1)
    kv = au.make_cache(gen, int(held.sum()) + 2, kind)
    table = torch.full((pages + 2,), -1, dtype=torch.int32, device="cuda")
    table[:pages][held] = torch.randperm(int(held.sum()), generator=gen, device="cuda").int()
    at = torch.arange(S, device="cuda")
    slots = table.long()[at // 64] * 64 + at % 64
    dead = torch.ones(kv["kv_pool"].shape[0] * 64, dtype=torch.bool, device="cuda")
    dead[slots[token]] = False
    for name in ("kv_scale", "kr_pool") if kind != "bf16" else ("kv_pool",):
        kv[name].flatten(0, 1)[dead] = float("nan")
    return dict(kv=kv, table=table, seen=seen, token=token, slots=slots,
                w_uk=au.normal(gen, 128, 128, 512, std=512 ** -0.5), w_uv=au.normal(gen, 128, 128, 512, std=512 ** -0.5),
                q_c=au.normal(gen, T, 128, 128, std=heads_std), q_r=au.normal(gen, T, 128, 64, std=heads_std))


def reference(x, heads):
    """The heads' attention with keys and values rounded once to bf16, as they are kept between the kernels."""
    c, kr = au.cache_values(x["kv"], x["slots"][x["token"]])
    c = c.float().bfloat16().double()
    k, v = (torch.einsum("pc,hdc->hpd", c, x[w][heads].double()).bfloat16() for w in ("w_uk", "w_uv"))
    return au.attend64(x["q_c"][:, heads], x["q_r"][:, heads], k, v, kr, seen=x["seen"][:, x["token"]])


def run(x, S, W, n, **kw):
    out = torch.full_like(x["q_c"], float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.mla_prefill_window(block_table_row=x["table"], seq_len=S, window=W, sinks=n, q_c=x["q_c"], q_r=x["q_r"],
                               w_uk=x["w_uk"], w_uv=x["w_uv"], out=out, dev_error=err, **x["kv"], **kw)
    assert binding.mla_read_device_error(err) == 0
    return out


# Keys and values are fp32 sums of 512 exact products, off by at most a = 512 2^-23 sum |c w| (absolutely: a sum
# near zero has no small relative error), and a sum that lies on the other side of a bf16 border than the exact one
# differs by a whole step, 2 U relative.  Values: 2 U and a.  Scores: sum_d |q_d| a * scale, and, if at most one
# product in sixteen crosses a border, 2^-4 2 U sum |q k| * scale, which is below 16 for N(0, 1) queries and keys;
# the weights follow with twice that.
def bounds(x, heads):
    c = au.cache_values(x["kv"], x["slots"][x["token"]])[0].abs()
    a = [512 * 2.0 ** -23 * float(torch.einsum("pc,hdc->hpd", c, x[w][heads].double().abs()).max()) for w in ("w_uk", "w_uv")]
    scores = float(x["q_c"][:, heads].double().abs().sum(dim=-1).max()) * a[0] * au.SCALE + 2.0 ** -4 * 2 * au.U * 16
    return dict(extra=2 * au.U + 2 * scores, absolute=a[1])


CASES = [(1, 1, 1, 0), (64, 64, 16, 0), (300, 300, 1, 0), (300, 300, 1, 3), (300, 257, 64, 4), (513, 300, 129, 128),
         (1000, 270, 700, 5), (1000, 400, 128, 0), (1500, 129, 255, 130), (2000, 600, 100, 700), (777, 513, 5000, 0),
         (777, 513, 5000, 9), (3000, 256, 1024, 64), (4100, 300, 33, 2)]


@pytest.mark.parametrize("S,T,W,n", CASES)
def test_chunk(S, T, W, n):
    x = draw(S, T, W, n, seed=S + T + W + n)
    out = run(x, S, W, n)
    heads = [0, 77, 127]
    au.check(out[:, heads], reference(x, heads), keys=min(S, W + n), **bounds(x, heads), what=f"S={S} T={T} W={W} n={n}")
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("kind", ["fp8", "nvfp4"])
@pytest.mark.parametrize("S,T,W,n", [(900, 300, 200, 70), (700, 256, 511, 0)])
def test_chunk_quantised(kind, S, T, W, n):
    x = draw(S, T, W, n, kind, seed=S)
    out = run(x, S, W, n)
    heads = [3, 64]
    au.check(out[:, heads], reference(x, heads), keys=min(S, W + n), **bounds(x, heads))


# wide windows, whose rows go to pairs of CTAs when the groups of 256 are nearly full
@pytest.mark.parametrize("S,T,W,n", [(2222, 250, 1024, 7), (1999, 499, 1500, 0), (1300, 1300, 1100, 0), (2500, 723, 2500, 0),
                                     (2600, 1003, 1200, 700), (2500, 330, 1100, 900)])
def test_chunk_wide(S, T, W, n):
    x = draw(S, T, W, n, seed=S + T + W + n)
    out = run(x, S, W, n)
    heads = [0, 77, 127]
    au.check(out[:, heads], reference(x, heads), keys=min(S, W + n), **bounds(x, heads), what=f"S={S} T={T} W={W} n={n}")
    assert torch.isfinite(out.float()).all()


# many short segments for each worker: one tile, two, three
@pytest.mark.parametrize("S,T,W,n", [(2048, 2048, 1, 0), (2049, 2048, 1, 1), (2100, 2048, 130, 0), (4100, 2100, 130, 5)])
def test_chunk_short_segments(S, T, W, n):
    x = draw(S, T, W, n, seed=S + T + W + n)
    out = run(x, S, W, n)
    heads = [0, 77, 127]
    au.check(out[:, heads], reference(x, heads), keys=min(S, W + n), **bounds(x, heads), what=f"S={S} T={T} W={W} n={n}")
    assert torch.isfinite(out.float()).all()


def test_whole_window_is_the_causal_chunk():
    """A window as long as the sequence sees what mla_prefill_decompressed sees."""
    S, T = 900, 300
    x = draw(S, T, S, 0, seed=8)
    want = torch.empty_like(x["q_c"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.mla_prefill_decompressed(block_table_row=x["table"], seq_len=S, q_c=x["q_c"], q_r=x["q_r"], w_uk=x["w_uk"],
                                     w_uv=x["w_uv"], out=want, dev_error=err, **x["kv"])
    got = run(x, S, S, 0)
    # both within a few roundings of bf16 of the same sums
    assert (got.double() - want.double()).norm() <= 2 * au.U * want.double().norm()


def test_workspace_given_and_guarded():
    S, T, W, n = 1000, 300, 200, 70
    x = draw(S, T, W, n, seed=4)
    size = binding.mla_prefill_window_workspace_bytes(S, T, W, n)
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(run(x, S, W, n, workspace=ws[:-64]), run(x, S, W, n))
    assert (ws[-64:] == 255).all()


def test_workspace_is_the_streams(monkeypatch):
    """A workspace that the call makes belongs to the stream that the call is sent to."""
    S, T, W, n = 600, 200, 100, 3
    x = draw(S, T, W, n, seed=11)
    want = run(x, S, W, n)
    side, seen, empty = torch.cuda.Stream(), [], torch.empty
    got, err = torch.empty_like(want), torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def spy(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    for stream in (side, side.cuda_stream):
        monkeypatch.setattr(torch, "empty", spy)
        binding.mla_prefill_window(block_table_row=x["table"], seq_len=S, window=W, sinks=n, q_c=x["q_c"], q_r=x["q_r"],
                                   w_uk=x["w_uk"], w_uv=x["w_uv"], out=got, dev_error=err, **x["kv"], stream=stream)
        monkeypatch.undo()
        side.synchronize()
        assert seen == [side.cuda_stream] and torch.equal(got, want) and int(err) == 0
        seen.clear()


def test_a_million_tokens():
    """Behind a long context only the window's and the sinks' pages are touched: every other table entry is -1."""
    S, T, W, n = 1048575, 130, 100, 70
    x = draw(S, T, W, n, seed=31)
    out = run(x, S, W, n)
    heads = [1, 126]
    au.check(out[:, heads], reference(x, heads), keys=W + n, **bounds(x, heads))


@pytest.mark.parametrize("S,T,W,n", [(900, 300, 200, 70), (2222, 250, 1024, 7)])
def test_captured_and_replayed(S, T, W, n):
    x, y = draw(S, T, W, n, seed=41), draw(S, T, W, n, seed=42)
    want = run(x, S, W, n), run(y, S, W, n)
    ws = torch.empty(binding.mla_prefill_window_workspace_bytes(S, T, W, n), dtype=torch.uint8, device="cuda")
    out, err = torch.empty_like(want[0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    z = {k: x[k].clone() for k in ("table", "q_c", "q_r", "w_uk", "w_uv")}
    pool = x["kv"]["kv_pool"].clone()
    call = lambda: binding.mla_prefill_window(  # noqa: E731
        block_table_row=z["table"], seq_len=S, window=W, sinks=n, q_c=z["q_c"], q_r=z["q_r"], w_uk=z["w_uk"], w_uv=z["w_uv"],
        out=out, dev_error=err, workspace=ws, kv_pool=pool)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in (0, 1, 0):
        for name, t in z.items():
            t.copy_((x, y)[k][name])
        pool.copy_((x, y)[k]["kv"]["kv_pool"])
        graph.replay()
        assert torch.equal(out, want[k]) and binding.mla_read_device_error(err) == 0


def test_bad_page():
    """A page that does not exist is reported, and the call ends."""
    S, T, W, n = 500, 200, 100, 3
    x = draw(S, T, W, n, seed=51)
    x["table"][6] = 1000000
    out, err = torch.empty_like(x["q_c"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(binding.mla_prefill_window_workspace_bytes(S, T, W, n), dtype=torch.uint8, device="cuda")
    binding.mla_prefill_window(block_table_row=x["table"], seq_len=S, window=W, sinks=n, q_c=x["q_c"], q_r=x["q_r"],
                               w_uk=x["w_uk"], w_uv=x["w_uv"], out=out, dev_error=err, workspace=ws, **x["kv"])
    assert binding.mla_read_device_error(err) == binding.MLA_DEVERR_BAD_PAGE

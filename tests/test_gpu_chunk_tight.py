"""mla_prefill_window in two halves, each within its own roundings: the keys and values that the call leaves in its
workspace against the cache and the weights, and the attention against exactly those keys and values.  So the bound
on an output is that of one softmax (attend_util), a tenth of what one key too many or too few changes, and every case
is tried with such wrong masks too."""
import math

import pytest
import torch

import attend_util as au
import test_gpu_window_chunk as chunks
from launch_util import launches_of
from mla_latent_kv_absorb_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def kept(ws, keys):
    """The rows [keys, 576], keys and values [128, keys, 128] that a call left in its workspace."""
    up = lambda n: (n + 1023) // 1024 * 1024  # noqa: E731
    k = up(keys * 1152)
    v = k + up(keys * 32768)
    cut = lambda at, n, *shape: ws[at:at + n].view(torch.bfloat16).view(*shape)  # noqa: E731
    return cut(0, keys * 1152, keys, 576), cut(k, keys * 32768, 128, keys, 128), cut(v, keys * 32768, 128, keys, 128)


def masks(S, T, W, n, token):
    """What the queries see, and masks that are wrong by one key."""
    pos, at = torch.arange(S - T, S)[:, None], torch.arange(S)
    window = lambda W, n, late=0: ((at <= pos + late) & ((at > pos - W) | (at < n)))[:, token]  # noqa: E731
    right = window(W, n)
    wrong = {"one key too long": window(W + 1, n), "one key too short": window(max(1, W - 1), n), "the next key": window(W, n, 1),
             "one sink more": window(W, n + 1), "one sink less": window(W, max(0, n - 1)),
             "the queries' own keys missing": right & ~(at == pos)[:, token]}
    # sixteen keys in a row that no query sees: half of an MMA step
    lost = torch.zeros(int(token.sum()), dtype=torch.bool)
    lost[lost.numel() // 2:lost.numel() // 2 + 16] = True
    wrong["sixteen keys lost"] = right & ~lost
    # (a key has a weight of about one over a row's keys: it is sure to show in the best of some rows, not in one)
    return right, {k: m for k, m in wrong.items() if int((m != right).any(dim=1).sum()) >= 16}


def worst(out, ref, keys):
    """The largest error of an output in units of its bound."""
    want, _, size, e = ref
    tol = (au.U + 2 * e[..., None] + 2.0 ** -20 + keys * 2.0 ** -23) * size + au.U * want.abs() + 1e-30
    return float(((out.double() - want).abs() / tol).max())


# alone: whether the rows go to CTAs alone, or to pairs (with 152 SMs)
CASES = [(256, 256, 64, 0, False), (256, 256, 1, 5, False), (250, 250, 129, 130, False), (3000, 250, 100, 5, False),
         (3000, 255, 130, 0, False), (555, 255, 130, 0, False), (511, 511, 300, 5, False), (768, 762, 500, 130, False),
         (2600, 1003, 1200, 700, False), (2222, 250, 1024, 7, False), (2500, 723, 2500, 0, False), (3000, 256, 1024, 64, False),
         (1999, 499, 1500, 0, False), (900, 300, 200, 70, True), (2500, 330, 1100, 900, True), (1300, 1300, 1100, 0, True),
         (4100, 300, 33, 2, True), (3000, 129, 128, 128, True)]


@pytest.mark.parametrize("kind,S,T,W,n,alone", [("bf16", *c) for c in CASES] + [
    (kind, *c) for kind in ("fp8", "nvfp4") for c in ((900, 300, 200, 70, True), (2222, 250, 1024, 7, False))])
def test_chunk(kind, S, T, W, n, alone):
    x = chunks.draw(S, T, W, n, kind, seed=S + T + W + n)
    keys = int(x["token"].sum())
    size = binding.mla_prefill_window_workspace_bytes(S, T, W, n)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    out = chunks.run(x, S, W, n, workspace=ws)
    rows, k, v = kept(ws, keys)

    # rows, keys and values: one rounding of the cache's value, then exact products, an fp32 sum and one rounding
    c, kr = au.cache_values(x["kv"], x["slots"][x["token"]])
    c = c.float().bfloat16().double()
    assert torch.equal(rows[:, :512].double(), c) and torch.equal(rows[:, 512:].double(), kr)
    heads = [0, 77, 127]
    for got, w in ((k, "w_uk"), (v, "w_uv")):
        want = torch.einsum("pc,hdc->hpd", c, x[w][heads].double())
        size = torch.einsum("pc,hdc->hpd", c.abs(), x[w][heads].double().abs())
        # half a step of bf16 where the sum lies, whose fp32 error is at most `slip`
        slip = 512 * 2.0 ** -23 * size
        assert ((got[heads].double() - want).abs() <= slip + au.bf16_step(want.abs() + slip) / 2).all()

    # the attention, head by head on the CPU
    right, wrong = masks(S, T, W, n, x["token"].cpu())
    assert wrong
    most = min(S, W + n)
    for h in heads:
        q_c, q_r, kh, vh, k_r = (t.cpu() for t in (x["q_c"][:, h:h + 1], x["q_r"][:, h:h + 1], k[h:h + 1], v[h:h + 1], rows[:, 512:]))
        got = out[:, h:h + 1].cpu()
        assert worst(got, au.attend64(q_c, q_r, kh, vh, k_r, seen=right), most) <= 1, f"head {h}"
        if h == 77:
            for what, mask in wrong.items():
                if bool(mask.any(dim=1).all()):
                    assert worst(got, au.attend64(q_c, q_r, kh, vh, k_r, seen=mask), most) > 1, what


@pytest.mark.parametrize("S,T,W,n,alone", CASES)
def test_who_takes_the_rows(S, T, W, n, alone):
    x = chunks.draw(S, T, W, n, seed=1)
    ws = torch.empty(binding.mla_prefill_window_workspace_bytes(S, T, W, n), dtype=torch.uint8, device="cuda")
    chunks.run(x, S, W, n, workspace=ws)
    out, err = torch.empty_like(x["q_c"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    names = [launch.name for launch in launches_of(lambda: binding.mla_prefill_window(
        block_table_row=x["table"], seq_len=S, window=W, sinks=n, q_c=x["q_c"], q_r=x["q_r"], w_uk=x["w_uk"], w_uv=x["w_uv"],
        out=out, dev_error=err, workspace=ws, **x["kv"]))]
    assert sum(f"attend_kernelILb1ELb{int(not alone)}E" in name for name in names) == 1 and len(names) == 3

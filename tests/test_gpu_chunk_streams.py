"""A chunk sent to a stream that is not the current one: what the call allocates and fills is that stream's."""
import pytest
import torch

import test_gpu_window_step as steps
from mla_latent_kv_absorb_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def spied(monkeypatch, call):
    """What call() returns and the streams that were current where it allocated."""
    seen = set()

    def spy(real):
        def made(*args, **kw):
            seen.add(torch.cuda.current_stream().cuda_stream)
            return real(*args, **kw)
        return made

    with monkeypatch.context() as m:
        for name in ("empty", "zeros", "from_numpy"):
            m.setattr(torch, name, spy(getattr(torch, name)))
        got = call()
    return got, seen


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("W,n", [(0, 0), (90, 3)])
def test_prefill_chunk(monkeypatch, T, W, n):
    S = 700
    x = steps.draw([S], T, W, n, seed=T + W)
    call = lambda **kw: binding.prefill_chunk(  # noqa: E731
        S, x["q_c"], x["q_r"], w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["table"][0], window=W, sinks=n, **x["kv"], **kw)
    want, err = call()
    assert binding.mla_read_device_error(err) == 0
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        (out, err), seen = spied(monkeypatch, lambda: call(stream=stream))
        assert seen == {side.cuda_stream} and torch.cuda.current_stream() == torch.cuda.default_stream()
        side.synchronize()
        assert torch.equal(out, want) and int(err) == 0
    with torch.cuda.stream(side):  # and the other way round
        for stream in (torch.cuda.default_stream(), 0):
            torch.cuda.synchronize()
            (out, err), seen = spied(monkeypatch, lambda: call(stream=stream))
            assert seen == {0}
            torch.cuda.synchronize()
            assert torch.equal(out, want) and int(err) == 0


def test_decompressed_workspace(monkeypatch):
    S, T = 500, 300
    x = steps.draw([S], T, 0, 0, seed=1)
    out, err = torch.empty_like(x["q_c"]), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda **kw: binding.mla_prefill_decompressed(  # noqa: E731
        block_table_row=x["table"][0], seq_len=S, q_c=x["q_c"], q_r=x["q_r"], w_uk=x["w_uk"], w_uv=x["w_uv"], out=out,
        dev_error=err, **x["kv"], **kw)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        out.zero_()
        torch.cuda.synchronize()
        _, seen = spied(monkeypatch, lambda: call(stream=stream))
        side.synchronize()
        assert seen == {side.cuda_stream} and torch.equal(out, want) and int(err) == 0


def test_many_chunks_on_another_stream():
    """Chunks one behind the other on a side stream while the current stream takes memory: their plans and
    workspaces stay theirs."""
    S, T, W, n = 700, 8, 90, 3
    x = steps.draw([S], T, W, n, seed=9)
    call = lambda **kw: binding.prefill_chunk(  # noqa: E731
        S, x["q_c"], x["q_r"], w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["table"][0], window=W, sinks=n, **x["kv"], **kw)
    want, _ = call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        got.append(call(stream=side))
        junk = [torch.full((1 << k,), -1, dtype=torch.int32, device="cuda") for k in range(8, 20)]
        del junk
    side.synchronize()
    assert all(torch.equal(out, want) and int(err) == 0 for out, err in got)

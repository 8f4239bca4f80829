"""Workspaces of calls that go to the default stream while another is current: the default stream's memory."""
import pytest
import torch

import test_gpu_prefix as prefixes
import test_gpu_window_chunk as chunks
from mla_latent_kv_absorb_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


@pytest.mark.parametrize("form", ["prefix", "chunk"])
def test_workspace(monkeypatch, form):
    if form == "prefix":
        x = prefixes.draw(40, 300, 12)
        want, _ = prefixes.attend(x)
        prefix = binding.SharedPrefix.of(x["k"], x["v"], x["k_r"])
        call = lambda out, stream: binding.mla_prefix_attend(  # noqa: E731
            prefix, x["q_c"], x["q_r"], out, own_out=x["own_out"], own_lse=x["own_lse"], stream=stream)
    else:
        x = chunks.draw(600, 200, 100, 3, seed=11)
        want = chunks.run(x, 600, 100, 3)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call = lambda out, stream: binding.mla_prefill_window(  # noqa: E731
            block_table_row=x["table"], seq_len=600, window=100, sinks=3, q_c=x["q_c"], q_r=x["q_r"], w_uk=x["w_uk"],
            w_uv=x["w_uv"], out=out, dev_error=err, stream=stream, **x["kv"])
    out, seen, empty = torch.empty_like(want), [], torch.empty

    def spy(*args, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for stream in (torch.cuda.default_stream(), 0):
            with monkeypatch.context() as m:
                m.setattr(torch, "empty", spy)
                call(out, stream)
            torch.cuda.synchronize()
            assert seen == [0] and torch.equal(out, want)
            seen.clear()
            out.zero_()
            torch.cuda.synchronize()

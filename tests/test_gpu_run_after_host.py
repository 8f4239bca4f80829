"""DecodeStep.run after a run_host of other lengths: the lengths, and the plan, of the construction."""
import pytest
import torch

import test_gpu_window_step as steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


@pytest.mark.parametrize("W,n", [(0, 0), (500, 5)])
@pytest.mark.parametrize("kw", [{}, dict(fused_tail=True)])
def test_run_after_run_host(W, n, kw):
    lens, short = [3000, 700], [65, 64]
    x = steps.draw(lens, 1, 0, 0, seed=2)
    step = steps.make(x, lens, W, n, min_pages_per_split=2, **kw)
    want, lse, launches = step.run(x["q_c"], x["q_r"]).clone(), step.lse.clone(), step.launches_per_step
    assert step.info.num_combine > 0
    host = [t.cpu().pin_memory() for t in (x["q_c"], x["q_r"], torch.empty_like(want))]
    other = steps.make(x, short, W, n, min_pages_per_split=2).run(x["q_c"], x["q_r"]).cpu()
    for out in (None, host[2]):  # planned for the call, and captured
        assert torch.equal(step.run_host(host[0], host[1], seq_lens=short, out=out), other)
        step.out.zero_()
        step.lse.zero_()
        assert torch.equal(step.run(x["q_c"], x["q_r"]), want) and torch.equal(step.lse, lse)
        assert step.launches_per_step == launches and step.device_error() == 0


@pytest.mark.parametrize("W,n", [(0, 0), (2000, 5)])
def test_captured_step_after_run_host(W, n):
    """A run_host whose lengths need a larger workspace leaves a captured step the one it was captured with."""
    lens, longer = [70, 300], [3000, 2500]
    x = steps.draw(longer, 1, 0, 0, seed=3)
    step = steps.make(x, lens, W, n, min_pages_per_split=2)
    graph = step.capture(x["q_c"], x["q_r"])
    want, at = step.out.clone(), step.workspace.data_ptr()
    host = [t.cpu().pin_memory() for t in (x["q_c"], x["q_r"], torch.empty_like(want))]
    other = steps.make(x, longer, W, n, min_pages_per_split=2)
    assert 0 < step.info.workspace_bytes < other.info.workspace_bytes
    ref = other.run(x["q_c"], x["q_r"]).cpu()
    for out in (None, host[2]):
        assert torch.equal(step.run_host(host[0], host[1], seq_lens=longer, out=out), ref)
        assert step.workspace.data_ptr() == at
        step.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want) and step.device_error() == 0

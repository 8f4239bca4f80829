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

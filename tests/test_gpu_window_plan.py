"""The windowed decode takes its sinks from the plan, as the pages and holes that go with them."""
import pytest
import torch

import test_gpu_window_step as steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("kw", [{}, dict(fused_absorb=True)])
@pytest.mark.parametrize("W,n", [(100, 70), (64, 0), (200, 5)])
def test_sinks_are_the_plans(kind, kw, W, n):
    lens = [900, 130, 64, 1000]
    x = steps.draw(lens, 1, W, n, kind, seed=W + n)
    step = steps.make(x, lens, W, n, **kw)
    want, lse = step.run(x["q_c"], x["q_r"]).clone(), step.lse.clone()
    for other in (0, 1, n + 64, 2 ** 31 - 1):  # another plan's figures
        step.info.sinks = other
        step.out.zero_()
        assert torch.equal(step.run(x["q_c"], x["q_r"]), want) and torch.equal(step.lse, lse)
    assert step.device_error() == 0


@pytest.mark.parametrize("n", [2 ** 30, 2 ** 31 - 64, 2 ** 31 - 1])
def test_sinks_past_every_length(n):
    lens = [700, 64]
    x = steps.draw(lens, 1, 0, 0, seed=1)
    want = steps.make(x, lens, 2 ** 31 - 1, 0).run(x["q_c"], x["q_r"])
    assert torch.equal(steps.make(x, lens, 3, n).run(x["q_c"], x["q_r"]), want)

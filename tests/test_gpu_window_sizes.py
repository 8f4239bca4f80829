"""Sizes that 32 bits do not hold, at the calls under a window."""
import pytest
import torch

import test_gpu_window_chunk as chunks
import test_gpu_window_step as steps
from mla_latent_kv_absorb_gb300 import binding

pytestmark = pytest.mark.gpu
BIG = 2 ** 32


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def test_chunk():
    S, T = 500, 300
    x = chunks.draw(S, T, S, 0, seed=3)
    want = chunks.run(x, S, S, 0)
    for W, n in ((BIG + 16, 0), (BIG, 0), (16, BIG + 3), (BIG + 16, BIG)):
        assert torch.equal(chunks.run(x, S, W, n), want)  # everything is seen
    for W, n in ((-BIG + 16, 0), (16, -BIG + 3), (0, 0)):
        with pytest.raises(binding.MlaError):
            chunks.run(x, S, W, n)
    for size in (BIG + S, -BIG + S):
        with pytest.raises(binding.MlaError):
            chunks.run(x, size, S, 0, workspace=torch.empty(1 << 26, dtype=torch.uint8, device="cuda"))


def test_step():
    lens = [300, 65]
    x = steps.draw(lens, 1, 0, 0, seed=4)
    want = steps.make(x, lens, 2 ** 31 - 1, 0).run(x["q_c"], x["q_r"])
    for W, n in ((BIG + 16, 0), (BIG + 16, BIG + 1), (16, BIG + 3)):
        assert torch.equal(steps.make(x, lens, W, n).run(x["q_c"], x["q_r"]), want)
    for W, n in ((-BIG + 16, 0), (16, -BIG + 3)):
        with pytest.raises(binding.MlaError):
            steps.make(x, lens, W, n)


def test_step_from_host_memory():
    x = steps.draw([300], 1, 0, 0, seed=5)
    want = steps.make(x, [300], 2 ** 31 - 1, 0).run(x["q_c"], x["q_r"]).cpu()
    step = steps.make(x, [300], BIG + 16, 3)
    q_c, q_r = x["q_c"].cpu(), x["q_r"].cpu()
    assert torch.equal(step.run_host(q_c, q_r), want)
    host = [t.pin_memory() for t in (q_c, q_r, torch.empty_like(want))]
    assert torch.equal(step.run_host(host[0], host[1], out=host[2]), want)

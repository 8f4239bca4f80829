"""mla_prefix_attend: a row's result does not depend on what the other rows hold."""
import math

import pytest
import torch

import attend_util as au
from test_gpu_prefix import attend, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


@pytest.mark.parametrize("R,P", [(2, 300), (16, 1000), (128, 700), (129, 700), (300, 500)])
def test_other_rows(R, P):
    x = draw(R, P, R)
    keep = [0, R // 2, R - 1]
    want, want_lse = attend(x)
    want, want_lse = want[keep].clone(), want_lse[keep].clone()
    others = torch.ones(R, dtype=torch.bool, device="cuda")
    others[keep] = False
    gen = au.generator(1)
    for std in (0.0, 30.0):  # rows that move their maximum in every tile, and rows that never do
        y = dict(x, q_c=x["q_c"].clone(), q_r=x["q_r"].clone(), own_out=x["own_out"].clone(), own_lse=x["own_lse"].clone())
        y["q_c"][others] = au.normal(gen, R, 128, 128, std=std)[others]
        y["q_r"][others] = au.normal(gen, R, 128, 64, std=std)[others]
        y["own_out"][others] = float("nan")
        y["own_lse"][others] = -math.inf
        out, lse = attend(y)
        assert torch.equal(out[keep], want) and torch.equal(lse[keep], want_lse)

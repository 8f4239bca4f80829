"""mla_prefix_attend where keys score -infinity."""
import math

import pytest
import torch

import attend_util as au
from test_gpu_prefix import attend, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


def masked(R, P, dead, seed):
    """Inputs of which the tokens `dead` score -infinity for every row, and their result without those tokens."""
    x = draw(R, P, seed)
    x["q_c"][..., 0] = x["q_c"][..., 0].abs() + 0.5
    seen = torch.ones(R, P, dtype=torch.bool, device="cuda")
    seen[:, dead] = False
    ref = au.attend64(x["q_c"], x["q_r"], x["k"], x["v"], x["k_r"], seen=seen)
    x["k"][:, dead, 0] = -math.inf
    return x, ref


# 900 tokens are eight tiles, 152 CTAs (76 pairs) take some seven (fourteen) each: in these ranges pieces of CTAs lie
# wholly among the dead tokens, at a run's beginning, its middle and its end
@pytest.mark.parametrize("R", [5, 64, 140])
@pytest.mark.parametrize("dead", [slice(0, 640), slice(256, 700), slice(130, 900), slice(0, 899)])
def test_tokens_at_minus_infinity(R, dead):
    x, ref = masked(R, 900, dead, R)
    out, lse = attend(x, own=False)
    au.check(out, ref, keys=900, what="prefix alone")
    au.check_lse(lse, ref, keys=900)
    o = x["own_out"].double()
    ref = au.merge64([ref, (o, x["own_lse"].double(), o.abs(), torch.zeros_like(ref[3]))])
    out, lse = attend(x)
    au.check(out, ref, keys=900)
    au.check_lse(lse, ref, keys=900)


@pytest.mark.parametrize("R,P", [(1, 1), (33, 300), (140, 900)])
def test_the_whole_prefix_at_minus_infinity(R, P):
    """Then only the own tokens count; a row without any gets zeros and -infinity."""
    x, _ = masked(R, P, slice(0, P), R)
    x["own_lse"][::3] = -math.inf
    x["own_out"][::3] = float("nan")
    out, lse = attend(x)
    want, want_lse = x["own_out"].clone(), x["own_lse"].clone()
    want[::3] = 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)  # a weight of exactly one
    out, lse = attend(x, own=False)
    assert (out == 0).all() and (lse == -math.inf).all()

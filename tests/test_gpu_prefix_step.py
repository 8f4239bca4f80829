"""The step behind a shared prefix where its own part takes the fused kernels, or several items of a sequence."""
import pytest
import torch

import attend_util as au
from mla_latent_kv_absorb_gb300 import binding
from parity_util import TOL_BF16, TOL_FP8
from test_gpu_window_step import joined, own_and_whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    torch.cuda.set_device(0)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("fused", [{}, dict(fused_absorb=True), dict(fused_tail=True), dict(fused_absorb=True, fused_tail=True)])
@pytest.mark.parametrize("lens,q,split", [([1000, 70, 333], 1, True), ([700, 130], 3, True), ([64, 5, 200], 1, False)])
def test_fused_and_split(kind, fused, lens, q, split):
    P = 300
    x = own_and_whole(lens, P, kind, q, seed=sum(lens) + q)
    prefix = binding.SharedPrefix(P, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table_row=x["pre"], **x["kv"])
    kw = dict(min_pages_per_split=1, item_cost_pages=-1) if split else dict(max_clusters=1)
    step = binding.DecodeStep(lens, w_uk=x["w_uk"], w_uv=x["w_uv"], block_table=x["table"], queries_per_seq=q, prefix=prefix,
                              **x["kv"], **kw, **fused)
    assert (step.info.num_combine > 0) == split
    out = step.run(x["q_c"], x["q_r"])
    tol = TOL_BF16 if kind == "bf16" else TOL_FP8
    for r in range(len(lens) * q):
        want, lse = joined(x, r, P)
        err = (out[r].double() - want).abs()
        assert float((err - au.U * want.abs()).max()) <= tol["max_abs"] and float(err.norm() / want.norm()) <= tol["rel_l2"]
        assert float((step.lse[r].double() - lse).abs().max()) <= tol["max_abs"]
    want = out.clone()
    graph = step.capture(x["q_c"], x["q_r"])
    step.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out, want) and step.device_error() == 0

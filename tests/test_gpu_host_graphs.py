"""How many captured steps DecodeStep.run_host keeps: the one of its last pinned call, and none that
later calls cannot use."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from mla_latent_kv_absorb_gb300 import binding, synth  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def alive(monkeypatch):
    """The handles of the graphs that were made and not destroyed yet."""
    L, handles = binding.lib(), []
    create, destroy = L.mla_step_graph_create, L.mla_step_graph_destroy

    def made(*args):
        st = create(*args)
        if st == binding.MLA_OK:
            handles.append(args[-1]._obj.value)
        return st

    def gone(handle):
        handles.remove(handle.value)
        return destroy(handle)

    monkeypatch.setattr(L, "mla_step_graph_create", made)
    monkeypatch.setattr(L, "mla_step_graph_destroy", gone)
    return handles


def _step(lens):
    inp = synth.make_inputs(lens, seed=41, poison_tail=False)
    _, _, w_uk, w_uv, kv, bt = binding.inputs_to_device(inp, DEV)
    step = binding.DecodeStep(inp.seq_lens, w_uk=w_uk, w_uv=w_uv, block_table=bt, min_pages_per_split=2, **kv)
    return step, inp.q_c.pin_memory(), inp.q_r.pin_memory(), torch.empty(inp.batch, 128, 128, dtype=torch.bfloat16).pin_memory()


def test_new_lengths_keep_one_graph(alive):
    """The graph of the lengths before goes with the call that makes the new one."""
    step, q_c, q_r, out = _step([3000, 700])
    first = step.run_host(q_c, q_r, out=out).clone()
    short = step.run_host(q_c, q_r, seq_lens=[900, 65], out=out).clone()
    assert len(alive) == 1 and step._host_graph is not None
    assert torch.equal(step.run_host(q_c, q_r, seq_lens=[3000, 700], out=out), first)
    assert torch.equal(step.run_host(q_c, q_r, seq_lens=[900, 65], out=out), short)
    assert len(alive) == 1


def test_calls_without_a_graph_keep_none(alive):
    """Pinned once, then other lengths from pageable tensors: the graph names a workspace that may have
    been replaced, and no later call can use it."""
    step, q_c, q_r, out = _step([900, 65])
    step.run_host(q_c, q_r, out=out)
    assert len(alive) == 1
    step.run_host(q_c.clone(), q_r.clone(), seq_lens=[700, 64])
    assert alive == [] and step._host_graph is None


def test_a_failed_call_keeps_none(alive):
    """New lengths past the block table are refused; the graph of the old ones goes all the same, since
    the step has taken the new lengths."""
    step, q_c, q_r, out = _step([900, 65])
    step.run_host(q_c, q_r, out=out)
    with pytest.raises(ValueError):
        step.run_host(q_c, q_r, seq_lens=[900, 64 * 1000], out=out)
    assert alive == [] and step._host_graph is None


def test_the_step_takes_its_graph_along(alive):
    step, q_c, q_r, out = _step([900, 65])
    step.run_host(q_c, q_r, out=out)
    step.run_host(q_c, q_r, seq_lens=[700, 64], out=out)
    del step
    assert alive == []

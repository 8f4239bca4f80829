"""Windows, sinks and lengths that 32 bits do not hold: not another size, without a GPU."""
import pytest

from mla_latent_kv_absorb_gb300 import binding

BIG = 2 ** 32


def test_plans():
    lens = [100000, 70]
    whole = binding.mla_plan_splits(lens, 152, window=2 ** 31 - 1)[1].total_pages
    assert whole == 1563 + 2
    for W, n in ((BIG + 64, 0), (BIG, 0), (2 ** 63, 0), (64, BIG + 3), (BIG + 64, BIG)):
        info = binding.mla_plan_splits(lens, 152, window=W, sinks=n)[1]
        assert info.total_pages == whole and info.window > 0
    for W, n in ((-BIG + 64, 0), (64, -BIG + 3), (-(2 ** 63), 0), (0, BIG)):
        with pytest.raises(binding.MlaError) as e:
            binding.mla_plan_splits(lens, 152, window=W, sinks=n)
        assert e.value.status == binding.MLA_ERR_INVALID_ARG


def test_chunk_workspaces():
    size = binding.mla_prefill_window_workspace_bytes
    assert size(5000, 10, BIG + 100) == size(5000, 10, 100, BIG + 3) == size(5000, 10, 5000)
    for args in ((BIG + 5000, 10, 100), (5000, -BIG + 10, 100), (5000, 10, -BIG + 100), (5000, 10, 100, -BIG)):
        if args[0] > BIG:  # as long as 32 bits say, not 5,000
            assert size(*args) == size(2 ** 31 - 1, 10, 100)
            continue
        with pytest.raises(binding.MlaError):
            size(*args)

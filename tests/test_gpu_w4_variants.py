"""GPU parity of every kernel that mla_linear_w4 chooses between, against the formula in 64 bits (the
tolerance is test_gpu_w4.py's), with a check of the choice: linear_w4_kernel<group, row tiles> on
mma.sync, 128 threads, or rows_kernel<group> on tensor memory, 640 threads."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from launch_util import launches_of  # noqa: E402
from test_gpu_w4 import DEV, FORMATS, _assert_product, _weight  # noqa: E402

from mla_latent_kv_absorb_gb300 import binding  # noqa: E402

pytestmark = pytest.mark.gpu


def _product(rows, heads, n, k, fmt, group, zero, chosen):
    """The product of random x against its formula; `chosen` is the kernel's name and row tiles."""
    w, value = _weight(heads, n, k, fmt, group, zero, n + rows)
    x = torch.randn(rows, heads, k, generator=torch.Generator().manual_seed(rows + k)).bfloat16().to(DEV)
    out = torch.full((rows, heads, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    call = lambda: binding.mla_linear_w4(x, w, out)  # noqa: E731
    launch, = launches_of(call)
    tiles = "" if chosen == "rows" else f"Li{chosen}E"
    name = f"{'rows_kernel' if chosen == 'rows' else 'linear_w4_kernel'}ILi{group}E{tiles}E"
    assert name in launch.name, (name, launch.name)
    assert launch.block == ((640, 1, 1) if chosen == "rows" else (128, 1, 1))
    call()
    _assert_product(out, x, value)
    return launch


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("rows,tiles", [(5, 1), (12, 2), (24, 3), (29, 4), (37, 5), (41, 6), (45, 6), (48, 6), (50, 8), (64, 8)])
@pytest.mark.parametrize("heads,n,k", [
    (1, 8190, 256),       # all warps over the outputs
    (128, 128, 512),      # two warps over k: the step's value projection
])
def test_products_on_mma_sync(fmt, group, zero, heads, n, k, rows, tiles):
    _product(rows, heads, n, k, fmt, group, zero, tiles)


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("rows", [41, 45, 48])
def test_products_of_two_warps_over_k_in_clusters(fmt, group, zero, rows):
    """4,096 -> 4,099: two warps over k, clusters of two or four, six row tiles."""
    launch = _product(rows, 1, 4099, 4096, fmt, group, zero, 6)
    assert launch.grid[0] in (2 * 65, 4 * 65)


# a shape that takes the kernel on tensor memory for each format at 33 rows or more
DENSE = {128: (1, 8200, 4096), 64: (1, 8200, 4096), 16: (1, 8200, 4096), 32: (128, 512, 128)}


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("rows", [33, 34, 47, 48])
def test_48_columns_of_tensor_memory(fmt, group, zero, rows):
    """33 to 48 rows: three chunks of 16 columns, more slots of x."""
    _product(rows, 128, 512, 128, fmt, group, zero, "rows")
    if group != 32:
        _product(max(rows, 37), *DENSE[group], fmt, group, zero, "rows")


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("heads,n,k,rows", [
    (1, 4096, 4096, 1152),    # two warps over k in the packed layout
    (1, 3950, 4096, 1101),    # the same, outputs end inside a tile, the last block of rows short
    (1, 2048, 8192, 2330),    # four warps over k
    (1, 1900, 8064, 2100),    # the same, half a pair at the end, k ends inside the packed steps
])
def test_pairs_of_tiles_in_turn_over_split_layouts(fmt, group, zero, heads, n, k, rows):
    """So many blocks of rows that a thread block takes several pairs of tiles, of weights whose packed
    layout has two or four warps over k."""
    launch = _product(rows, heads, n, k, fmt, group, zero, "rows")
    assert launch.grid[0] < (n + 255) // 256


@pytest.mark.parametrize("fmt,group,zero", FORMATS)
@pytest.mark.parametrize("heads,n,k,rows", [
    (1, 16500, 2112, 57), (1, 8200, 4096, 64), (1, 4096, 4096, 192), (1, 2048, 8192, 250), (128, 512, 128, 30),
    (64, 384, 192, 60), (3, 3000, 1024, 100), (1, 40000, 64, 64), (1, 65000, 320, 49)])
def test_parity_sizes_take_tensor_memory(fmt, group, zero, heads, n, k, rows):
    """Which of the sizes that test_gpu_w4.py compares as 'in tensor memory' take that kernel."""
    k = max(k - k % max(group, 32), group)
    size = binding.lib().mla_w4_packed_bytes  # the choice goes by sizes alone: zeros do as weights
    codes = torch.zeros(heads, n, k // 2, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(heads, n, k // group, dtype=torch.bfloat16 if fmt == "int4" else torch.uint8, device=DEV)
    w = binding.W4Weight(codes, scale, zero=scale.byte() if zero else None, group=group)
    assert size(w._ref) == w.packed.numel()
    x = torch.zeros(rows, heads, k, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(rows, heads, n, dtype=torch.bfloat16, device=DEV)
    launch, = launches_of(lambda: binding.mla_linear_w4(x, w, out))
    assert f"rows_kernelILi{group}E" in launch.name, launch.name

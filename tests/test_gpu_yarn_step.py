"""YaRN in the step: its temperature belongs to the whole head, of which the rotation turns 64 of 192
elements, so it goes into the softmax scale and the rotation's magnitude is 1."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from parity_util import TOL_BF16, assert_close  # noqa: E402

from mla_latent_kv_absorb_gb300 import binding, synth  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _turn(x, positions, freq):
    """x [..., 64] in 64 bits, interleaved pairs turned by positions [...] times freq."""
    angle = positions.double()[..., None] * freq
    z = torch.view_as_complex(x.double().unflatten(-1, (32, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle)).flatten(-2)


def test_yarn_temperature_of_the_whole_head():
    """run_tokens with magnitude 1 and softmax_scale = m^2 / sqrt(192) is attention over queries and keys
    both scaled by m = 0.1 ln(factor) + 1 as a whole, content and rotated part."""
    factor, trained, lens = 40.0, 4096, [300, 65, 1]
    inp = synth.make_inputs(lens, seed=91)
    _, _, w_uk, w_uv, kv, bt = binding.inputs_to_device(inp, DEV)
    m = 0.1 * math.log(factor) + 1.0
    rope = binding.Rope(64, scaling="yarn", factor=factor, original_len=trained, magnitude=1.0)
    step = binding.DecodeStep(inp.seq_lens, w_uk=w_uk, w_uv=w_uv, block_table=bt, rope=rope,
                              softmax_scale=m * m / math.sqrt(192.0), **kv)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3, 128, 192, generator=g).bfloat16().to(DEV)
    row = (torch.randn(3, 576, generator=g) * 0.5).bfloat16().to(DEV)
    pos = torch.tensor([150000, 64, 0], dtype=torch.int32, device=DEV)
    slots = torch.tensor([int(inp.block_table[b, (S - 1) // 64]) * 64 + (S - 1) % 64 for b, S in enumerate(lens)],
                         dtype=torch.int32, device=DEV)
    out = step.run_tokens(q, row[:, :512], row[:, 512:], pos, slots)
    assert step.device_error() == 0

    freq = []
    for i in range(32):   # the ramp runs from pair 10 to pair 23 (test_rope_w4_host.py works it out)
        f, t = 10000.0 ** (-i / 32), min(max((i - 10) / 13, 0.0), 1.0)
        freq.append(f * (1 - t) + f / factor * t)
    freq = torch.tensor(freq, dtype=torch.float64, device=DEV)
    q_r = _turn(q[..., 128:], pos[:, None].expand(3, 128), freq)
    k_new = _turn(row[:, 512:], pos, freq)
    pool = inp.pool.double().reshape(-1, 576).to(DEV)
    want = []
    for b, S in enumerate(lens):
        idx = torch.tensor([int(inp.block_table[b, p // 64]) * 64 + p % 64 for p in range(S)], device=DEV)
        c, kr = pool[idx, :512].clone(), pool[idx, 512:].clone()
        c[-1], kr[-1] = row[b, :512].double(), k_new[b]
        k_c = torch.einsum("hdc,sc->hsd", w_uk.double(), c)
        logits = torch.einsum("hd,hsd->hs", m * q[b, :, :128].double(), m * k_c) + (m * q_r[b]) @ (m * kr).t()
        p = (logits / math.sqrt(192.0)).softmax(-1)
        want.append(torch.einsum("hc,hdc->hd", p @ c, w_uv.double()))
    assert_close(out, torch.stack(want), TOL_BF16, "out")

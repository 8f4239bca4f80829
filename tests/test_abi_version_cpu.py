"""The header, the library and the binding agree on the layout of what they pass, and a program can tell."""
import ctypes
import os
import shutil
import subprocess

import pytest

from mla_latent_kv_absorb_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"mla_plan_options": binding.PlanOptions, "mla_plan_info": binding.PlanInfo, "mla_step_buffers": binding.StepBuffers,
           "mla_rope_options": binding.RopeOptions, "mla_rope_config": binding.RopeConfig, "mla_w4_weight": binding.W4Struct}


def test_the_library_tells_its_version():
    assert binding.lib().mla_abi_version() == binding.MLA_ABI_VERSION


def test_another_version_is_refused(monkeypatch):
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "MLA_ABI_VERSION", binding.MLA_ABI_VERSION + 1)
    with pytest.raises(RuntimeError, match="ABI version"):
        binding.lib()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_a_program_built_with_the_header(tmp_path):
    """Sizes and places of the structs' members as a C program has them."""
    lines = ["#include <stdio.h>", '#include "mla.h"', "int main(void) {", 'printf("%d\\n", MLA_ABI_VERSION);']
    want = [binding.MLA_ABI_VERSION]
    for name, struct in STRUCTS.items():
        lines.append(f'printf("%d\\n", (int)sizeof({name}));')
        want.append(ctypes.sizeof(struct))
        for member, *_ in struct._fields_:
            lines.append(f'printf("%d\\n", (int)offsetof({name}, {member}));')
            want.append(getattr(struct, member).offset)
    lines += ["return 0; }"]
    source, program = tmp_path / "p.c", tmp_path / "p"
    source.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", program, source], check=True)
    got = subprocess.run([program], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == want

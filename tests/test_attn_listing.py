"""The wait states in front of the attention kernels' loads to LDS, in the
listing of the built library (CPU only).

These loads are assembly blocks, for which the compiler counts no wait states,
while it may write a buffer's words with vector instructions (readfirstlane,
or readlane where it keeps scalars in vector registers) at any place before
them.  gfx9 wants five wait states between such a write and a buffer
instruction that reads it.
"""
import os
import re
import shutil
import subprocess

import pytest

import gated_delta_rule_amd as kda

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
IN_BLOCK = re.compile(r"s_nop|s_mov_b32 m0,|s_add_u32 m0, m0,|buffer_load_dword(x4)? .* offen lds$")


def listings(lib, folder):
    """Instructions of each of the library's kernels that loads to LDS."""
    at = os.path.join(folder, "lib.so")
    shutil.copy(lib, at)
    subprocess.run([OBJDUMP, "--offloading", at], check=True, capture_output=True)
    for name in sorted(os.listdir(folder)):
        if name.endswith("gfx950"):
            text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", os.path.join(folder, name)], check=True, capture_output=True,
                                  text=True).stdout
            for part in re.split(r"\n(?=[0-9a-f]+ <)", text):
                code = [re.sub(r"\s+", " ", line.split("//")[0]).strip() for line in part.splitlines()[1:]]
                if any(c.endswith(" offen lds") for c in code):
                    yield part.split("<")[1].split(">")[0], [c for c in code if c]


def states(instruction):
    return int(instruction.split()[1], 0) + 1 if instruction.startswith("s_nop") else 1


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_five_wait_states_stand_before_every_load_to_lds(tmp_path):
    if not os.path.exists(kda.library_path()):
        from gated_delta_rule_amd import build
        build.build()
    kernels = loads = 0
    for name, code in listings(kda.library_path(), str(tmp_path)):
        kernels += 1
        for i, c in enumerate(code):
            if c.endswith(" offen lds"):
                loads += 1
                seen = 0
                for before in reversed(code[:i]):
                    if seen >= 5 or not IN_BLOCK.match(before):
                        break
                    seen += states(before)
                assert seen >= 5, f"{name}: {seen} wait states before {c!r}"
    assert kernels >= 26 and loads > 500, (kernels, loads)   # forward, line, step, backward

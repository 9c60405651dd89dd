"""Rules of the instruction set that the compiler keeps by itself but not
inside inline assembly, checked in the built kernels (CPU only: the library's
own code objects are disassembled)."""
import os
import re
import shutil
import subprocess

import pytest

ns = pytest.importorskip("newton_schulz_amd")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


@pytest.fixture(scope="module")
def instructions(tmp_path_factory):
    """The instructions of every kernel, one code object after another."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    d = tmp_path_factory.mktemp("objects")
    shutil.copy(os.path.join(os.path.dirname(ns.__file__), "libnvfp4ns.so"), d / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=d, check=True, capture_output=True)
    lines = []
    for f in sorted(os.listdir(d)):
        if "gfx950" in f:
            r = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f], cwd=d, check=True, capture_output=True, text=True)
            lines += [s.strip() for s in r.stdout.splitlines()]
    return [s for s in lines if s]


def test_m0_is_written_a_wait_state_before_lds_loads(instructions):
    """A load into LDS takes its LDS base from M0, which a scalar instruction
    must have written at least one wait state (any other instruction) before."""
    loads = 0
    for before, line in zip(instructions, instructions[1:]):
        op = line.split()[0]
        if re.match(r"(global|scratch)_load_lds_", op) or (op.startswith("buffer_load") and re.search(r"\blds\b", line)):
            loads += 1
            assert not re.match(r"s_\w+\s+m0\b", before), f"{before} / {line}"
    assert loads > 100


def _scalars(text):
    """Numbers of the scalar registers named in an operand list."""
    out = set()
    for a, b, c in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= set(range(int(a), int(b) + 1)) if a else {int(c)}
    return out


def test_addresses_are_not_scalars_that_a_vector_instruction_just_wrote(instructions):
    """Five wait states lie between a vector instruction that writes a scalar
    register and a memory access that reads it."""
    checked = 0
    for i, line in enumerate(instructions):
        line = line.split("//")[0]
        if "_load_lds_" not in line:
            continue
        used, states = _scalars(line), 0
        checked += bool(used)
        for before in reversed(instructions[max(0, i - 8):i]):
            before = before.split("//")[0].strip()
            if before.endswith(":"):
                continue
            if before.startswith("v_"):
                assert not used & _scalars(before.split(",")[0]), f"{before} / {line}"
            states += int(before.split()[1], 0) + 1 if before.startswith("s_nop") else 1
            if states >= 5:
                break
    assert checked > 100

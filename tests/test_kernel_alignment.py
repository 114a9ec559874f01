"""Alignment of what the row norms move in 16-byte pieces, asked of the compiler (no GPU needed)."""
import os
import re
import subprocess

import pytest

from weight_state_recurrence_b200 import build

NORM = os.path.join(build.CSRC, "norm.cuh")


def test_rows_in_registers_are_aligned_to_their_pieces(tmp_path):
    src = tmp_path / "align.cu"
    src.write_text(f'#include "{NORM}"\n'
                   "using namespace linattn::norm;\n"
                   "static_assert(alignof(Raw<16, true, __nv_bfloat16>) >= 16);\n"
                   "static_assert(alignof(Raw<16, true, float>) >= 16);\n"
                   "static_assert(sizeof(Raw<16, true, __nv_bfloat16>) == 16);\n")
    subprocess.check_call([build.nvcc(), *build.NVCC_FLAGS, "-c", "-o", str(tmp_path / "align.o"), str(src)])


def test_arrays_read_as_pieces_say_so():
    with open(NORM) as f:
        text = f.read()
    local = re.findall(r"^\s*(alignas\(16\) )?__nv_bfloat162 p\[", text, re.M)
    assert local and all(local)

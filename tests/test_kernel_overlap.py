"""Declarations of the kernels that start before the grid in front of them has ended, read from the
sources (no GPU needed).

Such a kernel waits for that grid (grid_dependency_wait) before it reads what it wrote.  A pointer
declared `const ... __restrict__` says that nothing changes what it points to during the whole kernel, so
the loads through it may take the read-only path and may be moved across the wait.  Only the call's own
inputs, which no kernel writes, may be declared so.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir,
                    "weight_state_recurrence_b200", "csrc")
# inputs of a call, by the names that the entry points give them
INPUTS = {"q", "k", "v", "g", "beta", "lam", "S_init", "z_init", "dout", "dS_final", "x", "w", "b", "dy",
          "kpm"}
FILES = ["delta_tc.cuh", "delta_bwd_tc.cuh", "norm.cuh", "causal_seg_tc.cuh", "causal_bwd_tc.cuh",
         "global_tc.cuh"]


def kernels(text):
    """(name, parameters, body) of every __global__ function, comments taken out."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__ void\s+(?:__launch_bounds__\([^{;]*?\)\s+)?(\w+)\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        params, start = text[m.end():at - 1], text.index("{", at)
        depth, end = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), params, text[start:end]


@pytest.mark.parametrize("name", FILES)
def test_what_an_overlapped_kernel_reads_is_not_declared_constant(name):
    with open(os.path.join(CSRC, name)) as f:
        found = list(kernels(f.read()))
    waiting = [x for x in found if "grid_dependency_wait" in x[2] or "run<" in x[2]]
    assert waiting, f"no kernel of {name} waits for the grid before it"
    for kernel, params, _ in waiting:
        constant = set(re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", params))
        assert constant <= INPUTS, f"{kernel}: {sorted(constant - INPUTS)}"


def test_every_kernel_is_looked_at():
    names = {k for p in glob.glob(os.path.join(CSRC, "*.cuh")) for k, _, _ in kernels(open(p).read())}
    assert {"delta_prep_kernel", "delta_chain_kernel", "delta_carry_kernel", "delta_sweep_kernel",
            "delta_grad_kernel", "norm_bwd_sum_kernel"} <= names

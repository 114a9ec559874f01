"""Refusals of the delta-rule and norm helpers that allocate (no GPU needed: each is refused before
anything is allocated or launched)."""
import pytest
import torch

from weight_state_recurrence_b200 import linattn


def T(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def test_axes_of_q():
    b = T(2, 4, dtype=torch.float32)
    for q in (T(2, 4, 64), T(1, 1, 2, 4, 64)):
        with pytest.raises(ValueError):
            linattn.delta_fwd(q, q, q, None, b)
        with pytest.raises(ValueError):
            linattn.delta_bwd(q, q, q, None, b, q)


def test_beta_is_required():
    q = T(1, 2, 4, 64)
    with pytest.raises(ValueError, match="beta"):
        linattn.delta_bwd(q, q, q, None, None, q)


def test_a_norm_needs_an_axis():
    x = torch.tensor(1.0)
    with pytest.raises(ValueError):
        linattn.norm_fwd(x)
    with pytest.raises(ValueError):
        linattn.norm_bwd(x, None, x)

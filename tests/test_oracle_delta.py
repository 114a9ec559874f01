"""Pins of the delta-rule and row-norm oracle (CPU)."""
import math

import pytest
import torch

from oracle import delta as od

F = torch.float64


def case(seed, B, H, N, dk, dv, gate=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=F)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q, k, v = unit(r(B, H, N, dk)), unit(r(B, H, N, dk)), r(B, H, N, dv)
    g = -torch.exp(r(B, H, N) - 2) if gate else None
    return q, k, v, g, torch.sigmoid(r(B, H, N)), 0.3 * r(B, H, dk, dv)


def test_worked_example():
    # dk = 2, dv = 1, a = 1/2, beta = 1: orthonormal keys, then the first key again
    k = torch.tensor([[[[1., 0.], [0., 1.], [1., 0.]]]], dtype=F)
    v = torch.tensor([[[[8.], [4.], [6.]]]], dtype=F)
    q = torch.ones_like(k)
    g = torch.full((1, 1, 3), -math.log(2.0), dtype=F)
    out, S = od.delta(q, k, v, g, torch.ones(1, 1, 3, dtype=F))
    # S: (8, 0) -> (4, 4) -> (2 + (6 - 2), 2)
    assert out.flatten().tolist() == pytest.approx([8.0, 8.0, 8.0])
    assert S.flatten().tolist() == pytest.approx([6.0, 2.0])


def test_a_full_write_is_read_back():
    # beta = 1 and a unit key: the state returns v for that key
    q, k, v, g, beta, S0 = case(1, 1, 2, 7, 8, 4)
    out, _ = od.delta(k, k, v, g, torch.ones_like(beta), S0)
    torch.testing.assert_close(out, v)


def test_no_write_keeps_the_state_and_minus_infinity_clears_it():
    q, k, v, g, beta, S0 = case(2, 1, 1, 5, 4, 4)
    out, S = od.delta(q, k, v, None, torch.zeros_like(beta), S0)
    torch.testing.assert_close(S, S0)
    g = g.clone()
    g[0, 0, 3] = -math.inf
    a, _ = od.delta(q, k, v, g, beta, S0)
    b, _ = od.delta(q[:, :, 3:4], k[:, :, 3:4], v[:, :, 3:4], None, beta[:, :, 3:4])
    assert torch.isfinite(a).all()
    torch.testing.assert_close(a[:, :, 3], b[:, :, 0])


def test_split_sequence_continues():
    q, k, v, g, beta, S0 = case(3, 2, 2, 9, 8, 16)
    out, S = od.delta(q, k, v, g, beta, S0)
    o1, S1 = od.delta(q[:, :, :4], k[:, :, :4], v[:, :, :4], g[:, :, :4], beta[:, :, :4], S0)
    o2, S2 = od.delta(q[:, :, 4:], k[:, :, 4:], v[:, :, 4:], g[:, :, 4:], beta[:, :, 4:], S1)
    torch.testing.assert_close(torch.cat([o1, o2], 2), out)
    torch.testing.assert_close(S2, S)


def test_gradients_by_central_differences():
    args = list(case(4, 1, 1, 5, 4, 3))
    gen = torch.Generator().manual_seed(9)
    do = torch.randn(1, 1, 5, 3, generator=gen, dtype=F)
    dS = torch.randn(1, 1, 4, 3, generator=gen, dtype=F)
    q, k, v, g, beta, S0 = args
    got = od.delta_grad(q, k, v, g, beta, do, S0, dS)

    def loss(*a):
        out, S = od.delta(*a)
        return float((out * do).sum() + (S * dS).sum())

    for n, x in enumerate(args):
        want = torch.zeros_like(x)
        for e in range(x.numel()):
            h = 1e-6
            up, dn = x.clone(), x.clone()
            up.view(-1)[e] += h
            dn.view(-1)[e] -= h
            a, b = list(args), list(args)
            a[n], b[n] = up, dn
            want.view(-1)[e] = (loss(*a) - loss(*b)) / (2 * h)
        name = ("dq", "dk", "dv", "dg", "dbeta", "dS")[n]
        torch.testing.assert_close(got[name], want, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_by_central_differences(rms):
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(3, 6, generator=gen, dtype=F) + 0.5
    w = torch.randn(6, generator=gen, dtype=F)
    dy = torch.randn(3, 6, generator=gen, dtype=F)
    y = od.norm(x, w, None, 1e-3, rms)
    if not rms:
        torch.testing.assert_close((y / w).mean(-1), torch.zeros(3, dtype=F), atol=1e-12, rtol=0)
    dx, dw, db = od.norm_grad(x, w, dy, 1e-3, rms)
    torch.testing.assert_close(db, dy.sum(0))
    for t, want in ((x, dx), (w, dw)):
        for e in range(t.numel()):
            h = 1e-6
            up, dn = t.clone(), t.clone()
            up.view(-1)[e] += h
            dn.view(-1)[e] -= h
            f = lambda s: float((od.norm(s if t is x else x, w if t is x else s, None, 1e-3, rms)
                                 * dy).sum())
            assert (f(up) - f(dn)) / (2 * h) == pytest.approx(float(want.view(-1)[e]), rel=1e-6,
                                                              abs=1e-8)

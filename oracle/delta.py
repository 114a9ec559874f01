"""Gated delta rule and row norm oracle (torch float64, any device).

TEST INFRASTRUCTURE ONLY, under the same rule as the rest of ``oracle/``:
only ``tests/`` and ``__graft_entry__.smoke()`` may use it; the product never
imports it, and this module imports nothing from the product.

The rule is written token by token, as it is defined:

    r_i = v_i - a_i S_{i-1}^T k_i,  S_i = a_i S_{i-1} + k_i (beta_i r_i)^T,
    o_i = S_i^T q_i,                a_i = exp(g_i),

and its gradients come from autograd on those lines.  The tests pin the
forward by a worked example and by properties of the rule, the gradients by
central differences.
"""
from __future__ import annotations

import torch


def _f64(x, like=None):
    return None if x is None else x.detach().to(torch.float64)


def _walk(q, k, v, g, beta, S):
    outs = []
    for i in range(q.shape[2]):
        if g is not None:
            S = S * torch.exp(g[:, :, i])[..., None, None]
        r = v[:, :, i] - (S * k[:, :, i, :, None]).sum(-2)
        S = S + k[:, :, i, :, None] * (beta[:, :, i, None] * r)[..., None, :]
        outs.append((S * q[:, :, i, :, None]).sum(-2))
    out = torch.stack(outs, 2) if outs else v.new_zeros(v.shape)
    return out, S


def _start(q, v, S_init):
    B, H, _, dk = q.shape
    if S_init is not None:
        return _f64(S_init)
    return torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device=q.device)


def delta(q, k, v, g, beta, S_init=None):
    """(out [B,H,N,dv], S_final [B,H,dk,dv]) in float64."""
    return _walk(_f64(q), _f64(k), _f64(v), _f64(g), _f64(beta), _start(q, v, S_init))


def delta_grad(q, k, v, g, beta, dout, S_init=None, dS_final=None):
    """Gradients of sum(dout out) + sum(dS_final S_final) as a dict of float64
    tensors: dq, dk, dv, dg (at g = 0 when g is None), dbeta, dS."""
    if g is None:
        g = torch.zeros_like(beta)
    leaf = [_f64(t).clone().requires_grad_(True) for t in (q, k, v, g, beta)]
    S0 = _start(q, v, S_init).clone().requires_grad_(True)
    out, S = _walk(*leaf, S0)
    loss = (out * _f64(dout)).sum()
    if dS_final is not None:
        loss = loss + (S * _f64(dS_final)).sum()
    got = torch.autograd.grad(loss, leaf + [S0], allow_unused=True)
    got = [torch.zeros_like(x) if y is None else y for x, y in zip(leaf + [S0], got)]
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dS"), got))


def norm(x, weight=None, bias=None, eps=1e-5, rms=False):
    """Row norm over the last axis in float64."""
    x = _f64(x)
    m = torch.zeros_like(x[..., :1]) if rms else x.mean(-1, keepdim=True)
    y = (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * _f64(weight)
    return y if bias is None else y + _f64(bias)


def norm_grad(x, weight, dy, eps=1e-5, rms=False):
    """(dx, dweight, dbias) in float64; dweight is the gradient at 1 without a weight."""
    xl = _f64(x).clone().requires_grad_(True)
    d = x.shape[-1]
    w = torch.ones(d, dtype=torch.float64, device=x.device) if weight is None else _f64(weight)
    w = w.clone().requires_grad_(True)
    m = torch.zeros_like(xl[..., :1]) if rms else xl.mean(-1, keepdim=True)
    y = (xl - m) / torch.sqrt(((xl - m) ** 2).mean(-1, keepdim=True) + eps) * w
    dx, dw = torch.autograd.grad((y * _f64(dy)).sum(), (xl, w))
    return dx, dw, _f64(dy).reshape(-1, d).sum(0)

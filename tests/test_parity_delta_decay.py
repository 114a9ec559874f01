"""GPU parity of the gated delta rule under one slow gate for all tokens.

A decay that is rounded to fp32 is off by up to 2^-25, and by the same 2^-25 at every token when the gate
stays the same: over N tokens that is N 2^-25 of the state.  The gates here are such that exp(g), or exp(64 g) for
a chunk of 64 tokens, lies in the middle between two fp32 numbers.

Tolerances, derived.  With beta = 0 the state only decays, S_N = exp(g N) S_0, by x <- x + l x, l = exp(g) - 1,
each time rounded to a multiple of u, the step of fp32 at x.  The roundings of one x do not add in
quadrature: l x / u, whose fraction is rounded off, itself changes by l^2 x / u a token only (0.0058 just below
1), so the roundings run through saw teeth.  A whole tooth sums to 0 up to one half step; of a
part of one there is at most 1 / 8 of its length, u / (8 l^2 x) steps.  Relative to x:
  part of a tooth  u^2 / (8 l^2 x^2),  u / x at most 2^-23: 2^-49 / g^2; twice, where the walk crosses a power of 2
  whole teeth      N l^2 x / u of them, a half step each: N g^2 2^24 times 2^-24 at most.
Segments join by M, which starts at 1 and stays near it, so that u / x is 2^-24 / M and all of them have the same
error: with M > 0.97 a part of a tooth is 2^-51 / (0.97 g)^2, and there are at most 32 segments.  What is left of the
decay's own rounding is relative to l: N |g| 2^-23.  All of it together stays well below N 2^-25.
"""
import math

import pytest
import torch

from oracle import delta as od
from test_parity_delta import BF, DEV, F32, make, rel, tol_out, tol_state

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SLOW, SLOW64 = -1.8626629753271118e-05, -1.932618033606559e-05   # off by 2.98e-8 below


def test_the_gates_are_what_they_are_for():
    for n, g in ((1, SLOW), (64, SLOW64)):
        e = math.exp(n * g)
        assert abs(float(torch.tensor(e, dtype=torch.float64).float()) - e) > 0.99 * 2.0 ** -25 * e


def still(seed, B, H, N, dk, dv, dtype, g):
    q, k, v, _, beta, S0 = make(seed, B, H, N, dk, dv, dtype)
    return q, k, v, torch.full_like(beta, g), torch.zeros_like(beta), S0


def tol(N, segments):
    part, teeth, rest = 2.0 ** -49 / SLOW ** 2, N * SLOW ** 2, N * abs(SLOW) * 2.0 ** -23
    joined = 2.0 ** -51 / (0.97 * SLOW) ** 2 if segments else 0.0
    t = 2 * part + teeth + rest + 32 * joined
    assert t < 0.5 * N * 2.0 ** -25
    return t


@pytest.mark.parametrize("BH,N,dk,dv", [((1, 2), 8192, 16, 16), ((1, 3), 8001, 64, 32), ((5, 31), 4096, 32, 16)])
def test_cuda_cores(cuda_lib, BH, N, dk, dv):
    q, k, v, g, beta, S0 = still(1, *BH, N, dk, dv, F32, SLOW)
    want, t = math.exp(N * float(g[0, 0, 0])) * S0.double(), tol(N, BH[0] * BH[1] < 100)
    _, S = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    assert rel(S, want) <= tol(N, False)
    got = cuda_lib.delta_bwd(q, k, v, g, beta, torch.zeros_like(v), S0, S0, want_dS_init=True)
    assert rel(got[5], want) <= t


def test_cuda_cores_with_writes(cuda_lib):
    q, k, v, g, beta, S0 = still(2, 1, 4, 4096, 16, 16, F32, SLOW)
    beta += 1e-3
    out, S = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    o_w, S_w = od.delta(q, k, v, g, beta, S0)
    assert rel(out, o_w) <= tol_out(F32, 4096, 16) and rel(S, S_w) <= tol_state(F32, 4096, 16)


@pytest.mark.parametrize("g", [-0.7, -4.0])
@pytest.mark.parametrize("dk,dv", [(16, 16), (64, 32)])
def test_strong_gates_on_cuda_cores(cuda_lib, g, dk, dv):
    # what is left of the state is as exact, relative to itself, as exp's two steps of 2^-23 and a rounding a token
    N = 20
    q, k, v, gate, beta, S0 = still(4, 1, 2, N, dk, dv, F32, g)
    want = math.exp(N * float(gate[0, 0, 0])) * S0.double()
    _, S = cuda_lib.delta_fwd(q, k, v, gate, beta, S0)
    assert rel(S, want) <= N * (4 + 1) * U
    got = cuda_lib.delta_bwd(q, k, v, gate, beta, torch.zeros_like(v), S0, S0, want_dS_init=True)
    assert rel(got[5], want) <= N * (4 + 1) * U


def test_single_tokens(cuda_lib):
    q, k, v, _, beta, S0 = make(3, 2, 3, 0, 64, 32, F32, lead3=False)
    # a slow gate over many tokens, and a strong one whose remainder is as exact as exp
    for N, g, t in ((6000, SLOW, tol(6000, False)), (20, -4.0, 20 * (4 + 1) * U)):
        gate, S = torch.full_like(beta, g), S0.clone()
        for _ in range(N):
            cuda_lib.delta_step(q, k, v, gate, torch.zeros_like(beta), S)
        assert rel(S, math.exp(N * float(gate[0, 0])) * S0.double()) <= t


def tol_chunks(N, segments):
    """The same for a decay a chunk of 64 tokens.  Here l^2 x / u is 25 a chunk and more: what is rounded off
    jumps about, and n roundings of at most 2^-24 add in quadrature, taken twice over.  Segments share M's."""
    n = N // 64
    t = 2 * math.sqrt(n * segments) * U + 2 * N * abs(SLOW64) * 2.0 ** -24
    assert t < 0.5 * n * 2.0 ** -25
    return t


@pytest.mark.parametrize("BH,N,segments", [((4, 37), 16384, 1), ((1, 2), 1 << 18, 38)])
def test_tensor_cores(cuda_lib, BH, N, segments):
    q, k, v, g, beta, S0 = still(5, *BH, N, 64, 64, BF, SLOW64)
    _, S = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    assert rel(S, math.exp(N * float(g[0, 0, 0])) * S0.double()) <= tol_chunks(N, segments)


@pytest.mark.parametrize("d", [64, 128])
def test_tensor_core_gradient(cuda_lib, d):
    q, k, v, g, beta, S0 = still(6, 2, 3, 16384, d, d, BF, SLOW64)
    got = cuda_lib.delta_bwd(q, k, v, g, beta, torch.zeros_like(v), S0, S0, want_dS_init=True)
    assert rel(got[5], math.exp(16384 * float(g[0, 0, 0])) * S0.double()) <= tol_chunks(16384, 1)


@pytest.mark.parametrize("g", [-0.02, -0.25])
def test_strong_gates_on_tensor_cores(cuda_lib, g):
    # a chunk's decay of a quarter, and of 1e-7: as exact as exp's two steps of 2^-23, the rounding of its argument
    # and one of the product
    N = 256
    q, k, v, gate, beta, S0 = still(7, 1, 3, N, 128, 128, BF, g)
    want = math.exp(N * float(gate[0, 0, 0])) * S0.double()
    _, S = cuda_lib.delta_fwd(q, k, v, gate, beta, S0)
    t = N // 64 * (4 + 1 + 64 * abs(g)) * U
    assert rel(S, want) <= t
    got = cuda_lib.delta_bwd(q, k, v, gate, beta, torch.zeros_like(v), S0, S0, want_dS_init=True)
    assert rel(got[5], want) <= t

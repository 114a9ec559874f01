"""GPU parity of the gated delta rule against the fp64 oracle.

Tolerances, derived.  Every error is taken relative to the scale of what it
sits in, by the 2-norm of a tensor's difference over the 2-norm of the tensor.

* A result rounded to bf16 is off by at most 2^-8 of each value: OUT_BF16.
* fp32 arithmetic: a reduction over dk and a handful of roundings a token give
  at most (dk + 4) 2^-24 of the state's column norm (unit keys,
  Cauchy-Schwarz); the recurrence does not amplify (|I - beta k k^T| <= 1), and
  the errors of N tokens add as independent ones: (dk + 4) 2^-24 sqrt(N).
* Where the matrix units run, an fp32 operand enters them as a pair of bf16
  values, which leaves 2^-16 of it; at most six such operands stand between a
  token's inputs and an output, once a chunk of 64 tokens:
  6 * 2^-16 sqrt(N / 64 + 1).
* The gradients add the reverse recurrence to the forward one: twice that.  dg
  is a sum over token pairs whose parts are one order above it: 8 times.
"""
import math

import pytest
import torch

from oracle import delta as od

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def rel(got, want):
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def tol_state(dtype, N, dk):
    t = (dk + 4) * 2.0 ** -24 * math.sqrt(N)
    return t + (6 * 2.0 ** -16 * math.sqrt(N / 64 + 1) if dtype == BF else 0.0)


def tol_out(dtype, N, dk):
    return tol_state(dtype, N, dk) + (2.0 ** -8 if dtype == BF else 0.0)


def make(seed, B, H, N, dk, dv, dtype, gate="soft", lead3=True, dev=DEV):
    gen = torch.Generator(device=dev).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)
    lead = (B, H, N) if lead3 else (B, H)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)
    q = (unit(r(*lead, dk)) * dk ** -0.5).to(dtype)
    k = unit(r(*lead, dk) + 0.5 * r(B, H, *([1] * (len(lead) - 2)), dk)).to(dtype)
    v = r(*lead, dv).to(dtype)
    beta = torch.sigmoid(r(*lead))
    g = None
    if gate != "none":
        g = -torch.exp(1.5 * r(*lead) + (0.0 if gate == "hard" else -4.0))
    if gate == "reset":
        g = torch.where(torch.rand(lead, generator=gen, device=dev) < 0.05,
                        torch.full_like(g, -math.inf), g)
    return q, k, v, g, beta, 0.2 * r(B, H, dk, dv)


LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 128, 200, 321]
DIMS = [(16, 16), (16, 128), (32, 64), (64, 32), (64, 64), (64, 128), (128, 16), (128, 64), (128, 128)]


def check_fwd(lib, a, state):
    q, k, v, g, beta, S0 = a
    N, dk = q.shape[2], q.shape[3]
    S0 = S0 if state else None
    out, S = lib.delta_fwd(q, k, v, g, beta, S0)
    o_w, S_w = od.delta(q, k, v, g, beta, S0)
    assert rel(out, o_w) <= tol_out(q.dtype, N, dk)
    assert rel(S, S_w) <= tol_state(q.dtype, N, dk)
    only, none = lib.delta_fwd(q, k, v, g, beta, S0, want_state=False)
    assert none is None and torch.equal(only, out)
    assert lib.linattn_device_status() == 0


@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_forward_lengths(cuda_lib, N, dtype):
    check_fwd(cuda_lib, make(N, 2, 3, N, 128, 128, dtype), N % 2 == 0)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_forward_head_sizes(cuda_lib, dk, dv, dtype):
    check_fwd(cuda_lib, make(dk + dv, 1, 3, 150, dk, dv, dtype), True)


@pytest.mark.parametrize("gate", ["none", "soft", "hard", "reset"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_gates(cuda_lib, gate, dtype, d):
    check_fwd(cuda_lib, make(7, 2, 2, 300, d, d, dtype, gate), True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_forward_many_heads(cuda_lib, dtype):
    check_fwd(cuda_lib, make(11, 5, 67, 70, 64, 64, dtype), False)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_forward_on_cuda_cores(cuda_lib, dk, dv):
    # bf16 on the family that every other type and size runs on
    with cuda_lib.kernel_choice(cuda_lib.LINATTN_OP_DELTA, cuda_lib.LINATTN_KERNEL_CUDA_CORES):
        check_fwd(cuda_lib, make(8, 2, 2, 150, dk, dv, BF), True)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_cuda_cores_with_more_heads_than_multiprocessors(cuda_lib, dk, dv, dtype):
    with cuda_lib.kernel_choice(cuda_lib.LINATTN_OP_DELTA, cuda_lib.LINATTN_KERNEL_CUDA_CORES):
        check_fwd(cuda_lib, make(13, 5, 31, 45, dk, dv, dtype, "reset"), True)
        check_bwd(cuda_lib, 14, 5, 31, 45, dk, dv, dtype, "soft", True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_sequence(cuda_lib, dtype):
    check_fwd(cuda_lib, make(12, 1, 2, 4001, 128, 128, dtype), False)


@pytest.mark.parametrize("BH,N", [((1, 7), 15000), ((2, 37), 2047), ((3, 37), 1279), ((3, 37), 2300),
                                  ((4, 37), 700)])
def test_two_slabs(cuda_lib, BH, N):
    # where the heads leave SMs free a long enough sequence is worked on in two
    # pieces, the second one's records made beside the first one's chain
    check_fwd(cuda_lib, make(N, *BH, N, 64, 64, BF), N % 2 == 0)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_repeated_keys_and_full_writes(cuda_lib, dtype):
    # every key the same and beta = 1: the solve inside a chunk at its worst
    # (each token overwrites what the one before wrote)
    q, k, v, _, beta, S0 = make(13, 1, 2, 130, 128, 128, dtype)
    k = k[:, :, :1].expand_as(k).contiguous()
    check_fwd(cuda_lib, (q, k, v, None, torch.ones_like(beta), S0), True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_writes_past_the_target(cuda_lib, dtype):
    # beta above 1 turns the old value round (1 - beta |k|^2 near -0.9), with
    # repeated keys at every second token
    q, k, v, _, beta, S0 = make(16, 1, 2, 140, 128, 128, dtype)
    k[:, :, ::2] = k[:, :, :1]
    check_fwd(cuda_lib, (q, k, v, None, torch.full_like(beta, 1.9), S0), True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gates_above_zero(cuda_lib, dtype):
    # outside what the rule is for, but used as given
    q, k, v, g, beta, S0 = make(17, 1, 2, 140, 64, 64, dtype)
    check_fwd(cuda_lib, (q, k, v, (0.02 * torch.randn_like(g)).contiguous(), beta, S0), True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_nan_stays_in_its_head(cuda_lib, dtype):
    for which in range(5):
        a = list(make(18, 1, 3, 100, 128, 128, dtype))
        ref = cuda_lib.delta_fwd(*a)
        a[which] = a[which].clone()
        a[which][0, 1, 70] = float("nan")
        out, S = cuda_lib.delta_fwd(*a)
        assert torch.equal(out[:, ::2], ref[0][:, ::2]) and torch.equal(S[:, ::2], ref[1][:, ::2])
        assert out[0, 1, 70].isnan().all()
        if which > 0:      # not q: what it reaches, it reaches for good
            assert S[0, 1].isnan().any() and out[0, 1, 99].isnan().any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_padding_tokens_leave_the_state(cuda_lib, dtype):
    q, k, v, g, beta, S0 = make(14, 2, 2, 96, 128, 128, dtype)
    beta[:, :, 50:], g[:, :, 50:] = 0, 0
    _, S = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    cut = lambda x: x[:, :, :50].contiguous()
    _, S50 = cuda_lib.delta_fwd(cut(q), cut(k), cut(v), cut(g), cut(beta), S0)
    t = tol_state(dtype, 96, 128)
    assert rel(S, S50) <= 2 * t


def test_empty_sequence_copies_the_state(cuda_lib):
    q, k, v, g, beta, S0 = make(15, 1, 2, 0, 64, 32, F32)
    out, S = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    assert out.shape == (1, 2, 0, 32) and torch.equal(S, S0)
    _, S = cuda_lib.delta_fwd(q, k, v, g, beta)
    assert not S.any()
    dS = torch.randn_like(S0)
    got = cuda_lib.delta_bwd(q, k, v, g, beta, torch.empty_like(v), S0, dS, want_dS_init=True)
    assert torch.equal(got[5], dS)


# ------------------------------------------------------------ single tokens
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", ["none", "soft", "reset"])
def test_step(cuda_lib, dk, dv, dtype, gate):
    for B, H in ((1, 1), (3, 5), (40, 16)):
        q, k, v, g, beta, S0 = make(B, B, H, 0, dk, dv, dtype, gate, lead3=False)
        one = lambda x: None if x is None else x.unsqueeze(2)
        o_w, S_w = od.delta(one(q), one(k), one(v), one(g), one(beta), S0)
        S = S0.clone()
        out = cuda_lib.delta_step(q, k, v, g, beta, S)
        assert rel(out, o_w[:, :, 0]) <= tol_out(F32, 1, dk) + (2.0 ** -8 if dtype == BF else 0)
        assert rel(S, S_w) <= tol_out(F32, 1, dk)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_then_steps_equal_one_call(cuda_lib, dtype):
    q, k, v, g, beta, S0 = make(21, 2, 4, 100, 128, 128, dtype)
    out, S_all = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    cut = lambda x, a, b: x[:, :, a:b].contiguous()
    o1, S = cuda_lib.delta_fwd(*(cut(x, 0, 90) for x in (q, k, v, g, beta)), S0)
    o = [o1]
    for i in range(90, 100):
        at = lambda x: x[:, :, i].contiguous()
        o.append(cuda_lib.delta_step(at(q), at(k), at(v), at(g), at(beta), S).unsqueeze(2))
    assert rel(torch.cat(o, 2), out) <= 2 * tol_out(dtype, 100, 128)
    assert rel(S, S_all) <= 2 * tol_state(dtype, 100, 128)


# ------------------------------------------------------------ backward
def check_bwd(lib, seed, B, H, N, dk, dv, dtype, gate, state):
    q, k, v, g, beta, S0 = make(seed, B, H, N, dk, dv, dtype, gate)
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    do = torch.randn(B, H, N, dv, generator=gen, device=DEV).to(dtype)
    S0, dS = (S0, 0.3 * torch.randn(B, H, dk, dv, generator=gen, device=DEV)) if state else (None, None)
    got = dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dS"),
                   lib.delta_bwd(q, k, v, g, beta, do, S0, dS, want_dS_init=True)))
    want = od.delta_grad(q, k, v, g, beta, do, S0, dS)
    again = lib.delta_bwd(q, k, v, g, beta, do, S0, dS, want_dS_init=True)
    for x, y in zip(got.values(), again):
        assert (x is None and y is None) or torch.equal(x, y)
    for n in ("dq", "dk", "dv"):
        assert rel(got[n], want[n]) <= 2 * tol_out(dtype, N, dk), n
    for n in ("dbeta", "dS"):
        assert rel(got[n], want[n]) <= 2 * tol_state(dtype, N, dk), n
    if g is None:
        assert got["dg"] is None
    else:
        # a head whose first gate is a reset passes nothing to g: absolute there
        assert rel(got["dg"], want["dg"]) <= 8 * tol_state(dtype, N, dk)
    assert lib.linattn_device_status() == 0


@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_backward_lengths(cuda_lib, N, dtype):
    # one token alone has no token pair: its dg is what S_init hands on
    check_bwd(cuda_lib, N, 1, 3, N, 128, 128, dtype, "soft", N % 2 == 1)


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_backward_head_sizes(cuda_lib, dk, dv, dtype):
    check_bwd(cuda_lib, dk * dv, 2, 2, 100, dk, dv, dtype, "soft", True)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_backward_on_cuda_cores(cuda_lib, dk, dv):
    with cuda_lib.kernel_choice(cuda_lib.LINATTN_OP_DELTA, cuda_lib.LINATTN_KERNEL_CUDA_CORES):
        check_bwd(cuda_lib, dk + dv, 2, 2, 100, dk, dv, BF, "soft", True)


@pytest.mark.parametrize("gate", ["none", "soft", "hard", "reset"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("state", [False, True])
def test_backward_gates(cuda_lib, gate, dtype, state):
    check_bwd(cuda_lib, 31, 1, 4, 200, 128, 128, dtype, gate, state)


def test_gradient_of_an_absent_gate_is_the_one_at_zero(cuda_lib):
    q, k, v, _, beta, S0 = make(33, 1, 2, 70, 64, 64, F32, "none")
    do = torch.randn_like(v)
    dg, ws = torch.empty_like(beta), torch.empty(
        cuda_lib.linattn_delta_bwd_workspace(1, 2, 70, 64, 64, F32), dtype=torch.uint8, device=DEV)
    dq, dk, dv, db = (torch.empty_like(x) for x in (q, k, v, beta))
    cuda_lib.linattn_delta_bwd(q, k, v, None, beta, S0, do, None, dq, dk, dv, dg, db, None, ws)
    want = od.delta_grad(q, k, v, None, beta, do, S0)
    assert rel(dg, want["dg"]) <= 8 * tol_state(F32, 70, 64)
    dq2 = torch.empty_like(dq)
    cuda_lib.linattn_delta_bwd(q, k, v, torch.zeros_like(beta), beta, S0, do, None, dq2, dk, dv, None,
                               db, None, ws)
    assert torch.equal(dq, dq2)


def test_gradient_against_differences(cuda_lib):
    # fp32: the loss moves along a random direction as the gradient says
    q, k, v, g, beta, S0 = make(34, 1, 2, 90, 64, 64, F32)
    do, dS = torch.randn_like(v), torch.randn_like(S0)
    got = cuda_lib.delta_bwd(q, k, v, g, beta, do, S0, dS, want_dS_init=True)
    args = [q, k, v, g, beta, S0]
    dirs = [torch.randn_like(x) * x.abs().mean() for x in args]
    # central differences of the fp64 oracle along it: error h^2, far below the tolerance
    h = 1e-4
    f = lambda sgn: (lambda o, S: float((o * do.double()).sum() + (S * dS.double()).sum()))(
        *od.delta(*(x.double() + sgn * h * y.double() for x, y in zip(args, dirs))))
    want = (f(1) - f(-1)) / (2 * h)
    have = sum(float((x.double() * y.double()).sum()) for x, y in zip(got, dirs))
    size = sum(float(x.double().norm() * y.double().norm()) for x, y in zip(got, dirs))
    assert abs(have - want) <= 8 * tol_state(F32, 90, 64) * size + 1e-5 * abs(want)


# ------------------------------------------------------------ how calls are made
def test_streams_and_graph_capture(cuda_lib):
    q, k, v, g, beta, S0 = make(41, 2, 2, 130, 128, 128, BF)
    do = torch.randn(v.shape, device=DEV).to(BF)
    want = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    grads = cuda_lib.delta_bwd(q, k, v, g, beta, do, S0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, S = torch.empty_like(v), torch.empty_like(S0)
    wf = torch.empty(cuda_lib.linattn_delta_fwd_workspace(2, 2, 130, 128, 128, BF),
                     dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    cuda_lib.linattn_delta_fwd(q, k, v, g, beta, S0, out, S, wf, side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(S, want[1])
    # captured: forward, a step from its state, and the backward
    at = lambda x: x[:, :, 0].contiguous()
    qs, ks, vs, gs, bs = (at(x) for x in (q, k, v, g, beta))
    ws = torch.empty(cuda_lib.linattn_delta_bwd_workspace(2, 2, 130, 128, 128, BF),
                     dtype=torch.uint8, device=DEV)
    bufs = [torch.empty_like(x) for x in (q, k, v, g, beta)]
    so = torch.empty_like(vs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.linattn_delta_fwd(q, k, v, g, beta, S0, out, S, wf)
        cuda_lib.linattn_delta_step(qs, ks, vs, gs, bs, S, so)
        cuda_lib.linattn_delta_bwd(q, k, v, g, beta, S0, do, None, *bufs, None, ws)
    out.zero_()
    S.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    ref = want[1].clone()
    so_ref = cuda_lib.delta_step(qs, ks, vs, gs, bs, ref)
    assert torch.equal(out, want[0]) and torch.equal(S, ref) and torch.equal(so, so_ref)
    for x, y in zip(bufs, grads):
        assert torch.equal(x, y)


@pytest.mark.parametrize("BH,N,dk,dv", [((1, 1), 512, 128, 128), ((1, 1), 4001, 128, 128),
                                        ((2, 8), 4093, 64, 64), ((1, 16), 2000, 64, 128),
                                        ((3, 5), 1999, 128, 64), ((2, 16), 3001, 128, 128),
                                        ((1, 33), 5000, 64, 64), ((3, 8), 6073, 128, 128),
                                        ((4, 9), 3067, 64, 128)])
@pytest.mark.parametrize("gate", ["soft", "reset", "none"])
def test_segments(cuda_lib, BH, N, dk, dv, gate):
    # few heads: segments of the sequence side by side, joined by their transitions
    a = make(N + dk, *BH, N, dk, dv, BF, gate)
    check_fwd(cuda_lib, a, gate != "none")


def test_two_slabs_captured_and_beside_another_call(cuda_lib):
    pieces(cuda_lib, 2, 37, 2000)


def test_segments_captured_and_beside_another_call(cuda_lib):
    pieces(cuda_lib, 2, 4, 2000)


def test_segments_with_the_last_prepared_later(cuda_lib):
    # captured, and beside another call: its records are made beside the transitions
    pieces(cuda_lib, 2, 16, 3580)


def pieces(cuda_lib, B, H, N):
    a, b = make(46, B, H, N, 128, 128, BF), make(47, B, H, N, 128, 128, BF)
    want = [cuda_lib.delta_fwd(*x) for x in (a, b)]
    n = cuda_lib.linattn_delta_fwd_workspace(B, H, N, 128, 128, BF)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out = [(torch.empty_like(x[2]), torch.empty_like(x[5])) for x in (a, b)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cuda_lib.linattn_delta_fwd(*a, out[0][0], out[0][1], ws[0])
    cuda_lib.linattn_delta_fwd(*b, out[1][0], out[1][1], ws[1], side)
    graph.replay()
    cuda_lib.linattn_delta_fwd(*b, out[1][0], out[1][1], ws[1], side)
    graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(out, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert cuda_lib.linattn_device_status() == 0


def test_two_calls_at_once(cuda_lib):
    a, b = make(42, 4, 8, 500, 128, 128, BF), make(43, 4, 8, 500, 128, 128, BF)
    wa, wb = cuda_lib.delta_fwd(*a), cuda_lib.delta_fwd(*b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    ra = cuda_lib.delta_fwd(*a, stream=s1)
    rb = cuda_lib.delta_fwd(*b, stream=s2)
    torch.cuda.synchronize()
    for x, y in zip(wa + wb, ra + rb):
        assert torch.equal(x, y)


def test_nothing_is_written_behind_the_outputs(cuda_lib):
    # outputs in the middle of a larger buffer: what surrounds them stays
    q, k, v, g, beta, S0 = make(44, 1, 3, 77, 128, 64, BF)
    n = v.numel()
    big = torch.full((n + 4096,), 7.0, dtype=BF, device=DEV)
    out = big[2048:2048 + n].view(v.shape)
    ws = torch.empty(cuda_lib.linattn_delta_fwd_workspace(1, 3, 77, 128, 64, BF), dtype=torch.uint8,
                     device=DEV)
    cuda_lib.linattn_delta_fwd(q, k, v, g, beta, S0, out, None, ws)
    assert torch.equal(out, cuda_lib.delta_fwd(q, k, v, g, beta, S0)[0])
    assert (big[:2048] == 7).all() and (big[2048 + n:] == 7).all()


def test_a_layer_of_the_operators(cuda_lib):
    # norms and delta rule as a layer runs them, forward and backward
    B, H, N, d = 2, 4, 150, 128
    gen = torch.Generator(device=DEV).manual_seed(45)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)
    q, k, v = (r(B, H, N, d) for _ in range(3))
    g, beta = -torch.exp(r(B, H, N) - 3), torch.sigmoid(r(B, H, N))
    w, b, dy = 1 + 0.1 * r(d), 0.1 * r(d), r(B, H, N, d)
    out, S = cuda_lib.delta_attention(q, k, v, g, beta, w, b)
    unit = torch.full((d,), d ** -0.5, device=DEV)
    qn64, kn64 = (od.norm(x, unit * s, None, 1e-6, True) for x, s in ((q, d ** -0.5), (k, 1.0)))
    o64, S64 = od.delta(qn64, kn64, v, g, beta)
    t = tol_state(F32, N, d)
    # the norm divides by the read-out's size, row by row: a small row's error
    # grows by (rms of all rows / its own); 8 covers these inputs' rows
    assert rel(out, od.norm(o64, w, b)) <= 8 * t
    assert rel(S, S64) <= t
    L, R = cuda_lib.LINATTN_NORM_LAYER, cuda_lib.LINATTN_NORM_RMS
    qn = cuda_lib.norm_fwd(q, unit * d ** -0.5, None, 1e-6, R)
    kn = cuda_lib.norm_fwd(k, unit, None, 1e-6, R)
    o, _ = cuda_lib.delta_fwd(qn, kn, v, g, beta)
    do, dw, db = cuda_lib.norm_bwd(o, w, dy, 1e-5, L)
    dqn, dkn, dv, dg, dbeta, _ = cuda_lib.delta_bwd(qn, kn, v, g, beta, do)
    dq, _, _ = cuda_lib.norm_bwd(q, unit * d ** -0.5, dqn, 1e-6, R, False, False)
    dk, _, _ = cuda_lib.norm_bwd(k, unit, dkn, 1e-6, R, False, False)
    do64, dw64, db64 = od.norm_grad(o64, w, dy)
    want = od.delta_grad(qn64, kn64, v, g, beta, do64)
    for have, ref in ((dv, want["dv"]), (dbeta, want["dbeta"]), (dw, dw64), (db, db64),
                      (dq, od.norm_grad(q, unit * d ** -0.5, want["dq"], 1e-6, True)[0]),
                      (dk, od.norm_grad(k, unit, want["dk"], 1e-6, True)[0])):
        assert rel(have, ref) <= 16 * t
    assert rel(dg, want["dg"]) <= 64 * t


@pytest.mark.parametrize("BH,N,dk,dv", [((1, 1), 2000, 128, 128), ((1, 2), 1500, 16, 16),
                                        ((2, 3), 1025, 16, 128), ((1, 5), 993, 128, 16),
                                        ((2, 4), 1001, 64, 32), ((1, 3), 1700, 32, 64)])
@pytest.mark.parametrize("gate", ["soft", "reset", "none"])
def test_backward_on_cuda_cores_in_segments(cuda_lib, BH, N, dk, dv, gate):
    # few heads and many tokens: both recurrences in segments joined by their transitions
    check_bwd(cuda_lib, N + dk, *BH, N, dk, dv, F32, gate, gate != "none")

"""GPU parity of the gated delta rule on each way its host layer may cut a call, and at the sizes where
the tensor-core backward runs in earnest.

Which way a forward takes shows in the workspace it asks for: a record for every chunk of every head,
and behind them nothing (one piece), one state a head (two slabs), or the states and transitions of
segments.  Each test says which one it is for and fails when the call goes another way, so that a changed
plan cannot leave a path without its test.  The plans are those of a device with 148 multiprocessors.

Tolerances: as derived in test_parity_delta.py.  Heads do not meet: where two calls differ in the heads
beside one only, that head's results are equal bit by bit.
"""
import pytest
import torch

from oracle import delta as od
from test_parity_delta import (BF, DEV, F32, check_bwd, check_fwd, make, rel, tol_out, tol_state)

pytestmark = pytest.mark.gpu
CORES = ("LINATTN_OP_DELTA", "LINATTN_KERNEL_CUDA_CORES")


def on_cores(lib):
    return lib.kernel_choice(*(getattr(lib, x) for x in CORES))


def way(lib, B, H, N, dk, dv):
    """'one', 'slabs' or 'segments': how the bf16 forward of this shape is cut."""
    need = lambda b, h, n: lib.linattn_delta_fwd_workspace(b, h, n, dk, dv, BF)
    chunks = -(-N // 64)
    extra = need(B, H, N) - B * H * chunks * need(1, 1, 1)
    return {0: "one", B * H * dk * dv * 4: "slabs"}.get(extra, "segments")


def test_the_way_shows_in_the_workspace(cuda_lib):
    assert torch.cuda.get_device_properties(0).multi_processor_count == 148
    assert way(cuda_lib, 4, 37, 4096, 128, 128) == "one"        # a head to every multiprocessor
    assert way(cuda_lib, 1, 8, 4096, 128, 128) == "segments"
    assert way(cuda_lib, 4, 16, 4096, 128, 128) == "slabs"


# heads, tokens, sizes; the odd lengths end inside a chunk, 2561 with a chunk of one token
SLABS = [((4, 16), 4095, 128, 128), ((1, 64), 2500, 64, 64), ((2, 33), 2561, 64, 128),
         ((2, 37), 2999, 128, 64), ((3, 32), 3000, 64, 64), ((1, 50), 3007, 128, 128)]


@pytest.mark.parametrize("BH,N,dk,dv", SLABS)
@pytest.mark.parametrize("gate,state", [("soft", True), ("reset", False), ("none", True)])
def test_two_slabs(cuda_lib, BH, N, dk, dv, gate, state):
    assert way(cuda_lib, *BH, N, dk, dv) == "slabs"
    check_fwd(cuda_lib, make(N + dv, *BH, N, dk, dv, BF, gate), state)


@pytest.mark.parametrize("B,H,N,kind", [(2, 32, 3001, "slabs"), (2, 37, 2999, "slabs"),
                                        (2, 4, 2000, "segments"), (2, 16, 3580, "segments")])
def test_captured_and_beside_another_call(cuda_lib, B, H, N, kind):
    # two calls, a workspace each: one captured, the other on a stream of its own; replayed twice
    assert way(cuda_lib, B, H, N, 128, 128) == kind
    a, b = make(51, B, H, N, 128, 128, BF), make(52, B, H, N, 128, 128, BF)
    want = [cuda_lib.delta_fwd(*x) for x in (a, b)]
    n = cuda_lib.linattn_delta_fwd_workspace(B, H, N, 128, 128, BF)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out = [(torch.empty_like(x[2]), torch.empty_like(x[5])) for x in (a, b)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cuda_lib.linattn_delta_fwd(*a, out[0][0], out[0][1], ws[0])
    for _ in range(2):
        cuda_lib.linattn_delta_fwd(*b, out[1][0], out[1][1], ws[1], side)
        graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(out, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert cuda_lib.linattn_device_status() == 0


@pytest.mark.parametrize("BH,N,kind", [((2, 32), 2600, "slabs"), ((1, 8), 2011, "segments")])
def test_a_prefill_in_two_calls(cuda_lib, BH, N, kind):
    # both halves cut, the second one from the first one's state
    q, k, v, g, beta, S0 = make(53, *BH, 2 * N, 64, 64, BF)
    assert way(cuda_lib, *BH, N, 64, 64) == kind
    want, S_want = od.delta(q, k, v, g, beta, S0)
    half = lambda x, i: x[:, :, i * N:(i + 1) * N].contiguous()
    out, S = [], S0
    for i in range(2):
        o, S = cuda_lib.delta_fwd(*(half(x, i) for x in (q, k, v, g, beta)), S)
        out.append(o)
    assert rel(torch.cat(out, 2), want) <= tol_out(BF, 2 * N, 64)
    assert rel(S, S_want) <= tol_state(BF, 2 * N, 64)


# ------------------------------------------------------------ workspaces of the size asked for
def guarded(n, start):
    """n bytes in the middle of a buffer of 0xa5, from `start` on, and a look at what is round them."""
    buf = torch.full((start + n + 4096,), 0xa5, dtype=torch.uint8, device=DEV)
    return buf[start:start + n], lambda: bool((buf[:start] == 0xa5).all() and (buf[start + n:] == 0xa5).all())


@pytest.mark.parametrize("start", [1024, 1040])
@pytest.mark.parametrize("BH,N,dk,dv", [((1, 3), 77, 128, 64), ((2, 32), 2561, 64, 128),
                                        ((2, 4), 1025, 128, 128), ((2, 16), 3580, 64, 64)])
def test_the_forward_stays_in_its_workspace(cuda_lib, BH, N, dk, dv, start):
    q, k, v, g, beta, S0 = make(54, *BH, N, dk, dv, BF)
    want = cuda_lib.delta_fwd(q, k, v, g, beta, S0)
    ws, whole = guarded(cuda_lib.linattn_delta_fwd_workspace(*BH, N, dk, dv, BF), start)
    out, S = torch.empty_like(v), torch.empty_like(S0)
    cuda_lib.linattn_delta_fwd(q, k, v, g, beta, S0, out, S, ws)
    assert torch.equal(out, want[0]) and torch.equal(S, want[1]) and whole()


@pytest.mark.parametrize("start", [1024, 1040])
@pytest.mark.parametrize("BH,N,dk,dv,dtype", [((1, 3), 77, 128, 64, BF), ((5, 31), 130, 64, 128, BF),
                                              ((1, 2), 65, 32, 16, F32), ((2, 3), 1025, 16, 128, F32),
                                              ((5, 31), 45, 128, 128, F32)])
def test_the_backward_stays_in_its_workspace(cuda_lib, BH, N, dk, dv, dtype, start):
    q, k, v, g, beta, S0 = make(55, *BH, N, dk, dv, dtype)
    do = torch.randn(v.shape, device=DEV).to(dtype)
    want = cuda_lib.delta_bwd(q, k, v, g, beta, do, S0, S0, want_dS_init=True)
    ws, whole = guarded(cuda_lib.linattn_delta_bwd_workspace(*BH, N, dk, dv, dtype), start)
    got = cuda_lib.delta_bwd(q, k, v, g, beta, do, S0, S0, want_dS_init=True, workspace=ws)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert whole()


# ------------------------------------------------------------ the tensor-core backward
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("BH,N,gate,state", [((5, 31), 130, "soft", True), ((2, 40), 385, "reset", False),
                                             ((1, 2), 2049, "soft", True), ((1, 2), 2049, "hard", False)])
def test_backward_with_many_heads_and_long_sequences(cuda_lib, BH, N, dk, dv, gate, state):
    # 310 and 160 sweeps on 148 multiprocessors, and 33 chunks through the two stages
    check_bwd(cuda_lib, 56 + dk + dv, *BH, N, dk, dv, BF, gate, state)


def test_backward_of_a_training_step(cuda_lib):
    # 64 heads of 2048 tokens: some of them against the oracle, and against calls of their own
    q, k, v, g, beta, S0 = make(57, 4, 16, 2048, 128, 128, BF)
    do = torch.randn(v.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(58)).to(BF)
    got = cuda_lib.delta_bwd(q, k, v, g, beta, do)[:5]
    for b, h in ((0, 0), (1, 9), (3, 15)):
        at = lambda x: x[b:b + 1, h:h + 1].contiguous()
        one = [at(x) for x in (q, k, v, g, beta, do)]
        for x, y in zip(got, cuda_lib.delta_bwd(*one)):
            assert torch.equal(at(x), y)
        want = od.delta_grad(*one)
        for n, x in zip(("dq", "dk", "dv", "dg", "dbeta"), got):
            t = {"dg": 8 * tol_state(BF, 2048, 128), "dbeta": 2 * tol_state(BF, 2048, 128)}.get(
                n, 2 * tol_out(BF, 2048, 128))
            assert rel(at(x), want[n]) <= t, n
    assert cuda_lib.linattn_device_status() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("BH,N,d,dtype", [((1, 3), 100, 128, BF), ((1, 3), 200, 64, BF),
                                          ((1, 3), 100, 128, F32), ((1, 3), 1500, 16, F32)])
def test_nan_and_infinity_stay_in_their_head_in_the_backward(cuda_lib, value, BH, N, d, dtype):
    gen = torch.Generator(DEV).manual_seed(59)
    ins = list(make(60, *BH, N, d, d, dtype))
    ins.insert(5, torch.randn(ins[2].shape, device=DEV, generator=gen).to(dtype))
    ins.append(torch.randn(ins[6].shape, device=DEV, generator=gen))
    want = cuda_lib.delta_bwd(*ins, want_dS_init=True)
    for which in range(8):      # q, k, v, g, beta, dout, S_init, dS_final
        if which == 3 and value > 0:
            continue            # a gate is at most 0
        a = list(ins)
        a[which] = a[which].clone()
        a[which][0, 1, min(70, a[which].shape[2] - 1)] = value
        got = cuda_lib.delta_bwd(*a, want_dS_init=True)
        for x, y in zip(got, want):
            assert torch.equal(x[:, ::2], y[:, ::2]), which
        assert not all(bool(torch.isfinite(x[:, 1]).all()) for x in got), which
    assert cuda_lib.linattn_device_status() == 0


@pytest.mark.parametrize("BH,N,kind", [((1, 3), 1500, "segments"), ((1, 64), 2600, "slabs")])
def test_nan_stays_in_its_head_where_the_forward_is_cut(cuda_lib, BH, N, kind):
    assert way(cuda_lib, *BH, N, 64, 64) == kind
    ins = make(61, *BH, N, 64, 64, BF)
    want = cuda_lib.delta_fwd(*ins)
    for which in range(1, 5):
        a = list(ins)
        a[which] = a[which].clone()
        a[which][0, 1, 700] = float("nan")
        out, S = cuda_lib.delta_fwd(*a)
        assert torch.equal(out[:, ::2], want[0][:, ::2]) and torch.equal(S[:, ::2], want[1][:, ::2])
        # tokens of earlier chunks, and of segments before it, are as they were
        assert torch.equal(out[0, 1, :640], want[0][0, 1, :640])
        assert out[0, 1, 700].isnan().all() and out[0, 1, -1].isnan().any() and S[0, 1].isnan().any()


def test_backward_captured_beside_another_stream(cuda_lib):
    # more sweeps than multiprocessors, captured, with an eager call of other inputs beside it
    a, b = (make(s, 5, 16, 200, 128, 128, BF)[:5] for s in (62, 63))
    do = [torch.randn(x[2].shape, device=DEV).to(BF) for x in (a, b)]
    want = [cuda_lib.delta_bwd(*x, y)[:5] for x, y in zip((a, b), do)]
    n = cuda_lib.linattn_delta_bwd_workspace(5, 16, 200, 128, 128, BF)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    got = [[torch.empty_like(x) for x in w] for w in want]
    call = lambda i, x, stream=None: cuda_lib.linattn_delta_bwd(
        *x, None, do[i], None, *got[i], None, ws[i], stream)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(0, a)
    for _ in range(2):
        call(1, b, side)
        graph.replay()
    torch.cuda.synchronize()
    for g_, w in zip(got, want):
        for x, y in zip(g_, w):
            assert torch.equal(x, y)

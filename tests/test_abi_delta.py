"""Host-side refusals of the delta-rule and row-norm calls (no GPU needed):
every call below fails validation, so nothing is launched."""
import ctypes

import pytest
import torch

from weight_state_recurrence_b200 import linattn

OK, INV, UNS = linattn.LINATTN_OK, linattn.LINATTN_ERR_INVALID, linattn.LINATTN_ERR_UNSUPPORTED
P = ctypes.c_void_p
A = [P(0x7F0000000000 + i * 0x1000000) for i in range(20)]   # never dereferenced
MIS = P(0x7F00F0000008)


@pytest.fixture(scope="module")
def lib():
    return linattn.load()


def D(B=1, H=1, N=8, dk=64, dv=64, dtype=0, phi=linattn.LINATTN_PHI_IDENTITY):
    return linattn.linattn_dims(B, H, N, dk, dv, dtype, phi)


def fwd(lib, d=None, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S=A[5], out=A[6], Sf=A[7],
             ws=A[8], n=1 << 22)
    a.update(kw)
    return lib.linattn_delta_fwd(ctypes.byref(d or D()), *a.values(), None)


def bwd(lib, d=None, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S=A[5], do=A[6], dSf=A[7], dq=A[8],
             dk=A[9], dv=A[10], dg=A[11], db=A[12], dS=A[13], ws=A[14], n=1 << 22)
    a.update(kw)
    return lib.linattn_delta_bwd(ctypes.byref(d or D()), *a.values(), None)


def step(lib, d=None, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], g=A[3], beta=A[4], S=A[5], out=A[6])
    a.update(kw)
    return lib.linattn_delta_step(ctypes.byref(d or D()), *a.values(), None)


BAD_DIMS = [(D(B=-1), INV), (D(N=-1), INV), (D(dk=48), UNS), (D(dv=256), UNS), (D(dtype=2), UNS),
            (D(phi=linattn.LINATTN_PHI_ELU1), UNS), (D(phi=2), UNS),
            (D(B=1 << 10, H=1 << 10, N=1 << 10), UNS)]


@pytest.mark.parametrize("n", range(len(BAD_DIMS)))
def test_dims_are_checked(lib, n):
    d, want = BAD_DIMS[n]
    assert fwd(lib, d) == want
    assert bwd(lib, d) == want
    if d.N >= 0 and d.N < 1 << 10:
        assert step(lib, d) == want
    assert lib.linattn_delta_fwd_workspace(ctypes.byref(d)) == 0
    assert lib.linattn_delta_bwd_workspace(ctypes.byref(d)) == 0


def test_null_dims(lib):
    assert lib.linattn_delta_fwd(None, *A[:9], 0, None) == INV
    assert lib.linattn_delta_bwd(None, *A[:15], 0, None) == INV
    assert lib.linattn_delta_step(None, *A[:7], None) == INV
    assert lib.linattn_delta_bwd_workspace(None) == 0


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "out"])
def test_forward_and_step_need_their_buffers(lib, name):
    assert fwd(lib, **{name: None}) == INV
    assert step(lib, **{name: None}) == INV


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "S", "out", "Sf"])
def test_forward_alignment(lib, name):
    assert fwd(lib, **{name: MIS}) == INV


def test_forward_overlaps(lib):
    assert fwd(lib, out=A[2]) == INV           # over v
    assert fwd(lib, Sf=A[5]) == INV            # the state in place
    assert fwd(lib, out=A[7]) == INV           # two outputs
    assert fwd(lib, Sf=P(A[4].value + 16)) == INV
    assert fwd(lib, ws=A[6]) == INV


def test_forward_workspace(lib):
    need = lib.linattn_delta_fwd_workspace(ctypes.byref(D()))
    assert need > 0
    assert fwd(lib, n=need - 1) == INV
    assert fwd(lib, ws=None, n=0) == INV
    assert fwd(lib, ws=MIS) == INV
    # the CUDA-core path needs none, and neither does an empty sequence
    for d in (D(dk=32), D(dtype=1), D(N=0)):
        assert lib.linattn_delta_fwd_workspace(ctypes.byref(d)) == 0
    with linattn.kernel_choice(linattn.LINATTN_OP_DELTA, linattn.LINATTN_KERNEL_CUDA_CORES):
        assert lib.linattn_delta_fwd_workspace(ctypes.byref(D())) == 0
    assert lib.linattn_delta_fwd_workspace(ctypes.byref(D())) == need


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "do", "dq", "dk", "dv", "db", "ws"])
def test_backward_needs_its_buffers(lib, name):
    assert bwd(lib, **{name: None}) == INV


@pytest.mark.parametrize("name", ["q", "g", "S", "do", "dSf", "dq", "dk", "dv", "dg", "db", "dS", "ws"])
def test_backward_alignment(lib, name):
    assert bwd(lib, **{name: MIS}) == INV


def test_backward_overlaps_and_workspace(lib):
    assert bwd(lib, dq=A[0]) == INV
    assert bwd(lib, dS=A[7]) == INV
    assert bwd(lib, ws=A[8]) == INV
    assert bwd(lib, dg=A[12]) == INV
    need = lib.linattn_delta_bwd_workspace(ctypes.byref(D()))
    assert need > 0
    assert bwd(lib, n=need - 1) == INV
    assert lib.linattn_delta_bwd_workspace(ctypes.byref(D(N=0))) == 0


def test_step_refusals(lib):
    assert step(lib, S=None) == INV
    assert step(lib, S=MIS) == INV
    assert step(lib, out=A[5]) == INV
    assert step(lib, S=A[1]) == INV


def test_empty_batch_is_a_no_op(lib):
    d = D(B=0)
    assert lib.linattn_delta_fwd(ctypes.byref(d), *[None] * 9, 0, None) == OK
    assert lib.linattn_delta_bwd(ctypes.byref(d), *[None] * 15, 0, None) == OK
    assert lib.linattn_delta_step(ctypes.byref(d), *[None] * 7, None) == OK


# ------------------------------------------------------------ row norms
def nf(lib, rows=4, d=64, kind=0, dtype=0, eps=1e-5, **kw):
    a = dict(x=A[0], w=A[1], b=A[2])
    out = kw.pop("out", A[3])
    a.update(kw)
    return lib.linattn_norm_fwd(rows, d, kind, dtype, *a.values(), eps, out, None)


def nb(lib, rows=4, d=64, kind=0, dtype=0, eps=1e-5, n=1 << 22, **kw):
    a = dict(x=A[0], w=A[1], dy=A[2], dx=A[3], dw=A[4], db=A[5], ws=A[6])
    a.update(kw)
    return lib.linattn_norm_bwd(rows, d, kind, dtype, a["x"], a["w"], eps, a["dy"], a["dx"],
                                a["dw"], a["db"], a["ws"], n, None)


@pytest.mark.parametrize("call", [nf, nb])
def test_norm_arguments(lib, call):
    assert call(lib, rows=-1) == INV
    assert call(lib, d=0) == INV
    assert call(lib, d=8193) == UNS
    assert call(lib, rows=1 << 34, d=64) == UNS
    assert call(lib, kind=2) == UNS
    assert call(lib, dtype=3) == UNS
    for eps in (-1e-5, float("nan"), float("inf")):
        assert call(lib, eps=eps) == INV
    assert call(lib, x=None) == INV
    assert call(lib, x=MIS) == INV
    assert call(lib, w=MIS) == INV


def test_norm_buffers(lib):
    assert nf(lib, out=None) == INV
    assert nf(lib, out=A[0]) == INV
    assert nf(lib, b=MIS) == INV
    assert nf(lib, rows=0, x=None, out=None) == OK
    assert nb(lib, dy=None) == INV
    assert nb(lib, dx=None) == INV
    assert nb(lib, dx=A[2]) == INV
    assert nb(lib, dw=A[5]) == INV
    assert nb(lib, ws=A[4]) == INV
    assert nb(lib, dw=MIS) == INV
    assert nb(lib, rows=0, x=None, dy=None, dx=None, dw=None, db=None, ws=None, n=0) == OK


# ------------------------------------------------------------ the binding
def T(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def test_binding_checks_shapes_and_types():
    q, v = T(1, 2, 4, 64), T(1, 2, 4, 32)
    g = b = T(1, 2, 4, dtype=torch.float32)
    S = T(1, 2, 64, 32, dtype=torch.float32)
    f = linattn.linattn_delta_fwd
    bad = [dict(k=T(1, 2, 5, 64)), dict(v=T(1, 2, 5, 32)), dict(g=T(1, 2, 4)), dict(beta=None),
           dict(beta=T(1, 2, 5, dtype=torch.float32)), dict(S_init=T(1, 2, 32, 64, dtype=torch.float32)),
           dict(out=T(1, 2, 4, 64)), dict(out=v.float()), dict(q=T(2, 4, 64)), dict(k=q.float()),
           dict(S_final=S.double())]
    base = dict(q=q, k=q, v=v, g=g, beta=b, S_init=S, out=v, S_final=S)
    for change in bad:
        with pytest.raises(ValueError):
            f(**{**base, **change})
    with pytest.raises(ValueError):       # no CPU path
        f(**base)
    with pytest.raises(TypeError):
        f(**{**base, "q": q.half(), "k": q.half(), "v": v.half(), "out": v.half()})
    with pytest.raises(ValueError):
        linattn.linattn_delta_step(q, q, v, g, b, S, v)
    x = T(3, 64)
    with pytest.raises(ValueError):
        linattn.linattn_norm_fwd(x, T(64), None, 1e-5, 0, x)
    with pytest.raises(ValueError):
        linattn.linattn_norm_bwd(x, None, 1e-5, 0, T(4, 64), x)

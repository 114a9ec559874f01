"""GPU parity of the row norms against the fp64 oracle.

Tolerances, derived.  fp32 sums of d values by threads of 8 and a tree: at
most (8 + log2 d) roundings of 2^-24 each, the mean, the variance and a few
products after them: (24 + 2 log2 d) 2^-24 relative to the row.  A result
rounded to bf16 adds 2^-8 of each value.  The sums over rows add, per column,
rows / blocks terms in a row: errors of independent terms add in quadrature,
sqrt(rows) 2^-24 on top.  Inputs have |mean| <= 4 standard deviations; x - m
then loses at most 3 bits, 8 x.
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
    assert got.shape == want.shape and torch.isfinite(got).all()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def tol(d):
    return 8 * (24 + 2 * math.log2(d + 1)) * 2.0 ** -24


def make(seed, rows, d, dtype):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)
    x = (r(rows, d) * (0.5 + torch.rand(rows, 1, generator=gen, device=DEV)) + r(rows, 1).clamp(-2, 2)).to(dtype)
    return x, 1 + 0.3 * r(d), 0.3 * r(d), r(rows, d).to(dtype)


def check(lib, rows, d, dtype, kind, weight=True, bias=True, seed=0):
    x, w, b, dy = make(seed + rows + d, rows, d, dtype)
    w, b = (w if weight else None), (b if bias else None)
    rms = kind == lib.LINATTN_NORM_RMS
    rnd = 2.0 ** -8 if dtype == BF else 0.0
    y = lib.norm_fwd(x, w, b, 1e-5, kind)
    assert rel(y, od.norm(x, w, b, 1e-5, rms)) <= tol(d) + rnd
    dx, dw, db = lib.norm_bwd(x, w, dy, 1e-5, kind)
    dx_w, dw_w, db_w = od.norm_grad(x, w, dy, 1e-5, rms)
    assert rel(dx, dx_w) <= 2 * tol(d) + rnd
    more = math.sqrt(rows) * 2.0 ** -24
    assert rel(dw, dw_w) <= tol(d) + more
    assert rel(db, db_w) <= tol(d) + more
    again = lib.norm_bwd(x, w, dy, 1e-5, kind)
    for p, q in zip((dx, dw, db), again):
        assert torch.equal(p, q)
    only, none_w, none_b = lib.norm_bwd(x, w, dy, 1e-5, kind, want_dweight=False, want_dbias=False)
    assert none_w is None and none_b is None and torch.equal(only, dx)


# both sides of every change of threads to a row, odd widths, the largest
WIDTHS = [8, 9, 15, 16, 31, 64, 65, 100, 127, 128, 250, 256, 257, 511, 512, 777, 1024, 1030, 2048,
          2049, 4096, 4104, 5000, 8191, 8192]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_widths(cuda_lib, d, dtype):
    check(cuda_lib, 37, d, dtype, d % 2)


@pytest.mark.parametrize("rows", [1, 2, 3, 16, 33, 1000, 20011])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows(cuda_lib, rows, kind, dtype):
    check(cuda_lib, rows, 128, dtype, kind)
    check(cuda_lib, rows, 96, dtype, kind, weight=False, bias=False)


def test_many_rows(cuda_lib):
    check(cuda_lib, 300007, 64, BF, 0)


@pytest.mark.parametrize("d", [1, 2, 3, 5])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_narrow_rows(cuda_lib, d, dtype):
    # forward and RMS; the layer norm's dx of two values is a difference of
    # nearly equal numbers, so its error is taken against dy's size instead
    x, w, b, dy = make(d, 50, d, dtype)
    rnd = 2.0 ** -8 if dtype == BF else 0.0
    for kind in (0, 1):
        y = cuda_lib.norm_fwd(x, w, b, 1e-2, kind)
        want = od.norm(x, w, b, 1e-2, kind == 1)
        # x - m of a narrow row: m's rounding, relative to x, over the row's deviation
        far = float((y.double() - want).abs().max())
        assert far <= (rnd + 2.0 ** -18) * float(want.abs().max())
        dx, dw, db = cuda_lib.norm_bwd(x, w, dy, 1e-2, kind)
        dx_w, dw_w, db_w = od.norm_grad(x, w, dy, 1e-2, kind == 1)
        # 1 / sqrt(s + eps) <= 10: a rounding of w dy grows by that
        assert float((dx.double() - dx_w).abs().max()) <= rnd * float(dx_w.abs().max()) + 10 * 2.0 ** -18
        assert rel(db, db_w) <= tol(d) + 8 * 2.0 ** -24


def test_rows_of_one_value_and_nan(cuda_lib):
    x = torch.full((3, 64), 2.5, device=DEV)
    b = torch.randn(64, device=DEV)
    assert torch.equal(cuda_lib.norm_fwd(x, None, b), b.expand(3, 64))
    x[1, 5] = float("nan")
    y = cuda_lib.norm_fwd(x, None, b)
    assert y[1].isnan().all() and torch.equal(y[0], b) and torch.equal(y[2], b)
    # eps = 0: 0 / 0 in the rows of one value, and only there; rows past the
    # last add nothing to the sums
    x = torch.randn(5, 64, device=DEV)
    dy = torch.randn(5, 64, device=DEV)
    dx, dw, db = cuda_lib.norm_bwd(x, None, dy, 0.0)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert rel(dw, od.norm_grad(x, None, dy, 0.0)[1]) <= tol(64)


def test_no_rows(cuda_lib):
    x = torch.empty(0, 64, device=DEV)
    assert cuda_lib.norm_fwd(x).shape == (0, 64)
    dx, dw, db = cuda_lib.norm_bwd(x, None, x)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_leading_axes_and_offsets_in_a_buffer(cuda_lib):
    buf = torch.full((8 * 100 + 64,), 3.0, device=DEV)
    x = torch.randn(2, 4, 100, device=DEV)
    out = buf[32:32 + 800].view(2, 4, 100)
    cuda_lib.linattn_norm_fwd(x, None, None, 1e-5, 0, out)
    assert torch.equal(out.view(8, 100), cuda_lib.norm_fwd(x.view(8, 100)))
    assert (buf[:32] == 3).all() and (buf[832:] == 3).all()


def test_past_32_bit_offsets(cuda_lib):
    rows, d = (1 << 21) + 3, 1024            # 2^31 elements and more, 4 GB in bf16
    x = torch.empty(rows, d, dtype=BF, device=DEV)
    x[:5] = torch.randn(5, d, device=DEV).to(BF)
    x[5:-5] = 1.0
    x[-5:] = torch.randn(5, d, device=DEV).to(BF)
    y = cuda_lib.norm_fwd(x)
    for part in (slice(0, 5), slice(rows - 5, rows)):
        assert rel(y[part], od.norm(x[part])) <= tol(d) + 2.0 ** -8
    assert not y[5:9].any() and not y[-9:-5].any()


def test_capture_and_streams(cuda_lib):
    x, w, b, dy = make(3, 500, 256, BF)
    y = cuda_lib.norm_fwd(x, w, b)
    want = cuda_lib.norm_bwd(x, w, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cuda_lib.norm_bwd(x, w, dy, stream=side)
    side.synchronize()
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    out, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(cuda_lib.linattn_norm_bwd_workspace(500, 256), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.linattn_norm_fwd(x, w, b, 1e-5, 0, out)
        cuda_lib.linattn_norm_bwd(x, w, 1e-5, 0, dy, dx, dw, db, ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y)
    for p, q in zip((dx, dw, db), want):
        assert torch.equal(p, q)


def test_a_workspace_too_small_is_refused(cuda_lib):
    x, w, b, dy = make(4, 5000, 64, BF)
    n = cuda_lib.linattn_norm_bwd_workspace(5000, 64)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(n - 16, dtype=torch.uint8, device=DEV)
    for short in (ws, None):
        with pytest.raises(cuda_lib.LinattnError):
            cuda_lib.linattn_norm_bwd(x, w, 1e-5, 0, dy, dx, dw, None, short)
    cuda_lib.linattn_norm_bwd(x, w, 1e-5, 0, dy, dx, None, None, None)

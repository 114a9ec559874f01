"""GPU parity of the row norms where rows are narrow, constant or end in an exactly sized workspace.

Tolerances, derived.  The mean of d values is off by at most (d + 1) 2^-24 of the largest |x| of the row
(d - 1 additions, the product by 1 / d and its own rounding), and x - m by that and one rounding.  With
rstd <= eps^-1/2 the normalised value xh is off by (d + 2) 2^-24 max|x| eps^-1/2, and by (d + 4) 2^-24 of
itself for the variance, the root and two products.  A column of dw adds dy xh over the rows: those errors
times |dy|, and `rows` roundings of the running sum, at most 2^-24 of the sum of |dy xh| each.
"""
import pytest
import torch

from oracle import delta as od
from test_parity_norm import BF, DEV, F32, make

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("d", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kind", [0, 1])
def test_weight_gradient_of_narrow_rows(cuda_lib, d, dtype, kind):
    rows, eps = 50, 1e-2
    x, w, _, dy = make(100 + d, rows, d, dtype)
    _, dw, db = cuda_lib.norm_bwd(x, w, dy, eps, kind)
    _, dw_w, db_w = od.norm_grad(x, w, dy, eps, kind == 1)
    X, G = x.double(), dy.double().abs()
    xh = od.norm(x, None, None, eps, kind == 1).abs()
    far = (d + 2) * U * X.abs().amax(1, keepdim=True) * eps ** -0.5 + (d + 4) * U * xh
    bound = (G * far).sum(0) + rows * U * (G * (xh + far)).sum(0)
    assert ((dw.double() - dw_w).abs() <= bound).all()
    assert ((db.double() - db_w).abs() <= rows * U * G.sum(0)).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_row_of_one_value_without_eps(cuda_lib, dtype):
    # 64 times 2.5: the mean is exact, so this is 0 / 0, in this row and in what it is summed into only
    x, w, b, dy = make(120, 9, 64, dtype)
    x[4] = 2.5
    rest = [i for i in range(9) if i != 4]
    y = cuda_lib.norm_fwd(x, w, b, 0.0)
    dx, dw, db = cuda_lib.norm_bwd(x, w, dy, 0.0)
    assert y[4].isnan().all() and dx[4].isnan().all() and dw.isnan().all()
    assert torch.equal(y[rest], cuda_lib.norm_fwd(x[rest], w, b, 0.0))
    dx_rest, _, _ = cuda_lib.norm_bwd(x[rest], w, dy[rest], 0.0)
    assert torch.equal(dx[rest], dx_rest)
    # dy's own sum has no part of it: 9 roundings of the running sum at most
    want = dy.double().sum(0)
    assert ((db.double() - want).abs() <= 9 * U * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("d", [3, 64, 100, 2049])
@pytest.mark.parametrize("value", [1.1, -700.3])
def test_a_row_of_one_value_is_its_bias_up_to_the_mean(cuda_lib, d, value):
    # |x - m| <= (d + 2) 2^-24 |x|, over the root of eps
    x = torch.full((3, d), value, device=DEV)
    b = torch.randn(d, device=DEV)
    for eps in (1e-5, 1e-2):
        y = cuda_lib.norm_fwd(x, None, b, eps)
        far = (d + 2) * U * abs(value) * eps ** -0.5
        assert ((y - b).abs() <= far + 2 * U * (b.abs() + far)).all()


@pytest.mark.parametrize("rows,d,dtype", [(1, 8, BF), (5000, 64, BF), (777, 2049, F32), (300, 8192, BF)])
def test_the_sums_stay_in_their_workspace(cuda_lib, rows, d, dtype):
    x, w, _, dy = make(130, rows, d, dtype)
    want = cuda_lib.norm_bwd(x, w, dy)
    n = cuda_lib.linattn_norm_bwd_workspace(rows, d)
    buf = torch.full((n + 2048,), 0xa5, dtype=torch.uint8, device=DEV)
    got = cuda_lib.norm_bwd(x, w, dy, workspace=buf[1024:1024 + n])
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    assert (buf[:1024] == 0xa5).all() and (buf[1024 + n:] == 0xa5).all()

"""Layer norm of rows far from zero beside their spread, at widths that leave lanes
without a column."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests.test_dense_gpu import BF16, F32, check_norm, rand, run_norm  # noqa: E402


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 5, 7, 64, 100, 128, 200])
@pytest.mark.parametrize("power,eps", [(120, 1e-5), (-120, 1e-5), (100, 1e-16), (40, 1e-30), (3, 1e-5)])
def test_constant_rows(dt, dim, power, eps):
    """Rows of one value, whose size times 1/sqrt(eps) is past fp32: xhat is 0 and every gradient finite."""
    x = rand(9, dim, seed=1)
    x[::2] = 2.0 ** power if power > 0 else -(2.0 ** -power)
    y, dx, dw, db = check_norm(x.to(dt), rand(dim, seed=2).to(dt), rand(dim, seed=3).to(dt),
                               rand(9, dim, seed=4).to(dt), eps=eps)
    for t in (y, dx, dw, db):
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("dim", [5, 64, 100, 200, 1000, 3000])
@pytest.mark.parametrize("size", [1e25, 1e30, 1e34])
def test_spreads_past_fp32_are_infinite(dim, size):
    """The squares of the centred values overflow: rstd is 0, y = bias, nothing is NaN."""
    x, w, b, dy = size * rand(5, dim, seed=1), rand(dim, seed=2), rand(dim, seed=3), rand(5, dim, seed=4)
    y, dx, dw, db = run_norm(x, w, b, dy)
    assert bool((y == b).all())
    assert not dx.any() and not dw.any()
    assert bool(torch.isfinite(db).all())

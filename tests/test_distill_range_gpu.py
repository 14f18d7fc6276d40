"""Distillation where the products of logits and 1/temperature are far from zero:
masks of large finite values (whole rows, whole chunks beside live ones), maxima far
above the rest, low temperatures. Oracle and bounds are those of tests/dense_ref.py,
which count roundings; they hold at any size of the product, since only differences
from the row's maximum matter."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests import dense_ref as ref  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402
from tests.test_dense_gpu import BF16, F32, TYPES, check_distill, rand, run_distill, teacher  # noqa: E402

WIDE = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
SIZES = pytest.mark.parametrize("v", [300, 40000])      # one chunk a row, and several


@WIDE
@SIZES
@pytest.mark.parametrize("fill", [1e5, 1e7, 1e9, 3e9, 1e10, 1e15, 1e20, 1e29, 1e30, 1e35])
def test_masks_of_large_finite_values(dt, v, fill):
    z = rand(6, v, seed=1)
    z[0] = -fill                            # nothing left: every class alike
    z[1, :v // 2] = -fill                   # whole chunks masked beside live ones
    z[2] = -fill                            # all but one class
    z[2, 5] = 1.0
    z[3, 7] = fill                          # one class far above the rest
    z[4] = fill
    z[5, v // 2:] = -fill
    z[5, :v // 2] -= 2 * fill               # what is left of an offset row
    ids = torch.tensor([[0, 1, v - 1, 9], [v - 1, v - 2, v - 3, v - 4], [5, 5, 5, 5], [7, 7, 7, 7],
                        [3, 2, 1, v // 2], [v - 1, v - 2, v - 3, v // 2]], device=DEV)
    check_distill(z.to(dt), ids, rand(6, 4, seed=2), torch.ones(6, device=DEV), 1.0)


@SIZES
def test_listed_classes_behind_a_large_mask(v):
    """The teacher's classes are the masked ones: the loss is as large as the mask."""
    z = rand(3, v, seed=1)
    for r, fill in enumerate((1e6, 1e10, 1e20)):
        z[r, :v // 2] = -fill
    ids = torch.tensor([[0, 1, 2, v - 1]] * 3, device=DEV)
    check_distill(z, ids, rand(3, 4, seed=2), torch.ones(3, device=DEV), 1.0)


@SIZES
def test_rows_around_the_switch_of_the_exponents_form(v):
    """Maxima of the chunks on both sides of 2^24 / log2(e), some classes apart from each other."""
    step = torch.randint(-6, 7, (4, v), generator=torch.Generator().manual_seed(5)).to(DEV)
    z = 11629079.0 + step
    z[1::2] *= -1
    z[2:, :v // 2] -= torch.sign(z[2:, :v // 2]) * 20   # the first half's maximum is nearer to zero
    ids = torch.tensor([[0, 1, v // 2, v - 1]] * 4, device=DEV)
    check_distill(z, ids, rand(4, 4, seed=2), torch.ones(4, device=DEV), 1.0)


@TYPES
@SIZES
@pytest.mark.parametrize("power", [-13, -20, -30, -40])
def test_low_temperatures(dt, v, power):
    ids, tl, w = teacher(9, v, 5, seed=v)
    z = (2 * rand(9, v, seed=1)).to(dt)
    z[1, :] = z[1, :1]                      # all classes alike
    check_distill(z, ids, tl, w + 0.5, 2.0 ** power)


@TYPES
@pytest.mark.parametrize("v,top", [(300, 5), (16384, 64), (16385, 64), (40000, 9), (131072, 300)])
def test_one_call_gives_the_bits_of_two(dt, v, top):
    """Forward and backward apart, in one call, and the forward without statistics: the same bits."""
    ids, tl, w = teacher(7, v, top, seed=v)
    z = (2 * rand(7, v, seed=1)).to(dt)
    z[3, :v // 2] = -1e4
    say("distill bits", dt, v, top)
    (loss, dz), (loss2, dz2), only = run_distill(z, ids, tl, w, 2.0)
    assert torch.equal(loss, loss2) and torch.equal(loss, only)
    assert torch.equal(dz, dz2)

"""The gated block at the ends of its types' ranges, as its documentation states them."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests import dense_ref as ref  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402
from tests.test_dense_gpu import F16, F32, check_gate, gate_inputs, run_gate  # noqa: E402


@pytest.mark.parametrize("rows", [3, 70])
def test_f16_backward_factors_past_their_range(rows):
    """dout * up * act' up to 65504 is exact to the bounds; past it the row and the weights' gradients are
    infinite or NaN, never a finite wrong value, and the other rows keep their bits."""
    k, h = 64, 40
    x = torch.zeros(rows, k, dtype=F16, device=DEV)
    x[:, 0], x[:, 1] = 2.0 ** -8, 2.0 ** -4
    wg, wu = (torch.zeros(h, k, dtype=F16, device=DEV) for _ in range(2))
    wg[:, 0], wu[:, 1] = 2.0 ** -8, 2.0 ** 12               # gate 2^-16, up 256; every result stays in range
    dout = torch.full((rows, h), 1.0, dtype=F16, device=DEV)
    dout[1] = 255.0                                         # dg 65280
    good = check_gate(x, wg, wu, dout, "relu")
    assert bool(torch.isfinite(good[3]).all())
    dout[1] = 256.0                                         # dg 65536: past the type
    say("gate f16 range", rows)
    out, g, u, dx, dwg, dwu = run_gate(x, wg, wu, dout, "relu")
    assert not bool(torch.isfinite(dx[1, 0])) and not bool(torch.isfinite(dwg[:, 0]).any())
    keep = [r for r in range(rows) if r != 1]
    assert torch.equal(dx[keep], good[3][keep])
    assert torch.equal(out, good[0]) and bool(torch.isfinite(dwu).all())     # du stays in range


@pytest.mark.parametrize("rows", [5, 40])
def test_fp32_infinities_give_nan_and_stay_apart(rows):
    """An infinity in a row of x makes that row NaN, one in a row of a weight that column, and no other."""
    x, wg, wu, _ = gate_inputs(rows, 100, 90, F32, train=False)
    good = run_gate(x, wg, wu, None, "silu")[0]
    x2, wg2 = x.clone(), wg.clone()
    x2[3, 5] = math.inf
    wg2[7, 99] = -math.inf
    out = run_gate(x2, wg2, wu, None, "silu")[0]
    bad = torch.zeros_like(good, dtype=torch.bool)
    bad[3], bad[:, 7] = True, True
    assert bool(torch.isnan(out[bad]).all()) and torch.equal(out[~bad], good[~bad])


def test_fp32_range_of_full_accuracy():
    """Operands from 2^-100 up keep fp32's digits whatever the other factor is."""
    x, wg, wu, _ = gate_inputs(70, 128, 64, F32, train=False)
    for power in (-100, -60, 60, 100):
        a, b = x * 2.0 ** power, 2.0 ** -power
        got = run_gate(a, wg * b, wu, None, "relu")[0]
        # relu of products of the first's size, times the others': up is 2^power as large
        want = ref.gate(a, wg * b, wu, "relu")[0]
        assert ref.rel(got.double() * 2.0 ** -power, want * 2.0 ** -power) < 2.0 ** -20, power

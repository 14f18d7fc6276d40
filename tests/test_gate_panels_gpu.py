"""The gated block's forward where its inputs are copied into panels: products long enough
beside their inputs that this pays for aligned ones, and unaligned ones through the largest tiles."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from tests.test_dense_gpu import BF16, F16, check_gate, gate_inputs, run_gate  # noqa: E402


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("m,k,h,pad", [(8200, 136, 9000, 0),     # aligned, copied for their length
                                       (8100, 72, 9000, 8),      # the same out of wider rows
                                       (6000, 136, 9000, 0),     # aligned, shorter: as they are
                                       (5000, 131, 4100, 3)])    # unaligned
def test_forward_through_panels(dt, m, k, h, pad):
    ins = gate_inputs(m, k, h, dt, train=False)
    out = check_gate(*ins, "silu", pad)[0]
    assert torch.equal(out, run_gate(*ins, "silu", pad)[0])


def test_panels_and_plain_rows_give_the_same_bits():
    """The rows of a batch that is copied and of one that is not: the same tiles, the same sums."""
    x, wg, wu, _ = gate_inputs(8200, 200, 9000, BF16, train=False)
    long = run_gate(x, wg, wu, None, "gelu")[0]
    short = run_gate(x[:6000].clone(), wg, wu, None, "gelu")[0]
    assert torch.equal(long[:6000], short)

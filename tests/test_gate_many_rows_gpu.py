"""The gated block's copies of unaligned rows where they are more than one launch takes."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import tensor_train_compressed_amd as tte  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402
from tests.test_dense_gpu import BF16, gate_inputs  # noqa: E402


@pytest.mark.parametrize("rows,dim", [((1 << 22) - 1, 135), ((1 << 22) - 1, 8201)])
def test_rows_of_every_launch_are_copied(rows, dim):
    """An x of odd width, zero but for rows spread over it: their bits are those of a batch of these rows alone."""
    need = 2 * rows * (dim + 64) * 2 + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs more free device memory")
    say("gate many rows", rows, dim)
    hidden, at = 8, torch.tensor([0, 1, 17, 500_000, rows // 2, rows // 2 + 1, rows - 1_000_000, rows - 17, rows - 1])
    few, wg, wu, _ = gate_inputs(40, dim, hidden, BF16, train=False)    # more than the rows taken without tiles
    want = torch.empty(40, hidden, dtype=BF16, device=DEV)
    tte.tt_emb_gate_forward(few, wg, wu, want)
    x = torch.zeros(rows, dim, dtype=BF16, device=DEV)
    at = at.to(DEV)
    x[at] = few[:len(at)]
    out = torch.full((rows, hidden), float("nan"), dtype=BF16, device=DEV)
    tte.tt_emb_gate_forward(x, wg, wu, out)
    assert torch.equal(out[at], want[:len(at)])
    out[at] = 0
    assert not out.any()          # silu(0) * 0
    del x, out
    torch.cuda.empty_cache()

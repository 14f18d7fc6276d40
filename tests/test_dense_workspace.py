"""Workspaces of the dense operators: one sized for the largest batch serves every
smaller one (a program sizes its buffers once)."""
import random

import pytest

import tensor_train_compressed_amd as tte

torch = pytest.importorskip("torch")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def row_counts(rng):
    """From one row to many: every small count, the counts around tiles, and others."""
    around = [t * k + d for t in (16, 32, 128, 256) for k in (1, 2, 3, 5, 8, 16, 31, 64) for d in (-1, 0, 1)]
    return sorted({*range(0, 70), *around, *(rng.randrange(1, 40000) for _ in range(400))})


def rising(sizes):
    assert all(s > 0 for _, s in sizes)
    for (m, a), (n, b) in zip(sizes, sizes[1:]):
        assert a <= b, f"{n} rows need {b} bytes, {m} rows {a}"


def test_gate_workspace_serves_fewer_rows():
    rng = random.Random(3)
    widths = [(4096, 1024), (1024, 1024), (4096, 10240), (128, 512), (1, 1), (64, 20000), (20000, 64), (2056, 4200)]
    for dim, hidden in widths + [(rng.randrange(1, 9000), rng.randrange(1, 9000)) for _ in range(20)]:
        for dt in (F32, BF16):
            rising([(m, tte.tt_emb_gate_workspace_bytes(dt, m, dim, hidden)) for m in row_counts(rng)])


@pytest.mark.gpu
@pytest.mark.parametrize("dt,most,fewer,dim,hidden", [
    (BF16, 2049, (2048, 1500, 40, 3), 4096, 1024), (F16, 1100, (1024, 500, 20), 1024, 1024),
    (F32, 700, (512, 257, 33), 1024, 640)])
def test_gate_in_a_larger_batchs_workspace(dt, most, fewer, dim, hidden):
    """Forward and backward of fewer rows in it: the bits that a workspace of their own gives, and nothing past it."""
    from tests.test_dense_gpu import gate_inputs
    size = tte.tt_emb_gate_workspace_bytes(dt, most, dim, hidden)
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda:0")
    x, wg, wu, d = gate_inputs(most, dim, hidden, dt)
    for m in (most, *fewer):
        print("gate workspace", dt, m, dim, hidden, flush=True)
        outs = []
        for ws in (room[:size], None):
            out, g, u = (torch.empty(m, hidden, dtype=t, device="cuda:0") for t in (dt, F32, F32))
            dx, dwg, dwu = torch.empty_like(x[:m]), torch.empty_like(wg), torch.empty_like(wu)
            tte.tt_emb_gate_forward(x[:m], wg, wu, out, g, u, workspace=ws)
            tte.tt_emb_gate_backward(x[:m], wg, wu, g, u, d[:m], dx, dwg, dwu, workspace=ws)
            outs.append((out, g, u, dx, dwg, dwu))
        for a, b in zip(*outs):
            assert torch.equal(a, b)
        assert bool((room[size:] == 77).all())

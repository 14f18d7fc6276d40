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


def test_gate_forward_asks_for_its_own_workspace():
    """A token through large weights needs none of the training step's room; no forward needs more than training."""
    rng = random.Random(5)
    assert tte.tt_emb_gate_forward_workspace_bytes(BF16, 1, 4096, 10240) <= 4096
    for dim, hidden in [(4096, 1024), (4096, 10240), (512, 1536), (1, 1)]:
        for dt in (F32, F16):
            sizes = [(m, tte.tt_emb_gate_forward_workspace_bytes(dt, m, dim, hidden)) for m in row_counts(rng)]
            rising(sizes)
            assert all(s <= tte.tt_emb_gate_workspace_bytes(dt, m, dim, hidden) for m, s in sizes)
    assert tte.load_library().tt_emb_gate_forward_workspace_bytes(1, 2, 8, 0) == 0


def test_distill_workspace_serves_fewer_rows():
    rng = random.Random(4)
    for classes in [1, 2048, 4096, 4097, 16384, 16385, 50021, 131072, 1000000, 1 << 22] + \
            [rng.randrange(1, 300000) for _ in range(20)]:
        for dt in (F32, F16):
            rising([(m, tte.tt_emb_distill_workspace_bytes(dt, m, classes)) for m in range(1, 2100)])


def test_norm_workspace_serves_fewer_rows():
    for dim in (1, 100, 128, 129, 600, 1000, 2048, 4096, 9001, 16384):
        rising([(m, tte.tt_emb_norm_workspace_bytes(BF16, m, dim)) for m in range(0, 9000)])


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


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("most,fewer,dim,hidden", [(16, (3, 1), 1030, 700), (32, (17,), 520, 700), (33, (32, 1), 4096, 4200),
                                                   (1100, (1037, 300, 16), 1030, 700), (600, (512, 64), 4096, 1024)])
def test_gate_forward_in_its_own_workspace(dt, most, fewer, dim, hidden):
    from tests.test_dense_gpu import gate_inputs
    size = tte.tt_emb_gate_forward_workspace_bytes(dt, most, dim, hidden)
    full = torch.empty(tte.tt_emb_gate_workspace_bytes(dt, most, dim, hidden), dtype=torch.uint8, device="cuda:0")
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda:0")
    x, wg, wu, _ = gate_inputs(most, dim, hidden, dt, train=False)
    for m in (most, *fewer):
        print("gate forward workspace", dt, m, dim, hidden, flush=True)
        outs = []
        for ws in (room[:size], full, None):
            outs.append(torch.empty(m, hidden, dtype=dt, device="cuda:0"))
            tte.tt_emb_gate_forward(x[:m], wg, wu, outs[-1], workspace=ws)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        assert bool((room[size:] == 77).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [F32, F16], ids=["f32", "f16"])
@pytest.mark.parametrize("most,fewer,classes", [(1024, (1014, 700, 341, 9, 1), 16384), (300, (256, 255, 40), 50021)])
def test_distill_in_a_larger_batchs_workspace(dt, most, fewer, classes):
    """The same of every form of distillation."""
    from tests.test_dense_gpu import rand, teacher
    size = tte.tt_emb_distill_workspace_bytes(dt, most, classes)
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda:0")
    ids, tl, w = teacher(most, classes, 5, seed=1)
    z = rand(most, classes, seed=2, dt=dt)
    for m in (most, *fewer):
        print("distill workspace", dt, m, classes, flush=True)
        outs = []
        for ws in (room[:size], None):
            loss, loss2, stats = (torch.empty(*s, device="cuda:0") for s in ((m,), (m,), (m, 2)))
            dz, dz2 = torch.empty_like(z[:m]), torch.empty_like(z[:m])
            rows = z[:m], ids[:m], tl[:m]
            tte.tt_emb_distill_forward(*rows, loss, stats, temperature=2.0, workspace=ws)
            tte.tt_emb_distill_backward(*rows, stats, w[:m], dz, temperature=2.0)
            tte.tt_emb_distill_train(*rows, w[:m], loss2, dz2, temperature=2.0, workspace=ws)
            outs.append((loss, stats, dz, loss2, dz2))
        for a, b in zip(*outs):
            assert torch.equal(a, b)
        assert bool((room[size:] == 77).all())

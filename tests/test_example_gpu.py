"""The example that runs the table, the dense operators and distillation together:
its gradients against 64-bit differentiation of the same head, and its training."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import workloads as wl  # noqa: E402
from examples import distill_head as ex  # noqa: E402
from tests import dense_ref as ref  # noqa: E402
from tests.gpu_helpers import say  # noqa: E402

import tensor_train_compressed_amd as tte  # noqa: E402


def setup(dtype, batch=96, hidden=192, classes=700):
    p = wl.make("train11m", batch=batch)
    table = ex.Table(p)
    idx, off = torch.from_numpy(p.indices).to(ex.DEV), torch.from_numpy(p.offsets).to(ex.DEV)
    head = ex.Head(batch, p.dim, hidden, classes, dtype)
    ids, tl = ex.teacher_lists(batch, classes, 12, seed=3)
    pooled = torch.empty(batch, p.dim, device=ex.DEV)
    return table, head, table.plan(idx, off), pooled, ids, tl, idx, off


def test_head_gradients():
    """fp32: the loss, every gradient and the pooled rows' gradient against autograd in 64 bits."""
    table, head, plan, pooled, ids, tl, _, _ = setup(torch.float32)
    say("example head gradients")
    w = torch.full((pooled.shape[0],), 0.125, device=ex.DEV)
    tte.tt_emb_forward_train(plan, *table.cores, pooled)
    logits = head.forward(pooled, keep=True)
    tte.tt_emb_distill_train(logits, ids, tl, w, head.loss, head.dlogits, temperature=2.0, workspace=head.workspace)
    dpooled = head.backward(pooled.shape[0])
    x = pooled.double().cpu().requires_grad_()
    q = {k: v.double().cpu().requires_grad_() for k, v in head.params.items()}
    y = torch.nn.functional.layer_norm(x, (x.shape[1],), q["norm_weight"], q["norm_bias"], 1e-5)
    z = torch.nn.functional.silu(y @ q["w_gate"].t()) * (y @ q["w_up"].t()) @ q["classes"].t()
    there = ids.cpu() >= 0
    p = torch.softmax(torch.where(there, tl.double().cpu() / 2, -1e9), 1) * there
    lq = torch.gather(torch.log_softmax(z / 2, 1), 1, ids.cpu().clamp_min(0))
    loss = 4 * (torch.special.xlogy(p, p) - p * lq).sum(1)
    (loss * w.cpu().double()).sum().backward()
    # five operators in a row, each good to some tens of fp32 roundings of its sums
    bound = 5 * ref.LEVELS * ref.U32
    assert ref.rel(head.loss, loss.detach()) <= bound
    assert ref.rel(dpooled, x.grad) <= bound
    for k, v in q.items():
        assert ref.rel(head.grads[k], v.grad) <= bound, k


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_training_lowers_the_loss_and_a_bag_is_answered(dtype):
    table, head, plan, pooled, ids, tl, idx, off = setup(ex.DTYPES[dtype])
    say("example training", dtype)
    w = torch.full((pooled.shape[0],), 1.0 / pooled.shape[0], device=ex.DEV)
    means = []
    for _ in range(30):
        means.append(float(ex.train_step(table, head, plan, pooled, ids, tl, w, 2.0, lr=0.5, table_lr=0.05).mean()))
    assert means[-1] < 0.7 * means[0], means
    one = off[:2].contiguous()
    first = ex.answer(table, head, idx[:int(one[1])].contiguous(), one, torch.empty(1, pooled.shape[1], device=ex.DEV), 5)
    assert first.values.shape == (1, 5) and bool(torch.isfinite(first.values).all())

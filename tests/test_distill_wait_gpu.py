"""The wait of distillation's one-call form: a workgroup whose row's other parts have
not come forms them itself, from the logits, and gives the same bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import tensor_train_compressed_amd as tte  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402
from tests.test_dense_gpu import TYPES, rand, teacher  # noqa: E402


def train(z, ids, tl, w, polls):
    """(loss, dlogits) with workgroups that give up after `polls` polls (negative: the default)."""
    lib = tte.load_library()
    loss, dz = torch.full((len(z),), float("nan"), device=DEV), torch.full_like(z, float("nan"))
    was = lib.tt_distill_set_polls(polls)
    try:
        tte.tt_emb_distill_train(z, ids, tl, w, loss, dz, temperature=1.5)
    finally:
        lib.tt_distill_set_polls(was)
    torch.cuda.synchronize()
    return loss, dz


@TYPES
@pytest.mark.parametrize("m,v,top", [(3, 16385, 20), (4, 40000, 9), (5, 50021, 20), (2, 131072, 300), (2, 300001, 100),
                                     (600, 33000, 5)])
def test_parts_formed_by_the_waiting_workgroup(dt, m, v, top):
    """No poll, so that every workgroup forms every part; one poll, so that some are met and some formed."""
    ids, tl, w = teacher(m, v, top, seed=m + v)
    z = (2 * rand(m, v, seed=1)).to(dt)
    z[0, :v // 2] = -1e4
    z[1, 1::2] = -float("inf")
    say("distill wait", dt, m, v, top)
    want = train(z, ids, tl, w + 0.5, -1)
    assert bool(torch.isfinite(want[1]).all())
    for polls in (0, 1, 3):
        got = train(z, ids, tl, w + 0.5, polls)
        assert torch.equal(got[0], want[0]), polls      # (an infinite loss is its own equal)
        assert torch.equal(got[1], want[1]), polls


def test_the_setting_returns():
    lib = tte.load_library()
    was = lib.tt_distill_set_polls(7)
    assert lib.tt_distill_set_polls(-1) == 7
    assert lib.tt_distill_set_polls(-1) == was

"""Attention at the ends of its operands' ranges, forward and backward: large scores, whose
differences alone decide. Bounds count roundings, as those of tests/attend_ref.py do, but
do not grow with the scores: where a score is exact (one product, or a few whose
sum fp32 holds), nothing about its weight may depend on how far from zero it is."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import tensor_train_compressed_amd as tte  # noqa: E402
from tests import attend_ref as ref  # noqa: E402
from tests.dense_ref import check, product_slack, rounded  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402
from tests.test_attend_gpu import offsets_of  # noqa: E402
from tests.test_dense_gpu import BF16, F16, F32, TYPES, rand  # noqa: E402

F64, I64, I32 = torch.float64, torch.int64, torch.int32
U, U32 = ref.U, ref.U32
# |score| from which fp32 cannot hold a score times log2 e to better than a sixteenth
BORDER = 2.0 ** 20 / 1.4426950408889634


def weights_of(s):
    """Softmax of exact scores in 64 bits, and the bound of a weight's error in fp32: its exponent is a difference's
    product with log2 e (two roundings, of at most 128 bits where the weight is not 0), then a power of two."""
    p = torch.softmax(s, -1)
    x = (torch.logsumexp(s, -1, keepdim=True) - s).clamp(0, 128)
    return p, p * 8 * U32 * (1 + x) + 2.0 ** -126


# ------------------------------------------------ references of a running softmax

def border_scores(step):
    """Keys of 16 rows' sequences: 63 alike, then one that is `step` above them (past the first 63's weights by e^step),
    then some far below. Scores are multiples of 1/16 around the border."""
    base = torch.tensor([BORDER - 5.5 + 0.3 * i for i in range(16)], dtype=F64)
    base = (base * 16).round() / 16
    s = base[:, None].repeat(1, 150)
    s[:, 64] += step
    s[:, 63] -= 900.0
    s[:, 65:] -= 1000.0
    return s.to(DEV)


@pytest.mark.parametrize("dim", [32, 128])
def test_a_reference_that_passes_the_border(dim):
    """The running maximum goes from where scores times log2 e are rounded to where differences come first: what was summed
    before keeps its weight. One sequence a row of scores; every query sees the same."""
    s = border_scores(6.0)
    seqs, n = s.shape
    q = torch.zeros(seqs * n, dim, device=DEV)
    k = torch.zeros_like(q)
    q[:, 0] = 1.0
    k[:, 0] = s.flatten().float()
    assert torch.equal(k[:, 0].double(), s.flatten())
    v = rand(seqs * n, dim, seed=1)
    out = torch.empty_like(q)
    tte.tt_emb_attend_forward(q, k, v, offsets_of([n] * seqs), out, heads=1, kv_heads=1, causal=False, scale=1.0)
    p, e = weights_of(s)
    for i in range(seqs):
        r = slice(i * n, (i + 1) * n)
        vi = v[r].double()
        want = p[i:i + 1] @ vi
        bound = (e[i:i + 1] + 2 * product_slack(n) * p[i:i + 1]) @ vi.abs() + want.abs() * e[i].sum() + rounded(F32, want)
        check(out[r], want.expand(n, dim), bound.expand(n, dim), f"border, base {float(s[i, 0])}")


def test_rows_beside_one_past_the_border():
    """A row's weights are its own, whatever the scores of the rows beside it in a wave."""
    n, dim = 150, 32
    for m in (500000.0, 500000.375, 600001.125, 700000.6875, 123456.8125):
        q = torch.zeros(n, dim, device=DEV)
        k, v = torch.zeros_like(q), rand(n, dim, seed=1)
        q[:, 0] = 1.0
        k[:, 0] = m
        k[64, 0], k[63, 0], k[65:, 0] = m + 6, m - 900, m - 1000
        alone, beside = torch.empty_like(q), torch.empty_like(q)
        how = dict(heads=1, kv_heads=1, causal=False, scale=1.0)
        tte.tt_emb_attend_forward(q, k, v, offsets_of([n]), alone, **how)
        far = q.clone()
        far[::3, 0] = 16.0
        tte.tt_emb_attend_forward(far, k, v, offsets_of([n]), beside, **how)
        p, e = weights_of(k[:, 0].double()[None])
        want = p @ v.double()
        bound = (e + 2 * product_slack(n) * p) @ v.double().abs() + want.abs() * e.sum() + rounded(F32, want)
        own = torch.arange(n, device=DEV) % 3 != 0
        check(alone, want.expand(n, dim), bound.expand(n, dim), f"alone {m}")
        check(beside[own], want.expand(n, dim)[own], bound.expand(n, dim)[own], f"beside {m}")


@pytest.mark.parametrize("length", [120, 3000])
def test_paged_parts_on_both_sides_of_the_border(length):
    """Waves and workgroups whose largest scores lie on the two sides are joined at their own weights."""
    page, dim = 16, 32
    for i in range(6):
        m = round((BORDER - 1.0 + 0.3 * i) * 16) / 16
        s = torch.full((length,), m - 1000, dtype=F64, device=DEV)
        s[:30] = m
        s[40:60] = m + 1                          # another wave's
        s[length - 25:length - 5] = m + 1.5       # another wave's, of another workgroup where there are several
        pages = (length + page - 1) // page
        kp, vp = torch.zeros(pages, page, 1, dim, device=DEV), rand(pages * page, dim, seed=2).view(pages, page, 1, dim)
        kp.view(-1, dim)[:length, 0] = s.float()
        assert torch.equal(kp.view(-1, dim)[:length, 0].double(), s)
        q = torch.zeros(1, dim, device=DEV)
        q[0, 0] = 1.0
        out = torch.empty_like(q)
        tte.tt_emb_attend_paged(q, kp, vp, torch.arange(pages, device=DEV).to(I32)[None],
                                torch.tensor([length], device=DEV), out, scale=1.0)
        p, e = weights_of(s[None])
        vi = vp.view(-1, dim)[:length].double()
        want = p @ vi
        bound = (e + 2 * product_slack(length) * p) @ vi.abs() + want.abs() * e.sum() + rounded(F32, want)
        check(out, want, bound, f"paged border {m} {length}")

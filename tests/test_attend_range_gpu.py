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


# --------------------------------------------------- gradients at large scores

# |lse| up to which the backward takes it as it is (past that it forms maximum and sum again): four roundings of it and the
# conversions' constants, 5 U32 |lse|, are then what a weight is off by
TRUSTED = {F32: 32.0, BF16: 256.0, F16: 256.0}


def parts_of(t, heads):
    """[rows, heads * dim] as [heads, rows, dim] in 64 bits."""
    return t.double().reshape(t.shape[0], heads, -1).transpose(0, 1)


def exact_backward(q, k, v, dout, heads, kv, causal, scale, score_sums=False):
    """dq, dk, dv of one sequence whose scores q . k are exact in fp32 (or, with score_sums, are off by what their sums round),
    and their bounds: those of tests/attend_ref.py, with a weight's error that does not grow with the scores."""
    t, n = q.dtype, q.shape[0]
    g = heads // kv
    u = U[t] if t != F32 else 0.0
    q, dout = parts_of(q, heads), parts_of(dout, heads)
    k, v = (parts_of(x, kv).repeat_interleave(g, 0) for x in (k, v))
    kd, kn, kq = product_slack(q.shape[2]), product_slack(n), product_slack(g * n)
    seen = torch.ones(n, n, dtype=torch.bool, device=q.device)
    if causal:
        seen = seen.tril()
    s = (scale * q @ k.mT).masked_fill(~seen, -torch.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.softmax(s, -1)
    x = (lse - s).clamp(0, 128)
    e = 8 * U32 * (1 + x) + 5 * U32 * lse.abs().clamp(max=TRUSTED[t]) + kn
    if score_sums:
        e = e + kd * scale * (q.abs() @ k.abs().mT)
    out = p @ v
    # the forward's: its weights rounded too
    bo = rounded(t, out) + (p * (e + u + kn)) @ v.abs() + out.abs() * (p * e).sum(-1, keepdim=True)
    dp = dout @ v.mT
    delta = (dout * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    ddelta = (dout.abs() * bo).sum(-1, keepdim=True) + kd * (dout * out).abs().sum(-1, keepdim=True)
    eds = p * (e * (dp - delta).abs() + kd * (dout.abs() @ v.abs().mT) + ddelta + 4 * U32 * (dp.abs() + delta.abs()))
    # weights below 2^-126 are 0: an error of that size, times what the weight is multiplied by
    eds = eds + u * (ds.abs() + eds) + 2.0 ** -126 * (dp.abs() + delta.abs()) * seen
    ep = p * (e + u)
    # f16: half a step below its normal numbers is 2^-25; the largest factor of a row (dq) and of a key over the heads that
    # share it (dk) is multiplied to 2^9 or more, none by more than 2^60; weights by 2^14
    def low(by_key):
        if t != F16:
            return 2.0 ** -126 * seen
        top = ds.abs().amax(-2, keepdim=True).view(kv, g, 1, n).amax(1).repeat_interleave(g, 0) if by_key else \
            ds.abs().amax(-1, keepdim=True)
        return (2.0 ** -34 * top + 2.0 ** -85) * seen
    group = lambda y: y.view(kv, g, n, -1).sum(1)   # noqa: E731
    dq, dk, dv = scale * ds @ k, scale * group(ds.mT @ q), group(p.mT @ dout)
    bq = rounded(t, dq) + scale * (eds + low(False) + kn * ds.abs()) @ k.abs()
    bk = rounded(t, dk) + scale * group((eds + low(True) + kq * ds.abs()).mT @ q.abs())
    bv = rounded(t, dv) + group((ep + (2.0 ** -39 if t == F16 else 2.0 ** -126) * seen + kq * p).mT @ dout.abs())
    flat = lambda y: y.transpose(0, 1).flatten(1)   # noqa: E731
    return [flat(y) for y in (dq, dk, dv)], [flat(y) for y in (bq, bk, bv)]


def check_backward(q, k, v, dout, lengths, heads, kv, causal, scale, what):
    say("attend's range", what, q.dtype, lengths, heads, kv, q.shape[1] // heads, causal, scale)
    off = offsets_of(lengths)
    out, lse = torch.empty_like(dout), torch.empty(heads, q.shape[0], device=DEV)
    how = dict(heads=heads, kv_heads=kv, causal=causal, scale=scale)
    tte.tt_emb_attend_forward(q, k, v, off, out, lse, **how)
    got = [torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in (q, k, v)]
    tte.tt_emb_attend_backward(q, k, v, off, out, lse, dout, *got, **how)
    at = 0
    for n in lengths:
        r, at = slice(at, at + n), at + n
        want, bound = exact_backward(q[r], k[r], v[r], dout[r], heads, kv, causal, scale)
        for a, w, b, name in zip(got, want, bound, ("dq", "dk", "dv")):
            check(a[r], w, b, f"{what}: {name}")


SHAPES = pytest.mark.parametrize("lengths,heads,kv,dim,pad", [
    ([300], 2, 1, 64, 0), ([100, 60], 4, 2, 128, 0), ([300], 2, 2, 128, 0), ([290], 2, 1, 33, 1), ([300, 5], 2, 1, 128, 3),
    ([20, 24, 1, 31], 4, 4, 32, 0), ([200], 64, 32, 96, 0), ([330, 182], 64, 64, 64, 0)])


def spaced(t, pad):
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


@TYPES
@SHAPES
@pytest.mark.parametrize("scale", [2.0 ** -7, 2.0 ** -3, 4.0])
def test_gradients_of_sharp_scores(dt, lengths, heads, kv, dim, pad, scale):
    """Queries and keys of whole numbers: scores of up to some 10^4 that fp32 holds."""
    rows = sum(lengths)
    q, k = (spaced((rand(rows, n * dim, seed=s) * 12).round().clamp(-40, 40).to(dt), pad) for n, s in ((heads, 1), (kv, 2)))
    v = spaced(rand(rows, kv * dim, seed=3, dt=dt), pad)
    dout = spaced((rand(rows, heads * dim, seed=4) * (2.0 ** -8 if dt == F16 else 1.0)).to(dt), pad)
    for causal in (True, False):
        check_backward(q, k, v, dout, lengths, heads, kv, causal, scale, "sharp")


@TYPES
@SHAPES
@pytest.mark.parametrize("size", [2.0 ** 4, 2.0 ** 10, 2.0 ** 13, 2.0 ** 17, 2.0 ** 24, 2.0 ** 40, 2.0 ** 100])
def test_gradients_of_huge_scores(dt, lengths, heads, kv, dim, pad, size):
    """The keys with a row's largest score share its weight, however large that is; by the operands and by the scale."""
    if dt == F16 and size > 2.0 ** 13:
        pytest.skip("gradients past f16's range")
    rows = sum(lengths)
    j = torch.arange(rows, device=DEV)
    for by_scale in (True, False):
        a, b = (1.0, size) if by_scale else (size, 1.0)
        q, k = torch.zeros(rows, heads, dim, device=DEV), torch.zeros(rows, kv, dim, device=DEV)
        q[:, :, dim // 2] = torch.where(j % 2 == 0, a, -a)[:, None]
        k[:, :, dim // 2] = (j % 50 - 25)[:, None].float()
        q, k = (spaced(t.flatten(1).to(dt), pad) for t in (q, k))
        v = spaced(rand(rows, kv * dim, seed=3, dt=dt), pad)
        dout = spaced((rand(rows, heads * dim, seed=4) * (2.0 ** -8 if dt == F16 else 1.0)).to(dt), pad)
        check_backward(q, k, v, dout, lengths, heads, kv, False, b, f"huge {size} {'scale' if by_scale else 'query'}")


@TYPES
def test_gradients_do_not_depend_on_the_rows_beside(dt):
    """Rows past what the kept sum holds do not change the gradients of the queries beside them whose sum is taken as it
    is, to the bit (given the same outputs and sums of theirs)."""
    n, dim = 200, 64
    q, k, v, d = ((rand(n, dim, seed=s) * 4).round().to(dt) for s in range(1, 5))
    off = offsets_of([n])
    own = torch.arange(n, device=DEV) % 3 != 0
    res, kept = [], None
    for far in (False, True):
        x = q.clone()
        if far:
            x[::3] *= 16.0
        out, lse = torch.empty_like(q), torch.empty(1, n, device=DEV)
        how = dict(heads=1, kv_heads=1, causal=True, scale=0.125)
        tte.tt_emb_attend_forward(x, k, v, off, out, lse, **how)
        kept = kept or (out.clone(), lse.clone())
        out[own], lse[:, own] = kept[0][own], kept[1][:, own]
        g = [torch.empty_like(q) for _ in range(3)]
        tte.tt_emb_attend_backward(x, k, v, off, out, lse, d, *g, **how)
        assert bool((lse[0].abs() > TRUSTED[dt]).any()) or not far
        res.append(g[0])
    own &= kept[1][0].abs() <= TRUSTED[dt]
    assert int(own.sum()) > 20 and torch.equal(res[0][own], res[1][own])


@TYPES
def test_sharp_attention_trained(dt):
    """The sharp scale of the forward's test, with its gradients."""
    from tests.test_attend_gpu import check_attend
    check_attend(dt, [150, 90], 2, 1, 64, scale=30.0)


# ----------------------------------------------------- f16: the size of gradients

@pytest.mark.parametrize("lengths,heads,kv,dim,pad", [
    ([2048], 2, 1, 64, 0), ([1500], 2, 2, 128, 0), ([1111], 2, 1, 33, 1), ([900], 1, 1, 128, 3), ([120, 100, 128], 4, 2, 32, 0),
    ([700], 64, 32, 64, 0)])
@pytest.mark.parametrize("size", [2.0 ** -6, 2.0 ** -10, 2.0 ** -13])
@pytest.mark.parametrize("large", ["q", "k"])
def test_small_f16_gradients(lengths, heads, kv, dim, pad, size, large):
    """Gradients of the outputs far below 1, whose products with weights are below f16's range: those of queries, keys and
    values keep their digits. Large keys or queries bring the results back into it."""
    rows = sum(lengths)
    sq, sk = (2.0 ** 5, 2.0 ** -5) if large == "q" else (2.0 ** -5, 2.0 ** 5)
    q, k, v, dout = (spaced((rand(rows, n * dim, seed=s) * m).to(F16), pad) for n, s, m in (
        (heads, 1, sq), (kv, 2, sk), (kv, 3, 0.25), (heads, 4, size)))
    # scores of unit normals, not exact: 64 bits' of the same operands, within their sums' roundings
    check_small(q, k, v, dout, lengths, heads, kv, dim ** -0.5, "small")


@pytest.mark.parametrize("lengths,heads,kv,dim,pad", [([8, 31], 4, 2, 64, 0), ([300], 2, 1, 128, 0), ([40], 2, 1, 33, 1)])
def test_large_f16_gradients(lengths, heads, kv, dim, pad):
    """Products of the outputs' gradients with the values past f16's range, where the results are within it."""
    rows = sum(lengths)
    q, k, v, dout = (spaced((rand(rows, n * dim, seed=s) * m).to(F16), pad) for n, s, m in (
        (heads, 1, 2.0 ** -7), (kv, 2, 2.0 ** -7), (kv, 3, 2.0 ** 5), (heads, 4, 2.0 ** 10)))
    dp = parts_of(dout, heads)[0, :8] @ parts_of(v, kv)[0, :8].mT
    assert float(dp.abs().max()) > 2 * 65504
    check_small(q, k, v, dout, lengths, heads, kv, dim ** -0.5, "large")


def check_small(q, k, v, dout, lengths, heads, kv, scale, what):
    """check_backward with the roundings of scores that are not exact, in fp32 sums: what they take to weights and through
    them to the results, beside its bounds."""
    off = offsets_of(lengths)
    say("attend's f16 gradients", what, lengths, heads, kv, q.shape[1] // heads, float(dout.abs().max()))
    out, lse = torch.empty_like(dout), torch.empty(heads, q.shape[0], device=DEV)
    how = dict(heads=heads, kv_heads=kv, causal=False, scale=scale)
    tte.tt_emb_attend_forward(q, k, v, off, out, lse, **how)
    got = [torch.empty(t.shape, dtype=t.dtype, device=DEV) for t in (q, k, v)]
    tte.tt_emb_attend_backward(q, k, v, off, out, lse, dout, *got, **how)
    at = 0
    for n in lengths:
        r, at = slice(at, at + n), at + n
        want, bound = exact_backward(q[r], k[r], v[r], dout[r], heads, kv, False, scale, score_sums=True)
        for a, w, b, name in zip(got, want, bound, ("dq", "dk", "dv")):
            check(a[r], w, b, f"{what}: {name}")


# ------------------------------------------------------- the paged form's weights

@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("lengths,heads,kv,dim,page", [
    ([5000], 8, 2, 128, 16), ([255, 1, 33, 700], 4, 2, 64, 16), ([900, 2], 10, 5, 80, 49), ([40] * 9, 4, 4, 33, 8)])
def test_paged_weights_are_not_rounded_to_the_caches_type(dt, lengths, heads, kv, dim, page):
    """Outputs are off by their own rounding and fp32's sums; weights, in two parts of the type, by its square."""
    from tests.test_attend_gpu import pool
    say("paged weights", dt, lengths, heads, kv, dim, page)
    kp, vp, table = pool(dt, lengths, kv, dim, page)
    q = (1.5 * rand(len(lengths), heads * dim, seed=3)).to(dt)
    out = torch.empty_like(q)
    scale = dim ** -0.5
    tte.tt_emb_attend_paged(q, kp, vp, table, torch.tensor(lengths, device=DEV), out)
    g = heads // kv
    want, bound = (torch.empty(len(lengths), heads, dim, dtype=F64, device=DEV) for _ in range(2))
    kd = product_slack(dim)
    for i, n in enumerate(lengths):
        j = torch.arange(n, device=DEV)
        slot = table[i].long()[j // page] * page + j % page
        k, v = (x.view(-1, kv, dim)[slot].double().transpose(0, 1).repeat_interleave(g, 0) for x in (kp, vp))
        x = q[i].double().view(heads, 1, dim)
        s = scale * x @ k.mT
        p = torch.softmax(s, -1)
        e = kd * scale * (x.abs() @ k.abs().mT) + 4 * U32 * (1 + s.abs())
        kn = product_slack(2 * n)
        # (f16: weights are at 2^8 of the largest, half a step below its normal numbers is 2^-25)
        low = 2.0 ** -33 * p.amax(-1, keepdim=True) if dt == F16 else 2.0 ** -126
        o = p @ v
        b = rounded(dt, o) + (p * (e + 2 * U[dt] ** 2 + kn) + low) @ v.abs() + o.abs() * ((p * e).sum(-1, keepdim=True) + kn)
        want[i], bound[i] = o[:, 0], b[:, 0]
    check(out, want.flatten(1), bound.flatten(1), "paged weights")


# ----------------------------------------------------------- slots named twice

@TYPES
def test_append_to_slots_named_twice(dt):
    """Each element of such a slot is one of the rows' that name it; the other slots and the queries are as ever."""
    rows, heads, kv, dim = 60, 8, 4, 128
    q, k, v = (rand(rows, n * dim, seed=s, dt=dt) for n, s in ((heads, 1), (kv, 2), (kv, 3)))
    w, pos = torch.ones(dim, device=DEV), torch.arange(rows, device=DEV)
    freq = torch.tensor([0.1 * i for i in range(dim // 2)], dtype=F64, device=DEV)
    slots = torch.arange(rows, device=DEV) + 3
    slots[10], slots[40], slots[41] = slots[11].item(), slots[50].item(), slots[50].item()
    caches = [torch.full((80, kv * dim), 7.0, dtype=dt, device=DEV) for _ in range(2)]
    q_out = torch.empty_like(q)
    tte.tt_emb_rotate_append(q, k, v, w, w, pos, freq, slots, q_out, *(c.view(10, 8, kv, dim) for c in caches))
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    tte.tt_emb_rotate_forward(q, k, w, w, pos, freq, want_q, want_k)
    assert torch.equal(q_out, want_q)
    for c, rows_of in zip(caches, (want_k, v)):
        for slot in range(80):
            named = (slots == slot).nonzero().flatten()
            if not named.numel():
                assert bool((c[slot] == 7.0).all())
            else:
                assert bool((c[slot] == rows_of[named]).any(0).all()), slot


@TYPES
@pytest.mark.parametrize("length", [70, 3000])
def test_paged_infinities_stay_in_their_element(dt, length):
    """An infinity in a seen value reaches its element of the heads that read it, one in a token that is not seen nothing; a
    key whose scores are -inf is not seen."""
    heads, kv, dim, page = 4, 2, 64, 16
    pages = (length + page - 1) // page
    kp, vp = (rand(pages, page, kv, dim, seed=s, dt=dt) for s in (1, 2))
    q = rand(1, heads * dim, seed=3, dt=dt)
    table, lens = torch.arange(pages, device=DEV).to(I32)[None], torch.tensor([length - 3], device=DEV)
    good = torch.empty_like(q)
    tte.tt_emb_attend_paged(q, kp, vp, table, lens, good)
    bad = torch.empty_like(q)
    vp.view(-1, kv, dim)[length - 3:length, :] = float("inf")      # behind the sequence's last
    kp.view(-1, kv, dim)[length - 3:length, :] = float("nan")
    tte.tt_emb_attend_paged(q, kp, vp, table, lens, bad)
    assert torch.equal(good, bad)
    for value in (float("inf"), -float("inf"), float("nan")):
        vp.view(-1, kv, dim)[5, 1, 7] = value
        tte.tt_emb_attend_paged(q, kp, vp, table, lens, bad)
        hit = torch.zeros(heads, dim, dtype=torch.bool, device=DEV)
        hit[2:, 7] = True
        assert torch.equal(~torch.isfinite(bad.view(heads, dim)), hit)
        assert torch.equal(bad.view(heads, dim)[~hit], good.view(heads, dim)[~hit])
    # keys whose scores are -inf: as if they were not there
    vp.view(-1, kv, dim)[5, 1, 7] = 0.0
    kp.view(-1, kv, dim)[9, :, 3] = -float("inf")
    x = q.clone().view(heads, dim)
    x[:, 3] = x[:, 3].abs() + 0.5
    x = x.view(1, -1)
    tte.tt_emb_attend_paged(x, kp, vp, table, lens, bad)
    keep = torch.tensor([j for j in range(length - 3) if j != 9], device=DEV)
    k2, v2 = (torch.zeros(pages * page, kv, dim, dtype=dt, device=DEV) for _ in range(2))
    k2[:len(keep)], v2[:len(keep)] = kp.view(-1, kv, dim)[keep], vp.view(-1, kv, dim)[keep]
    want, bound = ref.paged(x, k2.view(pages, page, kv, dim), v2.view(pages, page, kv, dim), table, lens - 1, dim ** -0.5)
    check(bad, want, bound, "beside a key of -inf")


# ------------------------------------------------------ norms at the range's ends

@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_rotate_heads_past_the_range(dt):
    """A head whose squares overflow gives 0, and its gradients; one whose squares underflow gives u = x / sqrt(eps), without
    eps nothing finite. No other head of the row changes."""
    rows, heads, dim = 4, 3, 32
    q, k = rand(rows, heads * dim, seed=1, dt=dt), rand(rows, heads * dim, seed=2, dt=dt)
    w, pos = torch.ones(dim, device=DEV), torch.zeros(rows, dtype=I64, device=DEV)
    freq = torch.ones(0, dtype=F64, device=DEV)
    dy = rand(rows, heads * dim, seed=3, dt=dt)

    def both(x, eps):
        y, ko, dx, dk = (torch.empty_like(q) for _ in range(4))
        dw = [torch.empty_like(w) for _ in range(2)]
        tte.tt_emb_rotate_forward(x, k, w, w, pos, freq, y, ko, eps=eps)
        tte.tt_emb_rotate_backward(x, k, w, w, pos, freq, dy, dy, dx, dk, *dw, eps=eps)
        return y.view(rows, heads, dim), dx.view(rows, heads, dim)
    x = q.clone()
    x[1, :dim] = (q[1, :dim].float() * 1e25).to(dt)
    x[2, dim:2 * dim] = (q[2, dim:2 * dim].float() * 1e-25).to(dt)
    others = torch.ones(rows, heads, dtype=torch.bool, device=DEV)
    others[1, 0] = others[2, 1] = False
    for eps in (1e-6, 0.0):
        (y0, d0), (y, d) = both(q, eps), both(x, eps)
        assert torch.equal(y[others], y0[others]) and torch.equal(d[others], d0[others])
        assert bool((y[1, 0] == 0).all() and (d[1, 0] == 0).all())
        if eps:
            want = x.view(rows, heads, dim)[2, 1].double() / eps ** 0.5
            check(y[2, 1], want, rounded(dt, want) + 8 * U32 * want.abs(), "below eps")
        else:
            assert not bool(torch.isfinite(y[2, 1]).any())


# ------------------------------------------------------------- graphs, streams

class Step:
    """One training step of attention on buffers of its own."""

    def __init__(self, dt, seed):
        self.dt, self.heads, self.kv, self.dim, self.rows = dt, 8, 2, 64, 400
        self.q, self.k, self.v, self.d = (rand(self.rows, n * self.dim, seed=seed + i, dt=dt)
                                          for i, n in enumerate((self.heads, self.kv, self.kv, self.heads)))
        self.off = offsets_of([150, 0, 230, 20])
        size = tte.tt_emb_attend_workspace_bytes(dt, self.rows, self.heads, self.kv, self.dim)
        self.ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        self.res = self.buffers()

    def buffers(self):
        return [torch.zeros_like(t) for t in (self.q, self.q, self.k, self.v)] + [torch.zeros(self.heads, self.rows, device=DEV)]

    def run(self, res, stream=None):
        out, dq, dk, dv, lse = res
        how = dict(heads=self.heads, kv_heads=self.kv, scale=0.125, stream=stream)
        tte.tt_emb_attend_forward(self.q, self.k, self.v, self.off, out, lse, **how)
        tte.tt_emb_attend_backward(self.q, self.k, self.v, self.off, out, lse, self.d, dq, dk, dv, workspace=self.ws, **how)


@TYPES
def test_captured_backward_from_near_scores_to_far_and_back(dt):
    """Which rows form their sum again is found on the device: a captured step does as the eager one for every input."""
    s = Step(dt, 1)
    s.run(s.res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(s.res)
    for i, (far, grad) in enumerate(((1.0, 1.0), (3000.0, 2.0 ** -8), (1.0, 2.0 ** -12), (300.0, 1.0))):
        q = rand(*s.q.shape, seed=20 + i)
        q[::2] *= far
        s.q.copy_(q.to(dt))
        s.d.copy_((rand(*s.d.shape, seed=30 + i) * grad).to(dt))
        graph.replay()
        got = [t.clone() for t in s.res]
        torch.cuda.synchronize()
        assert (float(got[4].abs().max()) > TRUSTED[dt]) == (far > 1)
        eager = s.buffers()
        s.run(eager)
        for a, b in zip(got, eager):
            assert bool(torch.isfinite(a).all()) and torch.equal(a, b), i


@TYPES
def test_two_steps_at_once(dt):
    """Two steps on two streams, one of far scores, each with a workspace of its own."""
    steps = [Step(dt, 1), Step(dt, 11)]
    steps[1].q.mul_(300.0)
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        s.run(s.res)
    got = [s.buffers() for s in steps]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, st, g in zip(steps, streams, got):
            s.run(g, stream=st)
    torch.cuda.synchronize()
    for s, g in zip(steps, got):
        for a, b in zip(s.res, g):
            assert torch.equal(a, b)

"""The attention operators' kernels against their 64-bit definitions, at the
sizes, layouts, strides, types and values where they can go wrong. The bounds
are those of tests/attend_ref.py, which count roundings."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import tensor_train_compressed_amd as tte  # noqa: E402
from tests import attend_ref as ref  # noqa: E402
from tests.dense_ref import check  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402
from tests.test_dense_gpu import BF16, F16, F32, INF, NAN, TYPES, hole, padded, rand, untouched  # noqa: E402

I64, F64, I32 = torch.int64, torch.float64, torch.int32


def freqs(half, base=10000.0):
    return base ** (-torch.arange(half, dtype=F64, device=DEV) / max(half, 1))


# ------------------------------------------------------------------- rotation

def check_rotate(dt, wt, rows, heads, kv, dim, rot, pairs, pad=0, off=0, start=0, backward=True, eps=1e-6):
    say("rotate", dt, wt, rows, heads, kv, dim, rot, pairs, "pad", pad, "off", off)
    x = [rand(rows, n * dim, seed=i) * torch.exp(0.5 * rand(rows, 1, seed=9)) for i, n in ((1, heads), (2, kv))]
    q, k = (padded(t.to(dt), pad, off) for t in x)
    wq, wk = ((1 + 0.1 * rand(dim, seed=i)).to(wt) for i in (3, 4))
    pos = start + 37 * torch.arange(rows, device=DEV)
    freq = freqs(rot // 2)
    outs = [hole(rows, n * dim, dt, pad, off) for n in (heads, kv)]
    turn = (wq, wk, pos, freq)
    tte.tt_emb_rotate_forward(q, k, *turn, outs[0][0], outs[1][0], pairs=pairs, eps=eps)
    grads = None
    if backward:
        dy = [padded(rand(rows, n * dim, seed=i, dt=dt), pad, off) for i, n in ((5, heads), (6, kv))]
        dx = [hole(rows, n * dim, dt, pad, off) for n in (heads, kv)]
        dw = [torch.full_like(wq, NAN), torch.full_like(wk, NAN)]
        ws = torch.full((tte.tt_emb_rotate_workspace_bytes(dt, rows, heads, kv, dim),), 255, dtype=torch.uint8, device=DEV)
        tte.tt_emb_rotate_backward(q, k, *turn, *dy, dx[0][0], dx[1][0], *dw, pairs=pairs, eps=eps, workspace=ws)
        grads = dx, dw
    for i, (x, w, what) in enumerate(((q, wq, "q"), (k, wk, "k"))):
        if rows:
            untouched(*outs[i])
        args = (x, w, pos, freq, dim, pairs, eps)
        d = dy[i] if backward else None
        b = ref.rotate_bounds(*args, d, wt)
        check(outs[i][0], ref.rotate(*args)[0], b[0] if backward else b, f"{what} out")
        if backward:
            if rows:
                untouched(*dx[i])
            wx, ww = ref.rotate_grads(*args, d)
            check(dx[i][0], wx, b[1], f"d{what}")
            check(dw[i], ww, b[2], f"d{what} weight")
    return outs[0][0], outs[1][0], grads


@TYPES
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("rows,heads,kv,dim,rot,pad,off", [
    (1, 1, 1, 1, 0, 0, 0), (1, 1, 1, 2, 2, 0, 0), (3, 2, 1, 7, 4, 1, 1), (5, 4, 2, 16, 16, 0, 0), (2, 3, 3, 33, 32, 3, 0),
    (70, 10, 5, 80, 20, 3, 0), (9, 32, 8, 128, 128, 0, 0), (9, 32, 8, 128, 100, 8, 0), (5, 7, 1, 101, 100, 0, 1),
    (4, 2, 2, 256, 256, 0, 0), (3, 5, 1, 255, 34, 1, 1), (33, 1, 1, 64, 2, 0, 0), (4, 70, 70, 40, 40, 0, 0)])
def test_rotate_sizes(dt, pairs, rows, heads, kv, dim, rot, pad, off):
    check_rotate(dt, dt, rows, heads, kv, dim, rot, pairs, pad, off, start=5)


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
def test_rotate_fp32_weights(dt):
    check_rotate(dt, F32, 50, 6, 2, 72, 72, "halves")


def test_rotate_many_rows():
    """More rows than one pass of the backward's workgroups takes, and the forward with a wave a row."""
    check_rotate(F32, F32, 9001, 3, 1, 24, 24, "neighbours")
    check_rotate(BF16, F32, 5000, 2, 2, 128, 128, "halves")


def test_rotate_no_rows():
    check_rotate(F32, F32, 0, 2, 1, 16, 8, "halves")


@pytest.mark.parametrize("start", [-1000, 100000, 1 << 24, (1 << 31) + 12345])
def test_rotate_far_positions(start):
    """Positions whose angles fp32 does not hold."""
    check_rotate(F32, F32, 6, 2, 1, 64, 64, "halves", start=start)


def test_rotate_bad_heads_stay_apart():
    """A head with NaN or an infinity makes that head NaN (an infinity: where it is and its pair) and no other; zero heads
    are zeros."""
    q, k = rand(4, 64, seed=1), rand(4, 32, seed=2)
    w, pos, freq = 1 + 0.1 * rand(32, seed=3), torch.arange(4, device=DEV), freqs(8)
    good = torch.empty_like(q), torch.empty_like(k)
    tte.tt_emb_rotate_forward(q, k, w, w, pos, freq, *good)
    q2, k2 = q.clone(), k.clone()
    q2[1, 3], q2[2, 32 + 20], k2[3] = NAN, INF, 0.0
    got = torch.empty_like(q), torch.empty_like(k)
    tte.tt_emb_rotate_forward(q2, k2, w, w, pos, freq, *got)
    assert bool(got[0][1, :32].isnan().all()) and torch.equal(got[0][1, 32:], good[0][1, 32:])
    want = torch.zeros(32, device=DEV)
    want[20] = NAN                                    # not rotated: it alone
    assert torch.equal(got[0][2, 32:].isnan(), want.isnan()) and bool((got[0][2, 32:][~want.isnan()] == 0).all())
    assert torch.equal(got[0][[0, 3]], good[0][[0, 3]]) and torch.equal(got[1][:3], good[1][:3])
    assert bool((got[1][3] == 0).all())


@TYPES
@pytest.mark.parametrize("rows,heads,kv,dim,rot,page,pad", [
    (1, 32, 8, 128, 128, 16, 0), (1, 1, 1, 1, 0, 1, 0), (37, 6, 3, 80, 20, 7, 3), (300, 4, 4, 33, 32, 49, 1),
    (5000, 2, 1, 64, 64, 64, 0)])
def test_rotate_append(dt, rows, heads, kv, dim, rot, page, pad):
    say("rotate append", dt, rows, heads, kv, dim, rot, page)
    qkv = padded(rand(rows, (heads + 2 * kv) * dim, seed=1, dt=dt), pad)
    q, k, v = qkv[:, :heads * dim], qkv[:, heads * dim:(heads + kv) * dim], qkv[:, (heads + kv) * dim:]
    v[0, 0] = NAN                                     # values go as they are
    w, pos, freq = (1 + 0.1 * rand(dim, seed=3)).to(dt), torch.arange(rows, device=DEV) + 11, freqs(rot // 2)
    pages = (rows + page - 1) // page + 2
    slots = torch.randperm(pages * page, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)[:rows]
    if rows > 4:
        slots[1], slots[2], slots[3] = -1, pages * page, 1 << 40
    caches = [torch.full((pages * page * kv * dim + 5,), 77.0, dtype=dt, device=DEV) for _ in range(2)]
    kp, vp = (c[:-5].view(pages, page, kv, dim) for c in caches)
    q_out, q_wide = hole(rows, heads * dim, dt, pad)
    tte.tt_emb_rotate_append(q, k, v, w, w, pos, freq, slots, q_out, kp, vp)
    want_q, want_k = torch.empty(rows, heads * dim, dtype=dt, device=DEV), torch.empty(rows, kv * dim, dtype=dt, device=DEV)
    tte.tt_emb_rotate_forward(q, k, w, w, pos, freq, want_q, want_k)
    assert torch.equal(q_out, want_q)
    untouched(q_out, q_wide)
    keep = (slots >= 0) & (slots < pages * page)
    for c, rows_of in ((caches[0], want_k), (caches[1], v)):
        want = torch.full_like(c, 77.0)
        want[:-5].view(-1, kv * dim)[slots[keep]] = rows_of[keep]
        assert torch.equal(c.view(torch.uint8), want.view(torch.uint8))


# ------------------------------------------------------------------ attention

def packed(dt, rows, heads, kv, dim, pad=0, seed=1, size=1.5):
    """q, k and v as parts of one projection's rows."""
    wide = rand(rows, (heads + 2 * kv) * dim + pad, seed=seed)
    wide[:, :heads * dim] *= size
    wide = wide.to(dt)
    return wide[:, :heads * dim], wide[:, heads * dim:(heads + kv) * dim], wide[:, (heads + kv) * dim:(heads + 2 * kv) * dim]


def offsets_of(lengths, first=0):
    return torch.cumsum(torch.tensor([first, *lengths], dtype=I64, device=DEV), 0)


def run_attend(q, k, v, off, heads, kv, causal, scale, dout=None, pad=0, alone=True):
    """Outputs in buffers marked around them and where no sequence is; out, lse and, with dout, dq, dk, dv."""
    rows, dim, dt = q.shape[0], q.shape[1] // heads, q.dtype
    how = dict(heads=heads, kv_heads=kv, causal=causal, scale=scale)
    outs = [hole(rows, heads * dim, dt, pad)]
    lse = torch.full((heads, rows), 77.0, device=DEV)
    tte.tt_emb_attend_forward(q, k, v, off, outs[0][0], lse, **how)
    if alone:   # the form that serves: the same bits without lse
        bits = I32 if dt == F32 else torch.int16
        o = torch.full_like(outs[0][0], 77.0)
        tte.tt_emb_attend_forward(q, k, v, off, o, **how)
        assert torch.equal(o.contiguous().view(bits), outs[0][0].contiguous().view(bits))
    if dout is not None:
        outs += [hole(rows, n * dim, dt, pad) for n in (heads, kv, kv)]
        ws = torch.full((tte.tt_emb_attend_workspace_bytes(dt, rows, heads, kv, dim),), 255, dtype=torch.uint8, device=DEV)
        tte.tt_emb_attend_backward(q, k, v, off, outs[0][0], lse, dout, *(o[0] for o in outs[1:]), workspace=ws, **how)
    for o in outs:
        untouched(*o)
    return [outs[0][0], lse] + [o[0] for o in outs[1:]]


def check_attend(dt, lengths, heads, kv, dim, causal=True, scale=None, first=0, tail=0, pad=0, train=True, size=1.5):
    say("attend", dt, lengths, heads, kv, dim, "causal" if causal else "full", "first", first, "tail", tail, "pad", pad)
    rows = first + sum(lengths) + tail
    scale = dim ** -0.5 if scale is None else scale
    q, k, v = packed(dt, rows, heads, kv, dim, pad, size=size)
    dout = padded(rand(rows, heads * dim, seed=7, dt=dt), pad) if train else None
    # rows of no sequence hold what must reach nobody
    for t in (q, k, v, dout) if train else (q, k, v):
        t[:first], t[rows - tail:] = NAN, INF
    got = run_attend(q, k, v, offsets_of(lengths, first), heads, kv, causal, scale, dout, pad)
    want, bound = ref.attend(q, k, v, lengths, first, heads, kv, causal, scale, dout)
    end = rows - tail
    for i, what in enumerate(("out", "lse", "dq", "dk", "dv")[:len(got)]):
        a, w, b = (got[i].t(), want[i].t(), bound[i].t()) if what == "lse" else (got[i], want[i], bound[i])
        assert bool((a[:first] == 77.0).all() and (a[end:] == 77.0).all()), f"{what}: rows of no sequence were written"
        check(a[first:end], w[first:end], b[first:end], what)
    return got


@TYPES
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("lengths,heads,kv,dim,pad", [
    ([1], 1, 1, 1, 0), ([1, 0, 2, 0, 0, 31], 2, 1, 8, 0), ([31, 33, 1, 0, 64, 65], 4, 2, 32, 8), ([127, 129], 3, 3, 33, 1),
    ([300], 4, 1, 64, 0), ([130, 5, 257], 6, 3, 72, 5), ([40, 128], 2, 2, 96, 0), ([200, 1, 63], 8, 2, 128, 0),
    ([17, 24, 3, 21, 19, 31, 1, 22, 100, 9, 20, 14, 0, 25, 12, 8] * 5, 4, 4, 32, 0), ([77, 150], 2, 1, 127, 3)])
def test_attend_sizes(dt, causal, lengths, heads, kv, dim, pad):
    check_attend(dt, lengths, heads, kv, dim, causal, first=3, tail=5, pad=pad)


@TYPES
@pytest.mark.parametrize("dim", [16, 40, 64, 101, 128])
def test_attend_long(dt, dim):
    check_attend(dt, [1000, 523], 2, 1, dim)


@TYPES
@pytest.mark.parametrize("dim", [32, 64, 128])
def test_attend_many_heads(dt, dim):
    """As many tiles of keys as fill the chip: sums that are not split."""
    check_attend(dt, [600, 424], 64, 64, dim)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[128, 128, 128], [128, 130, 128], [255, 256, 257, 258]])
def test_attend_around_the_kernels_choices(dt, lengths):
    """Sequences around what one wave takes, and around what forms delta from the weights."""
    check_attend(dt, lengths, 4, 2, 64)
    check_attend(dt, lengths, 2, 2, 128, causal=False)


def test_attend_many_sequences():
    """More than 64, and more than 64 x 64, sequences to look through; most of them empty."""
    check_attend(BF16, [3, 0, 5, 1] * 60, 2, 1, 32)
    lengths = [0] * 9000
    for i in range(0, 9000, 97):
        lengths[i] = 1 + i % 40
    check_attend(F16, lengths, 1, 1, 16)


def test_attend_nothing():
    """No rows, no sequences, sequences without rows: nothing is written."""
    for rows, lengths in ((0, [0]), (5, []), (5, [0, 0, 0])):
        q, k, v = packed(BF16, rows, 2, 1, 16)
        d = rand(rows, 32, seed=3, dt=BF16)
        for t in run_attend(q, k, v, offsets_of(lengths), 2, 1, True, 1.0, d):
            assert bool((t == 77.0).all())


def test_attend_sequences_stay_apart():
    """NaN and infinities of one sequence reach no other, in no output."""
    lengths = [70, 45, 130]
    for dt in (F32, BF16):
        q, k, v = packed(dt, 245, 4, 2, 64)
        d = rand(245, 256, seed=7, dt=dt)
        off = offsets_of(lengths)
        good = run_attend(q, k, v, off, 4, 2, True, 0.125, d)
        for t in (q, k, v, d):
            t[70:115] = torch.tensor([NAN, INF, -INF], dtype=dt, device=DEV)[torch.arange(45, device=DEV) % 3][:, None]
        bad = run_attend(q, k, v, off, 4, 2, True, 0.125, d)
        for i, (a, b) in enumerate(zip(good, bad)):
            a, b = (a.t(), b.t()) if i == 1 else (a, b)
            assert torch.equal(a[:70], b[:70]) and torch.equal(a[115:], b[115:])
            assert bool(b[70:115].isnan().any())


@TYPES
@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_attend_flat_and_sharp(dt, scale):
    """Weights that are all alike, and weights of which one is all."""
    check_attend(dt, [150, 90], 2, 1, 64, scale=scale, train=scale < 1)


def test_attend_huge_scores():
    """Scores whose differences are past any exponent: the largest takes all, whatever their size; a score of -inf is
    not seen."""
    for dt, size in ((F32, 1e15), (F32, 1e6), (BF16, 1e9), (F16, 200.0)):
        n, dim = 140, 32
        k = torch.zeros(n, dim, device=DEV)
        k[:, 0] = torch.arange(n, device=DEV) % 50 - 25
        q = torch.zeros(n, dim, device=DEV)
        q[:, 0] = torch.where(torch.arange(n, device=DEV) % 2 == 0, size, -size)
        v = rand(n, dim, seed=3)
        q, k, v = (t.to(dt) for t in (q, k, v))
        out, lse = torch.empty_like(q), torch.empty(1, n, device=DEV)
        tte.tt_emb_attend_forward(q, k, v, offsets_of([n]), out, lse, heads=1, kv_heads=1, causal=False, scale=float(size))
        top = torch.where(torch.arange(n, device=DEV) % 2 == 0, 24.0, -25.0)
        want = torch.stack([v[k[:, 0].float() == t].double().mean(0) for t in top])
        check(out, want, 3 * ref.U[dt] * v.double().abs().max() * torch.ones_like(want), f"huge {dt} {size}")
        check(lse[0], q[:, 0].double() * top.double() * size, 4 * ref.U32 * 25.0 * size * q[:, 0].double().abs() + 8, "lse")
    k = rand(100, 16, seed=1)
    k[::3] = -INF
    q, v = rand(100, 16, seed=2).abs(), rand(100, 16, seed=3)
    out, lse = torch.empty_like(q), torch.empty(1, 100, device=DEV)
    tte.tt_emb_attend_forward(q, k, v, offsets_of([100]), out, lse, heads=1, kv_heads=1, scale=0.25)
    assert bool((out[0] == 0).all()) and float(lse[0, 0]) == -INF       # sees its own key alone
    keep = torch.arange(100, device=DEV) % 3 != 0
    want, bound = ref.attend(q[keep], k[keep], v[keep], [66], 0, 1, 1, True, 0.25)
    check(out[keep], want[0], bound[0], "beside -inf")


def test_attend_spread_weights_f16():
    """One score far above very many alike ones: f16 weights keep the digits of the many."""
    n, dim = 8192, 32
    q, k = torch.zeros(n, dim, dtype=F16, device=DEV), torch.zeros(n, dim, dtype=F16, device=DEV)
    q[:, 0], k[0, 0] = 1.0, 12.0
    v = rand(n, dim, seed=1, dt=F16) + 1
    check_rows = slice(n - 64, n)
    out = torch.empty_like(q)
    tte.tt_emb_attend_forward(q, k, v, offsets_of([n]), out, heads=1, kv_heads=1, causal=False, scale=1.0)
    w = torch.exp(12.0 * (torch.arange(n, device=DEV) == 0).double() - 12.0)
    want = (w[:, None] * v.double()).sum(0) / w.sum()
    # each weight is off by half a step of f16, all those alike the same way
    bound = 3 * ref.U[F16] * (w[:, None] * v.double().abs()).sum(0) / w.sum()
    check(out[check_rows], want.expand(64, dim), bound.expand(64, dim), "spread")


def test_attend_bad_offsets_stay_inside():
    """Offsets that decrease or lie outside the rows: whatever comes out, nothing outside the tensors is touched."""
    q, k, v = packed(BF16, 300, 2, 1, 64)
    d = rand(300, 128, seed=3, dt=BF16)
    for off in ([0, 200, 100, 300], [-50, 100, 5000], [1 << 40, -(1 << 40), 1 << 62], [300, 0], [250, 250, 0, 400, 10]):
        say("bad offsets", off)
        run_attend(q, k, v, torch.tensor(off, dtype=I64, device=DEV), 2, 1, True, 0.125, d, alone=False)
    torch.cuda.synchronize()


def test_attend_same_bits_again():
    q, k, v = packed(BF16, 700, 8, 2, 128)
    d = rand(700, 1024, seed=3, dt=BF16)
    off = offsets_of([333, 0, 360])
    a, b = (run_attend(q, k, v, off, 8, 2, True, 0.1, d) for _ in range(2))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_attend_gradients_against_differences():
    """fp32 outputs differenced along one direction: good to their rounding over the step, and the step squared."""
    heads, kv, dim, n = 4, 2, 32, 150
    q, k, v = (t.contiguous() for t in packed(F32, n, heads, kv, dim))
    d = rand(n, heads * dim, seed=7)
    off = offsets_of([n])
    got = run_attend(q, k, v, off, heads, kv, True, 0.2, d)
    h = 2.0 ** -7
    for i in range(3):
        along = rand(n, (heads, kv, kv)[i] * dim, seed=20 + i)
        ends = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * along
            out = torch.empty_like(q)
            tte.tt_emb_attend_forward(*x, off, out, heads=heads, kv_heads=kv, scale=0.2)
            ends.append((out.double() * d.double()).sum())
        slope = float(ends[0] - ends[1]) / (2 * h)
        want = float((got[2 + i].double() * along.double()).sum())
        # third derivatives of a softmax along unit-normal directions are of the sum's own size; scores move by
        # 0.2 |q| |along| ~ 6 a unit step
        size = float((got[2 + i].double().abs() * along.double().abs()).sum())
        assert abs(slope - want) <= (6 * h) ** 2 / 6 * size, (i, slope, want, size)


# ---------------------------------------------------------------------- paged

def pool(dt, lengths, kv, dim, page, extra=3, seed=5, wide=0):
    """A cache whose unused places hold NaN, and the table of its pages in no order, -1 where none is given."""
    used = [(n + page - 1) // page for n in lengths]
    pages = sum(used) + extra
    g = torch.Generator(device=DEV).manual_seed(seed)
    order = torch.randperm(pages, generator=g, device=DEV).to(I32)
    table = torch.full((len(lengths), max([1, *used]) + wide), -1, dtype=I32, device=DEV)
    kp, vp = (torch.full((pages, page, kv, dim), NAN, dtype=dt, device=DEV) for _ in range(2))
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
        if lengths[i]:
            j = torch.arange(lengths[i], device=DEV)
            slot = table[i].long()[j // page] * page + j % page
            for p in (kp, vp):
                p.view(-1, kv, dim)[slot] = torch.randn(lengths[i], kv, dim, generator=g, device=DEV).to(dt)
    return kp, vp, table


def check_paged(dt, lengths, heads, kv, dim, page, scale=None, pad=0, lens=None, pools=None, size=1.5):
    say("paged", dt, lengths, heads, kv, dim, "page", page, "pad", pad)
    kp, vp, table = pools or pool(dt, lengths, kv, dim, page)
    n = len(lengths)
    q = padded((size * rand(n, heads * dim, seed=3)).to(dt), pad)
    out, wide = hole(n, heads * dim, dt, pad)
    lens = torch.tensor(lengths, dtype=I64, device=DEV) if lens is None else lens
    ws = torch.full((tte.tt_emb_attend_paged_workspace_bytes(dt, n, heads, kv, dim),), 255, dtype=torch.uint8, device=DEV)
    scale = dim ** -0.5 if scale is None else scale
    tte.tt_emb_attend_paged(q, kp, vp, table, lens, out, scale=scale, workspace=ws)
    untouched(out, wide)
    want, bound = ref.paged(q, kp, vp, table, lens, scale)
    check(out, want, bound, "paged")
    return out


@TYPES
@pytest.mark.parametrize("lengths,heads,kv,dim,page,pad", [
    ([1], 1, 1, 1, 1, 0), ([0], 2, 1, 8, 16, 0), ([3, 0, 64, 1, 0, 65], 4, 4, 32, 64, 0), ([255, 256, 257], 8, 2, 128, 16, 0),
    ([5000], 32, 8, 128, 16, 8), ([700, 31, 33], 10, 5, 80, 49, 1), ([1000, 2], 7, 1, 33, 7, 0), ([300, 511], 40, 1, 64, 1, 3),
    ([600], 128, 2, 96, 300, 0), ([129, 1300], 6, 3, 101, 32, 0), ([20] * 70, 4, 2, 16, 8, 0)])
def test_paged_sizes(dt, lengths, heads, kv, dim, page, pad):
    check_paged(dt, lengths, heads, kv, dim, page, pad=pad)


@TYPES
def test_paged_long(dt):
    """Split over many workgroups and joined."""
    check_paged(dt, [40000, 17, 12345], 8, 2, 64, 16)


def test_paged_lengths_out_of_range():
    """A length past the table counts as the table's, one below zero as zero."""
    pools = pool(BF16, [64, 64, 64], 2, 32, 16)
    lens = torch.tensor([1 << 40, -5, 64], dtype=I64, device=DEV)
    out = check_paged(BF16, [64, 64, 64], 4, 2, 32, 16, lens=lens, pools=pools)
    assert bool((out[1] == 0).all())


def test_paged_bad_pages():
    """Tokens of pages outside the cache are not seen; a sequence of nothing else gives zeros; one page may serve twice."""
    kp, vp, table = pool(F32, [700, 300, 90], 2, 64, 16, wide=3)
    pages = kp.shape[0]
    table[0, 3], table[0, 40], table[0, 41] = pages, -7, 2 ** 31 - 1
    table[2, :] = -1
    table[1, 5] = table[1, 6] = table[0, 0]
    out = check_paged(F32, [700, 300, 90], 4, 2, 64, 16, pools=(kp, vp, table))
    assert bool((out[2] == 0).all())


def test_paged_table_out_of_a_wider_one():
    kp, vp, table = pool(BF16, [100, 40], 2, 64, 16)
    wide = torch.full((2, 50), 2 ** 30, dtype=I32, device=DEV)
    wide[:, 9:9 + table.shape[1]] = table
    check_paged(BF16, [100, 40], 4, 2, 64, 16, pools=(kp, vp, wide[:, 9:9 + table.shape[1]]))


def test_paged_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 elements and 2^32 bytes of the cache."""
    kv, dim, page = 8, 128, 16
    pages = (1 << 33) // (page * kv * dim * 2) + 40
    kp, vp = (torch.zeros(pages, page, kv, dim, dtype=BF16, device=DEV) for _ in range(2))
    table = (pages - 1 - torch.arange(40, device=DEV)).to(I32)[None].contiguous()
    table[0, 1] = pages // 2 + 3
    for p, s in ((kp, 1), (vp, 2)):
        p[table[0].long()] = rand(40, page, kv, dim, seed=s, dt=BF16)
    check_paged(BF16, [633], 16, 8, 128, 16, pools=(kp, vp, table))


def test_paged_huge_scores():
    for dt, size in ((F32, 1e15), (BF16, 1e9), (F16, 200.0)):
        n = 1500
        kp, vp, table = pool(dt, [n], 1, 32, 16)
        j = torch.arange(n, device=DEV)
        slot = table[0].long()[j // 16] * 16 + j % 16
        kp.view(-1, 32)[slot] = 0
        kp.view(-1, 32)[slot, 0] = (j % 50 - 25).to(dt)
        q = torch.zeros(1, 32, dtype=dt, device=DEV)
        q[0, 0] = size
        out = torch.empty_like(q)
        tte.tt_emb_attend_paged(q, kp, vp, table, torch.tensor([n], device=DEV), out, scale=float(size))
        want = vp.view(-1, 32)[slot][j % 50 == 49].double().mean(0)[None]
        check(out, want, 4 * ref.U[dt] * torch.full_like(want, 5.0), f"paged huge {dt}")


def test_paged_one_bad_head_stays_apart():
    """NaN in one key head's cache or query reaches only the heads that read it."""
    kp, vp, table = pool(BF16, [400, 90], 2, 64, 16)
    lens = torch.tensor([400, 90], device=DEV)
    q = rand(2, 256, seed=3, dt=BF16)
    good, bad = torch.empty_like(q), torch.empty_like(q)
    tte.tt_emb_attend_paged(q, kp, vp, table, lens, good)
    vp[table[0, 3].long(), 5, 1] = NAN
    q2 = q.clone()
    q2[1, :64] = NAN
    tte.tt_emb_attend_paged(q2, kp, vp, table, lens, bad)
    assert torch.equal(bad[0, :128], good[0, :128]) and bool(bad[0, 128:].isnan().all())
    assert torch.equal(bad[1, 64:], good[1, 64:]) and bool(bad[1, :64].isnan().all())


# ------------------------------------------------- together, graphs, streams

@TYPES
def test_a_layer_prompts_then_tokens(dt):
    """As they are used: the rows of a prompt are projected, rotated and attended; its keys and values go into the cache, and
    new tokens one by one give what the whole prompt with them gives."""
    heads, kv, dim, page, width = 4, 2, 32, 8, 64
    lengths, more = [37, 5, 70], 3
    total = [n + more for n in lengths]
    rows = sum(total)
    x = rand(rows, width, seed=1)
    w = rand(width, (heads + 2 * kv) * dim, seed=2) / width ** 0.5
    qkv = (x @ w).to(dt)
    q, k, v = qkv[:, :heads * dim], qkv[:, heads * dim:(heads + kv) * dim], qkv[:, (heads + kv) * dim:]
    wq, wk, freq = 1 + 0.1 * rand(dim, seed=3), 1 + 0.1 * rand(dim, seed=4), freqs(dim // 2)
    starts = [sum(total[:i]) for i in range(3)]
    pos = torch.cat([torch.arange(n, device=DEV) for n in total])
    qr, kr = torch.empty(rows, heads * dim, dtype=dt, device=DEV), torch.empty(rows, kv * dim, dtype=dt, device=DEV)
    tte.tt_emb_rotate_forward(q, k, wq.to(dt), wk.to(dt), pos, freq, qr, kr)
    full = torch.empty_like(qr)
    tte.tt_emb_attend_forward(qr, kr, v, offsets_of(total), full, heads=heads, kv_heads=kv)
    most = (max(total) + page - 1) // page
    kp, vp = (torch.full((3 * most, page, kv, dim), NAN, dtype=dt, device=DEV) for _ in range(2))
    table = torch.randperm(3 * most, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(I32).view(3, most)

    def slot(s, p):
        return table[s].long()[p // page] * page + p % page

    prompt = torch.cat([torch.arange(a, a + n, device=DEV) for a, n in zip(starts, lengths)])
    slots = torch.cat([slot(s, torch.arange(n, device=DEV)) for s, n in enumerate(lengths)])
    qp = torch.empty(len(prompt), heads * dim, dtype=dt, device=DEV)
    tte.tt_emb_rotate_append(q[prompt], k[prompt], v[prompt], wq.to(dt), wk.to(dt), pos[prompt], freq, slots, qp, kp, vp)
    assert torch.equal(qp, qr[prompt])
    for t in range(more):
        at = torch.tensor([a + n + t for a, n in zip(starts, lengths)], device=DEV)
        lens = torch.tensor([n + t for n in lengths], device=DEV)
        slots = torch.cat([slot(s, lens[s:s + 1]) for s in range(3)])
        q1, out = torch.empty(3, heads * dim, dtype=dt, device=DEV), torch.empty(3, heads * dim, dtype=dt, device=DEV)
        tte.tt_emb_rotate_append(q[at], k[at], v[at], wq.to(dt), wk.to(dt), pos[at], freq, slots, q1, kp, vp)
        tte.tt_emb_attend_paged(q1, kp, vp, table, lens + 1, out)
        want, bound = ref.paged(q1, kp, vp, table, lens + 1, dim ** -0.5)
        check(out, want, bound, "token")
        check(out, full[at].double(), 2 * bound, "token beside the prompt")   # each within its bound of the same


def test_captured_training_and_serving():
    """All calls in one graph, replayed on new inputs beside eager work: the eager results' bits."""
    dt, heads, kv, dim, rows = BF16, 8, 2, 64, 500
    q, k, v = (t.contiguous() for t in packed(dt, rows, heads, kv, dim))
    d = rand(rows, heads * dim, seed=3, dt=dt)
    off, pos, freq = offsets_of([123, 0, 300, 77]), torch.arange(rows, device=DEV), freqs(dim // 2)
    w = 1 + 0.1 * rand(dim, seed=4)
    kp, vp, table = pool(dt, [900, 40], kv, dim, 16)
    lens, slots = torch.tensor([900, 40], device=DEV), torch.arange(2, device=DEV) + 5
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (
        tte.tt_emb_rotate_workspace_bytes(dt, rows, heads, kv, dim), tte.tt_emb_attend_workspace_bytes(dt, rows, heads, kv, dim),
        tte.tt_emb_attend_paged_workspace_bytes(dt, 2, heads, kv, dim))]
    like = lambda *ts: [torch.zeros_like(t) for t in ts]   # noqa: E731
    out = dict(zip(("qr", "kr", "o", "dqr", "dkr", "dv", "dq", "dk", "dwq", "dwk"), like(q, k, q, q, k, v, q, k, w, w)))
    out["lse"], out["q1"], out["o1"] = torch.zeros(heads, rows, device=DEV), *like(q[:2], q[:2])
    how = dict(heads=heads, kv_heads=kv)

    def step(o):
        tte.tt_emb_rotate_forward(q, k, w, w, pos, freq, o["qr"], o["kr"])
        tte.tt_emb_attend_forward(o["qr"], o["kr"], v, off, o["o"], o["lse"], **how)
        tte.tt_emb_attend_backward(o["qr"], o["kr"], v, off, o["o"], o["lse"], d, o["dqr"], o["dkr"], o["dv"], workspace=ws[1],
                                   **how)
        tte.tt_emb_rotate_backward(q, k, w, w, pos, freq, o["dqr"], o["dkr"], o["dq"], o["dk"], o["dwq"], o["dwk"],
                                   workspace=ws[0])
        tte.tt_emb_rotate_append(q[:2], k[:2], v[:2], w, w, pos[:2], freq, slots, o["q1"], kp, vp)
        tte.tt_emb_attend_paged(o["q1"], kp, vp, table, lens, o["o1"], workspace=ws[2])

    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for i in range(3):
        for t, s in ((q, 30), (k, 40), (v, 50), (d, 60)):
            t.copy_(rand(*t.shape, seed=s + i, dt=dt))
        off.copy_(offsets_of([[123, 0, 300, 77], [0, 500, 0, 0], [250, 1, 2, 240]][i]))
        graph.replay()
        got = {n: t.clone() for n, t in out.items()}
        torch.cuda.synchronize()
        eager = {n: torch.zeros_like(t) for n, t in out.items()}
        for n in ("o", "dqr", "dkr", "dv", "lse"):     # rows of no sequence stay
            eager[n].copy_(out[n])
        step(eager)
        for n in out:
            assert torch.equal(got[n], eager[n]), (i, n)


def test_calls_on_another_stream():
    q, k, v = packed(F16, 300, 4, 4, 64)
    off = offsets_of([200, 100])
    a, b = torch.empty(300, 256, dtype=F16, device=DEV), torch.empty(300, 256, dtype=F16, device=DEV)
    kp, vp, table = pool(F16, [3000], 4, 64, 16)
    lens = torch.tensor([3000], device=DEV)
    c, e = torch.empty(1, 256, dtype=F16, device=DEV), torch.empty(1, 256, dtype=F16, device=DEV)
    tte.tt_emb_attend_forward(q, k, v, off, a, heads=4, kv_heads=4)
    tte.tt_emb_attend_paged(q[:1], kp, vp, table, lens, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    tte.tt_emb_attend_forward(q, k, v, off, b, heads=4, kv_heads=4, stream=s)
    tte.tt_emb_attend_paged(q[:1], kp, vp, table, lens, e, stream=s)
    s.synchronize()
    assert torch.equal(a, b) and torch.equal(c, e)


@pytest.mark.parametrize("most,fewer", [(64, (63, 9, 1)), (3, (2, 1)), (700, (300, 20))])
def test_paged_in_a_larger_batchs_workspace(most, fewer):
    heads, kv, dim = 8, 2, 32
    size = tte.tt_emb_attend_paged_workspace_bytes(BF16, most, heads, kv, dim)
    room = torch.full((size + 4096,), 77, dtype=torch.uint8, device=DEV)
    lengths = [(i * 617) % 3000 for i in range(most)]
    kp, vp, table = pool(BF16, lengths, kv, dim, 16)
    lens, q = torch.tensor(lengths, device=DEV), rand(most, heads * dim, seed=1, dt=BF16)
    for n in (most, *fewer):
        outs = [torch.empty(n, heads * dim, dtype=BF16, device=DEV) for _ in range(2)]
        for o, ws in zip(outs, (room[:size], None)):
            tte.tt_emb_attend_paged(q[:n], kp, vp, table[:n], lens[:n], o, workspace=ws)
        assert torch.equal(*outs) and bool((room[size:] == 77).all())

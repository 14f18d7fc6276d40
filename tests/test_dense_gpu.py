"""The dense operators' kernels against their 64-bit definitions, at the sizes,
strides, types and values where they can go wrong. The bounds are those of
tests/dense_ref.py, which count roundings."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import tensor_train_compressed_amd as tte  # noqa: E402
from tests import dense_ref as ref  # noqa: E402
from tests.gpu_helpers import DEV, say  # noqa: E402

F32, BF16, F16 = ref.F32, ref.BF16, ref.F16
NAN, INF = math.nan, math.inf
TYPES = pytest.mark.parametrize("dt", [F32, BF16, F16], ids=["f32", "bf16", "f16"])


def rand(*shape, seed, dt=F32):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(dt)


def padded(t, pad, off=0):
    """The same matrix with rows `pad` elements further apart, `off` into the buffer; the rest is NaN."""
    wide = torch.full((t.shape[0] * (t.shape[1] + pad) + off,), NAN, dtype=t.dtype, device=t.device)
    v = wide[off:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v


def hole(rows, cols, dt, pad=0, off=0):
    """An output matrix and the buffer around it, filled with a mark."""
    wide = torch.full((rows * (cols + pad) + off + 3,), 77.0, dtype=dt, device=DEV)
    return wide[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols], wide


def untouched(view, wide):
    """Nothing outside the view was written."""
    got = view.clone()
    view.fill_(77.0)
    assert bool((wide == 77.0).all()), "written outside the output"
    view.copy_(got)


# ---------------------------------------------------------------- layer norm

def run_norm(x, w, b, dy, eps=1e-5, pad=0, off=0):
    m, n = x.shape
    xs, dys = padded(x, pad, off), padded(dy, pad, off)
    y, ywide = hole(m, n, x.dtype, pad, off)
    dx, dxwide = hole(m, n, x.dtype, pad, off)
    mean, rstd = torch.full((m,), NAN, device=DEV), torch.full((m,), NAN, device=DEV)
    dw = torch.full_like(w, NAN)
    db = None if b is None else torch.full_like(w, NAN)
    ws = torch.full((tte.tt_emb_norm_workspace_bytes(x.dtype, m, n),), 255, dtype=torch.uint8, device=DEV)
    tte.tt_emb_norm_forward(xs, w, b, y, mean, rstd, eps=eps)
    tte.tt_emb_norm_backward(xs, w, mean, rstd, dys, dx, dw, db, workspace=ws)
    if m:
        untouched(y, ywide)
        untouched(dx, dxwide)
    return y, dx, dw, db


def check_norm(x, w, b, dy, eps=1e-5, pad=0, off=0, what="norm"):
    say(what, list(x.shape), x.dtype, w.dtype, "pad", pad, "off", off)
    y, dx, dw, db = run_norm(x, w, b, dy, eps, pad, off)
    wy = ref.norm(x, w, b, eps)[0]
    wx, ww, wb = ref.norm_grads(x, w, dy, eps)
    by, bx, bw, bb = ref.norm_bounds(x, w, b, dy, eps, w.dtype)
    ref.check(y, wy, by, f"{what} y")
    ref.check(dx, wx, bx, f"{what} dx")
    ref.check(dw, ww, bw, f"{what} dweight")
    if b is not None:
        ref.check(db, wb, bb, f"{what} dbias")
    return y, dx, dw, db


@TYPES
@pytest.mark.parametrize("rows,dim,pad,off", [
    (1, 1, 0, 0), (3, 7, 1, 1), (5, 16, 0, 0), (300, 128, 0, 0), (17, 129, 3, 0), (65, 512, 8, 0), (9, 513, 0, 1),
    (40, 1021, 11, 0), (33, 1024, 0, 0), (5, 1025, 2, 1), (1, 2048, 0, 0), (7, 2050, 6, 0), (530, 4096, 0, 0),
    (3, 4099, 1, 3), (2, 8192, 0, 0), (3, 8200, 24, 0), (260, 16384, 0, 0), (2, 16383, 1, 1)])
def test_norm_sizes(dt, rows, dim, pad, off):
    x = rand(rows, dim, seed=1) * torch.exp(0.5 * rand(rows, 1, seed=2)) + rand(rows, 1, seed=3)
    w, b = 1 + 0.1 * rand(dim, seed=4), 0.1 * rand(dim, seed=5)
    dy = rand(rows, dim, seed=6, dt=dt)
    check_norm(x.to(dt), w.to(dt), b.to(dt), dy, pad=pad, off=off)


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("dim", [100, 770, 3000])
def test_norm_fp32_weights_no_bias(dt, dim):
    w = 1 + 0.1 * rand(dim, seed=4)
    check_norm(rand(70, dim, seed=1, dt=dt), w, None, rand(70, dim, seed=2, dt=dt))


@TYPES
@pytest.mark.parametrize("rows,dim", [(127, 100), (129, 100), (32, 900), (33, 900), (4, 4000), (5, 4000), (2, 16000)])
def test_norm_around_one_workgroup(dt, rows, dim):
    """Batches that one workgroup takes, and the next larger ones."""
    w = 1 + 0.1 * rand(dim, seed=4)
    b = rand(dim, seed=5)
    check_norm(rand(rows, dim, seed=1, dt=dt), w.to(dt), b.to(dt), rand(rows, dim, seed=2, dt=dt))


def test_norm_many_rows():
    """More rows than one pass of the workgroups takes."""
    x, dy = rand(40000, 128, seed=1), rand(40000, 128, seed=2)
    check_norm(x, rand(128, seed=3), rand(128, seed=4), dy)
    check_norm(rand(9000, 600, seed=1, dt=BF16), rand(600, seed=3), rand(600, seed=4), rand(9000, 600, seed=2, dt=BF16))


def test_norm_offset_and_constant_rows():
    x = rand(6, 300, seed=1)
    x[0] += 1e4        # a large offset: the centred values carry the digits
    x[1] = 3.0         # constant: y = bias, dx = rstd-scaled by 1/sqrt(eps)
    x[2] *= 1e-6
    check_norm(x, rand(300, seed=2), rand(300, seed=3), rand(6, 300, seed=4))


def test_norm_far_rows():
    """Rows far from zero beside their spread: the statistics are good to the rounding of the inputs' own sums."""
    x = (rand(40, 3000, seed=1) + 3e4 * rand(40, 1, seed=2)).to(F32)
    y, mean, rstd = torch.empty_like(x), torch.empty(40, device=DEV), torch.empty(40, device=DEV)
    w, b = torch.ones(3000, device=DEV), torch.zeros(3000, device=DEV)
    tte.tt_emb_norm_forward(x, w, b, y, mean, rstd)
    wy, wm, wr, _ = ref.norm(x, w, b, 1e-5)
    # x - mean: the first mean is off by a few roundings of it, the second sum takes that off again,
    # each difference is off by half a step of itself
    assert float((mean.double() - wm[:, 0]).abs().max() / wm.abs().max()) <= 2 * ref.U32
    assert float((rstd.double() / wr[:, 0] - 1).abs().max()) <= ref.LEVELS * ref.U32
    assert float((y.double() - wy).abs().max()) <= ref.LEVELS * ref.U32 * float(wy.abs().max())


def test_norm_bad_rows_stay_apart():
    """A row with NaN or an infinity makes that row NaN and no other."""
    x, w, b, dy = rand(5, 200, seed=1), rand(200, seed=2), rand(200, seed=3), rand(5, 200, seed=4)
    good = run_norm(x, w, b, dy)
    x2 = x.clone()
    x2[1, 7], x2[3, 199] = NAN, INF
    y, dx, dw, db = run_norm(x2, w, b, dy)
    for r in (0, 2, 4):
        assert torch.equal(y[r], good[0][r]) and torch.equal(dx[r], good[1][r])
    for r in (1, 3):
        assert bool(torch.isnan(y[r]).all()) and bool(torch.isnan(dx[r]).all())
    assert torch.equal(db, good[3])


def test_norm_empty():
    x = torch.empty(0, 64, device=DEV)
    _, _, dw, db = run_norm(x, rand(64, seed=1), rand(64, seed=2), x)
    assert not dw.any() and not db.any()


# ------------------------------------------------------- gated feed-forward

def run_gate(x, wg, wu, dout, kind, pad=0, off=0):
    m, h = x.shape[0], wg.shape[0]
    xs = padded(x, pad, off)
    out, owide = hole(m, h, x.dtype, pad, off)
    need = tte.tt_emb_gate_workspace_bytes(x.dtype, m, x.shape[1], h)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    if dout is None:
        tte.tt_emb_gate_forward(xs, wg, wu, out, act=kind, workspace=ws)
        untouched(out, owide)
        return (out,)
    g, u = torch.full((m, h), NAN, device=DEV), torch.full((m, h), NAN, device=DEV)
    dx, dxwide = hole(m, x.shape[1], x.dtype, pad, off)
    dwg, dwu = torch.full_like(wg, NAN), torch.full_like(wu, NAN)
    tte.tt_emb_gate_forward(xs, wg, wu, out, g, u, act=kind, workspace=ws)
    ws.fill_(255)
    tte.tt_emb_gate_backward(xs, wg, wu, g, u, padded(dout, pad, off), dx, dwg, dwu, act=kind, workspace=ws)
    if m:
        untouched(out, owide)
        untouched(dx, dxwide)
    return out, g, u, dx, dwg, dwu


GATE_NAMES = ("out", "gate", "up", "dx", "dw_gate", "dw_up")


def check_gate(x, wg, wu, dout, kind, pad=0, off=0):
    say("gate", list(x.shape), wg.shape[0], x.dtype, kind, "pad", pad, "off", off, "train", dout is not None)
    got = run_gate(x, wg, wu, dout, kind, pad, off)
    want = ref.gate(x, wg, wu, kind)
    bounds = ref.gate_bounds(x, wg, wu, dout, kind)
    if dout is not None:
        want = (*want, *ref.gate_grads(x, wg, wu, dout, kind))
    t = x.dtype
    for a, b, c, name in zip(got, want, bounds, GATE_NAMES):
        ref.check(a, b, c, f"gate {name}")
        # the errors of the terms are independent: over an output they are off by no more than
        # one rounding of the result and one of a factor (fp32: 2^-24 of each partial sum)
        size = b.numel()
        if size > 1000:
            slack = 2 * ref.U[t] if t != F32 and name not in ("gate", "up") else 2.0 ** -20
            assert ref.rel(a, b) <= slack, (name, ref.rel(a, b))
    return got


def gate_inputs(m, k, h, dt, train=True):
    x, wg, wu = rand(m, k, seed=1, dt=dt), rand(h, k, seed=2) / k ** 0.5, rand(h, k, seed=3) / k ** 0.5
    return x, wg.to(dt), wu.to(dt), rand(m, h, seed=4, dt=dt) if train else None


GATE_SIZES = [(1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (2, 200, 72, 0, 0), (3, 7, 5, 1, 1), (5, 65, 129, 3, 0),
              (8, 512, 256, 0, 0), (15, 130, 66, 0, 1), (16, 1000, 1001, 8, 0), (17, 96, 1000, 0, 0),
              (33, 1031, 67, 1, 0), (64, 128, 512, 0, 0), (65, 256, 192, 0, 0), (100, 320, 1536, 8, 0),
              (129, 64, 300, 24, 0), (257, 520, 264, 0, 0), (300, 1030, 701, 3, 0), (513, 136, 1100, 0, 0),
              (1000, 1024, 640, 0, 0)]


@TYPES
@pytest.mark.parametrize("m,k,h,pad,off", GATE_SIZES)
def test_gate_sizes(dt, m, k, h, pad, off):
    kind = ("silu", "gelu", "relu")[(m + k + h) % 3]
    check_gate(*gate_inputs(m, k, h, dt), kind, pad, off)
    check_gate(*gate_inputs(m, k, h, dt, train=False), kind, pad, off)


@TYPES
@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_gate_activations(dt, kind):
    """Projections over the activations' whole range, zero among them."""
    x, wg, wu, d = gate_inputs(130, 72, 96, dt)
    x[0] = 0
    check_gate(x, (3 * wg.float()).to(dt), wu, d, kind)


@TYPES
def test_gate_larger(dt):
    check_gate(*gate_inputs(2100, 512, 1300, dt), "silu")


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("m,k,h", [(4200, 4104, 2100), (4100, 2056, 4200)])
def test_gate_large_tiles(dt, m, k, h):
    """Sizes that fill the chip with the largest tiles, none a multiple of them; the same bits again."""
    ins = gate_inputs(m, k, h, dt)
    for a, b in zip(check_gate(*ins, "silu"), run_gate(*ins, "silu")):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("m,k,h", [(4000, 520, 2000), (500, 264, 9000), (3000, 1032, 1100), (8200, 264, 300)])
def test_gate_tiles_of_each_size(dt, m, k, h):
    """Rows and columns for one round of the largest tiles, for the middle ones, and few rows beside many columns."""
    ins = gate_inputs(m, k, h, dt)
    for a, b in zip(check_gate(*ins, "silu"), run_gate(*ins, "silu")):
        assert torch.equal(a, b)


def test_gate_fp32_range():
    """fp32 operands keep their range: products of very large and very small values."""
    x, wg, wu, d = gate_inputs(70, 128, 64, F32)
    big = torch.where(torch.arange(70, device=DEV)[:, None] % 2 == 0, 1e18, 1e-18)
    got = run_gate(x * big, wg * 1e-3, wu * 1e3, d, "relu")
    want = ref.gate(x * big, wg * 1e-3, wu * 1e3, "relu")
    for a, b in zip(got[1:3], want[1:3]):
        for rows in (slice(0, None, 2), slice(1, None, 2)):
            assert ref.rel(a[rows], b[rows]) < 2.0 ** -20
    top = torch.full((2, 64), 3.4e38, device=DEV)    # rounding this to 8 digits would make it infinite
    wg = torch.zeros(64, 64, device=DEV)
    wg[:, 0] = 0.5
    got = run_gate(top, wg, wg, None, "relu")
    assert bool(torch.isinf(got[0]).all())           # 1.7e38 squared
    g, u = torch.empty(2, 64, device=DEV), torch.empty(2, 64, device=DEV)
    tte.tt_emb_gate_forward(top, wg, wg, torch.empty(2, 64, device=DEV), g, u, act="relu")
    assert float((g.double() / 1.7e38 - 1).abs().max()) < 2e-6


def test_gate_bad_rows_stay_apart():
    x, wg, wu, _ = gate_inputs(40, 100, 90, BF16, train=False)
    good = run_gate(x, wg, wu, None, "silu")[0]
    x2 = x.clone()
    x2[3, 5], x2[39, 0] = NAN, INF
    out = run_gate(x2, wg, wu, None, "silu")[0]
    keep = [r for r in range(40) if r not in (3, 39)]
    assert torch.equal(out[keep], good[keep])
    assert bool(torch.isnan(out[3]).all()) and not bool(torch.isfinite(out[39]).any())


@TYPES
def test_gate_empty(dt):
    x, wg, wu, d = gate_inputs(0, 70, 90, dt)
    got = run_gate(x, wg, wu, d, "gelu")
    assert not got[4].any() and not got[5].any()


# ---------------------------------------------------------------- distillation

def run_distill(z, ids, tl, w, t, pad=0, off=0):
    """loss, dlogits of the two calls, checked to be the bits of the one call."""
    m, v = z.shape
    zs = padded(z, pad, off)
    need = tte.tt_emb_distill_workspace_bytes(z.dtype, m, v)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    loss, only = torch.full((m,), NAN, device=DEV), torch.full((m,), NAN, device=DEV)
    stats = torch.full((m, 2), NAN, device=DEV)
    dz, wide = hole(m, v, z.dtype, pad, off)
    dz2, wide2 = hole(m, v, z.dtype, pad, off)
    tte.tt_emb_distill_forward(zs, ids, tl, only, temperature=t, workspace=ws)
    ws.fill_(255)
    tte.tt_emb_distill_forward(zs, ids, tl, loss, stats, temperature=t, workspace=ws)
    tte.tt_emb_distill_backward(zs, ids, tl, stats, w, dz, temperature=t)
    untouched(dz, wide)
    loss2 = torch.full((m,), NAN, device=DEV)
    ws.fill_(255)
    tte.tt_emb_distill_train(zs, ids, tl, w, loss2, dz2, temperature=t, workspace=ws)
    untouched(dz2, wide2)
    return (loss, dz), (loss2, dz2), only


def check_distill(z, ids, tl, w, t, pad=0, off=0):
    say("distill", list(z.shape), z.dtype, "top", ids.shape[1], "t", t, "pad", pad, "off", off)
    split, train, only = run_distill(z, ids, tl, w, t, pad, off)
    wl, wg, bl, bg = ref.distill(z, ids, tl, t)
    wg, bg = wg * w.double()[:, None], bg * w.double().abs()[:, None]
    for (loss, dz), how in ((split, "split"), (train, "train")):
        ref.check(loss, wl, bl, f"distill loss {how}")
        ref.check(dz, wg, bg + ref.rounded(z.dtype, wg), f"distill dlogits {how}")
    ref.check(only, wl, bl, "distill loss alone")
    return train


def teacher(m, v, top, seed, holes=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(v, generator=g)[:top] for _ in range(m)]) if top <= v else \
        torch.randint(0, v, (m, top), generator=g)
    tl = 3 * torch.randn(m, top, generator=g)
    if holes and top:
        ids[torch.rand(m, top, generator=g) < 0.2] = -1
        ids[::7] = -1           # empty lists
        tl[torch.rand(m, top, generator=g) < 0.05] = -INF
    w = torch.rand(m, generator=g)
    w[::5] = 0
    return ids.to(DEV), tl.to(DEV), w.to(DEV)


@TYPES
@pytest.mark.parametrize("m,v,top,pad,off", [
    (1, 1, 1, 0, 0), (1, 2, 3, 0, 1), (7, 1000, 5, 0, 0), (30, 1001, 1, 1, 0), (3, 5, 8, 3, 1), (5, 2048, 256, 8, 0),
    (9, 16384, 64, 0, 0), (9, 16385, 64, 0, 0), (4, 50021, 20, 5, 0), (3, 32768, 1024, 0, 1), (2, 131072, 300, 0, 0),
    (2, 300001, 100, 24, 0), (600, 1500, 20, 0, 0), (6, 8191, 10, 0, 0), (6, 65536, 10, 0, 0)])
def test_distill_sizes(dt, m, v, top, pad, off):
    ids, tl, w = teacher(m, v, top, seed=m + v)
    t = (1.0, 1.5, 2.0, 4.0)[(m + top) % 4]
    check_distill((2 * rand(m, v, seed=1)).to(dt), ids, tl, w, t, pad, off)


def test_distill_more_rows_than_one_launch_takes():
    """2^23 workgroups go in one launch."""
    m = (1 << 23) + 1001
    z = rand(m, 2, seed=1, dt=F16)
    ids = torch.randint(-1, 3, (m, 1), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    check_distill(z, ids, rand(m, 1, seed=3), rand(m, seed=4), 2.0)


def test_distill_no_list():
    z = rand(3, 100, seed=1)
    ids, tl, w = teacher(3, 100, 0, seed=1)
    loss, dz = check_distill(z, ids, tl, w + 1, 1.0)
    assert not loss.any() and not dz.any()


def test_distill_repeated_and_foreign_classes():
    z = rand(4, 500, seed=1)
    ids = torch.tensor([[5, 5, 5, 9], [499, 0, 499, 0], [500, -7, 1 << 40, 3], [1, 2, 3, 4]], device=DEV)
    check_distill(z, ids, rand(4, 4, seed=2), torch.ones(4, device=DEV), 2.0)


@TYPES
def test_distill_far_logits(dt):
    """One class far above the rest, and rows whose logits all lie far from zero."""
    z = rand(4, 3000, seed=1)
    z[0, 17] = 80.0
    z[1] -= 200.0
    z[2] += 1000.0
    ids, tl, w = teacher(4, 3000, 30, seed=3, holes=False)
    check_distill(z.to(dt), ids, tl * 4, w + 0.5, 1.0)


@pytest.mark.parametrize("v", [300, 40000])
def test_distill_masked_classes(v):
    """Student classes at -inf, whole chunks of them, the type's lowest value, and rows with nothing left."""
    z = rand(6, v, seed=1)
    ids, tl, w = teacher(6, v, 4, seed=3, holes=False)
    w = torch.ones_like(w)
    z[0, 100:] = -INF
    ids[0] = torch.tensor([1, 2, 3, 4])            # the list lies in what is left
    z[1, 50] = torch.finfo(F32).min
    ids[1] = torch.tensor([0, 1, 2, 3])
    z[2, :v - 100] = -INF
    ids[2] = torch.tensor([v - 1, v - 2, v - 3, v - 4])
    z[5], ids[5] = -INF, -1                        # nothing left, and an empty list: 0
    loss, dz = check_distill(z, ids, tl, w, 1.0)[:2]
    assert not dz[0, 100:].any() and not dz[5].any() and float(loss[5]) == 0.0
    # a listed class that the student masks: the loss is infinite, the gradient is not
    z[3, 7] = -INF
    ids[3] = torch.tensor([7, 8, 9, 10])
    z[4] = -INF                                    # nothing left, but a list: undefined
    ids[4] = torch.tensor([0, 1, 2, 3])
    split, train, only = run_distill(z, ids, tl, w, 1.0)
    for loss, dz in (split, train):
        assert float(loss[3]) == INF and bool(torch.isfinite(dz[3]).all())
        assert math.isnan(float(loss[4])) and bool(torch.isnan(dz[4]).all())
        assert bool(torch.isfinite(loss[[0, 1, 2, 5]]).all()) and bool(torch.isfinite(dz[[0, 1, 2, 5]]).all())


@TYPES
@pytest.mark.parametrize("v", [300, 40000])
def test_distill_lowest_values(dt, v):
    """Rows masked with the type's lowest value as a whole, but for one class, and in part: like any logits."""
    low = torch.finfo(dt).min
    z = rand(4, v, seed=1)
    z[0] = low
    z[1], z[1, 5] = low, 1.0
    z[2, v // 2:] = low
    z[3], z[3, 7] = low, -low                      # the type's largest
    ids = torch.tensor([[0, 1, v - 1, 9], [5, 5, 5, 5], [0, 1, 2, 3], [7, 7, 7, 7]], device=DEV)
    check_distill(z.to(dt), ids, rand(4, 4, seed=2), torch.ones(4, device=DEV), 1.0)


def test_distill_nan_rows_stay_apart():
    z = rand(4, 40000, seed=1)
    ids, tl, w = teacher(4, 40000, 9, seed=3, holes=False)
    w = w + 1
    good = run_distill(z, ids, tl, w, 1.0)[1]
    z2 = z.clone()
    z2[1, 39999], z2[2, 3] = NAN, INF
    loss, dz = run_distill(z2, ids, tl, w, 1.0)[1]
    for r in (0, 3):
        assert torch.equal(dz[r], good[1][r]) and torch.equal(loss[r], good[0][r])
    for r in (1, 2):
        assert math.isnan(float(loss[r])) and bool(torch.isnan(dz[r]).all())


def test_distill_gradient_against_differences():
    """The kernel's gradient against differences of the 64-bit loss."""
    z = rand(2, 40, seed=1)
    ids, tl, w = teacher(2, 40, 6, seed=3, holes=False)
    _, dz = run_distill(z, ids, tl, torch.ones_like(w), 1.5)[1]
    h = 1e-5
    for j in range(0, 40, 3):
        a, b = z.double(), z.double()
        a[:, j] += h
        b[:, j] -= h
        d = (ref.distill(a, ids, tl, 1.5)[0] - ref.distill(b, ids, tl, 1.5)[0]) / (2 * h)
        # differences: h^2 and 1e-16/h; the kernel: fp32 roundings of values up to about 1
        assert float((dz[:, j].double() - d).abs().max()) < 1e-7 + 100 * ref.U32


# ------------------------------------------------------------- together

def operators_once(seed):
    """Every operator once on fresh inputs: (inputs, a call, outputs)."""
    x, w, b, dy = rand(300, 256, seed=seed, dt=BF16), rand(256, seed=seed + 1), rand(256, seed=seed + 2), \
        rand(300, 256, seed=seed + 3, dt=BF16)
    y, dx, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(300, device=DEV), \
        torch.empty(300, device=DEV)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    xs, wg, wu, d = gate_inputs(200, 192, 320, BF16)
    xs = xs + seed
    xf, wgf, wuf, df = (v.float() for v in (xs, wg, wu, d))
    gate = [[torch.empty(200, 320, dtype=t.dtype, device=DEV), torch.empty(200, 320, device=DEV),
             torch.empty(200, 320, device=DEV), torch.empty_like(t), torch.empty(320, 192, dtype=t.dtype, device=DEV),
             torch.empty(320, 192, dtype=t.dtype, device=DEV)] for t in (xs, xf)]
    z = rand(20, 40000, seed=seed + 5, dt=F16)
    ids, tl, rw = teacher(20, 40000, 30, seed=seed)
    loss, dz = torch.empty(20, device=DEV), torch.empty_like(z)
    loss2, dz2, stats = torch.empty(20, device=DEV), torch.empty_like(z), torch.empty(20, 2, device=DEV)
    ws = [torch.empty(tte.tt_emb_norm_workspace_bytes(BF16, 300, 256), dtype=torch.uint8, device=DEV),
          torch.empty(max(tte.tt_emb_gate_workspace_bytes(t, 200, 192, 320) for t in (BF16, F32)), dtype=torch.uint8,
                      device=DEV),
          torch.empty(tte.tt_emb_distill_workspace_bytes(F16, 20, 40000), dtype=torch.uint8, device=DEV)]

    def call(stream=None):
        k = dict(stream=stream)
        tte.tt_emb_norm_forward(x, w, b, y, mean, rstd, **k)
        tte.tt_emb_norm_backward(x, w, mean, rstd, dy, dx, dw, db, workspace=ws[0], **k)
        for (o, g, u, gx, g1, g2), (a, p, q, e) in zip(gate, ((xs, wg, wu, d), (xf, wgf, wuf, df))):
            tte.tt_emb_gate_forward(a, p, q, o, g, u, workspace=ws[1], **k)
            tte.tt_emb_gate_backward(a, p, q, g, u, e, gx, g1, g2, workspace=ws[1], **k)
        tte.tt_emb_distill_train(z, ids, tl, rw, loss, dz, temperature=2.0, workspace=ws[2], **k)
        tte.tt_emb_distill_forward(z, ids, tl, loss2, stats, temperature=2.0, workspace=ws[2], **k)
        tte.tt_emb_distill_backward(z, ids, tl, stats, rw, dz2, temperature=2.0, **k)

    outs = [y, dx, mean, rstd, dw, db, *gate[0], *gate[1], loss, dz, loss2, dz2, stats]
    return [x, dy, xs, xf, z], call, outs


def far(t, stride):
    """The same rows `stride` elements apart."""
    v = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device=DEV).as_strided(t.shape, (stride, 1))
    return v.copy_(t)


def test_offsets_past_32_bits():
    """Rows whose elements lie more than 2^31 elements (2^32 bytes) into their buffers: the bits of near rows."""
    x, dy, w = rand(3, 200, seed=1, dt=BF16), rand(3, 200, seed=2, dt=BF16), rand(200, seed=3)
    got = [far(torch.empty_like(x), 1 << 30) for _ in range(2)]
    want = [torch.empty_like(x) for _ in range(2)]
    for (y, dx), (a, b) in ((got, (far(x, 1 << 30), far(dy, 1 << 30))), (want, (x, dy))):
        mean, rstd = torch.empty(3, device=DEV), torch.empty(3, device=DEV)
        tte.tt_emb_norm_forward(a, w, None, y, mean, rstd)
        tte.tt_emb_norm_backward(a, w, mean, rstd, b, dx, torch.empty_like(w))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    z = rand(3, 20000, seed=4, dt=F16)
    ids, tl, rw = teacher(3, 20000, 30, seed=5)
    loss = [torch.empty(3, device=DEV) for _ in range(2)]
    dz, dz2 = far(torch.empty_like(z), 1 << 30), torch.empty_like(z)
    tte.tt_emb_distill_train(far(z, 1 << 30), ids, tl, rw, loss[0], dz, temperature=2.0)
    tte.tt_emb_distill_train(z, ids, tl, rw, loss[1], dz2, temperature=2.0)
    assert torch.equal(*loss) and torch.equal(dz, dz2)
    del got, dz
    x, wg, wu, d = gate_inputs(1100, 72, 96, BF16)
    outs = []
    for a, b in ((far(x, 1 << 21), far(d, 1 << 21)), (x, d)):
        new = (lambda t: far(torch.empty_like(t), 1 << 21)) if a is not x else torch.empty_like
        out, dx, g, u = new(d), new(x), torch.empty(1100, 96, device=DEV), torch.empty(1100, 96, device=DEV)
        dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
        tte.tt_emb_gate_forward(a, wg, wu, out, g, u)
        tte.tt_emb_gate_backward(a, wg, wu, g, u, b, dx, dwg, dwu)
        outs.append((out, g, u, dx, dwg, dwu))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_same_bits_on_every_run():
    _, call, outs = operators_once(10)
    call()
    first = [o.clone() for o in outs]
    for _ in range(3):
        for o in outs:
            o.fill_(NAN)
        call()
        for a, b in zip(outs, first):
            assert torch.equal(a, b)


def test_other_stream_and_own_workspaces():
    """On a stream that is not the current one, with workspaces the calls allocate."""
    ins, call, outs = operators_once(20)
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.fill_(NAN)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    x, wg, wu, _ = gate_inputs(100, 100, 100, F16)
    a, b, c = (torch.full((100, 100), NAN, dtype=F16, device=DEV) for _ in range(3))
    side.wait_stream(torch.cuda.current_stream())
    tte.tt_emb_gate_forward(x, wg, wu, a)
    tte.tt_emb_gate_forward(x, wg, wu, b, stream=side)
    tte.tt_emb_gate_forward(x, wg, wu, c, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_graph_replays():
    """Captured once, replayed on new inputs with eager work between: each replay is the eager result."""
    ins, call, outs = operators_once(30)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        for i, t in enumerate(ins):
            t.copy_(rand(*t.shape, seed=100 * k + i, dt=t.dtype))
        for o in outs:
            o.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.fill_(NAN)
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)

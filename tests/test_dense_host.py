"""Checks of the dense operators that need no GPU: refusals on the host before
any launch, workspace sizes, and the closed-form gradients of the 64-bit
definitions against differences."""
import ctypes

import pytest

import tensor_train_compressed_amd as tte

torch = pytest.importorskip("torch")
from tests import dense_ref as ref  # noqa: E402

P = ctypes.c_void_p
A = P(4096)     # an aligned address that no refused call may touch
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
F = ctypes.c_float


def test_norm_refusals():
    lib = tte.load_library()

    def fwd(dtype=0, wdtype=0, x=A, ldx=8, w=A, b=None, y=A, ldy=8, mean=None, rstd=None, rows=2, dim=8, eps=1e-5):
        return lib.tt_emb_norm_forward(dtype, wdtype, x, ldx, w, b, y, ldy, mean, rstd, rows, dim, F(eps), None)

    assert fwd(dtype=3) == INVALID and fwd(dtype=-1) == INVALID
    assert fwd(wdtype=1) == UNSUPPORTED            # fp32 rows with bf16 weights
    assert fwd(dtype=1, wdtype=2) == UNSUPPORTED
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID and fwd(w=None) == INVALID
    assert fwd(ldx=7) == INVALID and fwd(ldy=7) == INVALID
    assert fwd(mean=A) == INVALID and fwd(rstd=A) == INVALID      # both or neither
    assert fwd(rows=-1) == INVALID and fwd(dim=0) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(dim=16385, ldx=16385, ldy=16385) == UNSUPPORTED
    assert fwd(rows=1 << 31) == UNSUPPORTED
    assert fwd(rows=0, x=None, y=None) == 0

    def bwd(x=A, ldx=8, w=A, mean=A, rstd=A, dy=A, lddy=8, dx=A, lddx=8, dw=A, db=A, rows=2, dim=8, ws=A, n=1 << 20):
        return lib.tt_emb_norm_backward(0, 0, x, ldx, w, mean, rstd, dy, lddy, dx, lddx, dw, db, rows, dim, ws, n, None)

    for k in ("x", "w", "mean", "rstd", "dy", "dx", "dw", "ws"):
        assert bwd(**{k: None}) == INVALID, k
    for k in ("ldx", "lddy", "lddx"):
        assert bwd(**{k: 7}) == INVALID, k
    assert bwd(ws=P(4096 + 16)) == INVALID
    assert bwd(n=16) == WORKSPACE
    assert lib.tt_emb_norm_workspace_bytes(0, 5, 8) >= 2 * 8 * 4
    assert lib.tt_emb_norm_workspace_bytes(0, 0, 8) > 0
    assert lib.tt_emb_norm_workspace_bytes(7, 5, 8) == 0 and lib.tt_emb_norm_workspace_bytes(0, 5, 0) == 0


def test_gate_refusals():
    lib = tte.load_library()

    def fwd(dtype=0, x=A, ldx=8, wg=A, wu=A, out=A, ldo=16, gate=None, up=None, rows=2, dim=8, hidden=16, act=0, ws=A,
            n=1 << 24):
        return lib.tt_emb_gate_forward(dtype, x, ldx, wg, wu, out, ldo, gate, up, rows, dim, hidden, act, ws, n, None)

    assert fwd(dtype=3) == INVALID
    for k in ("x", "wg", "wu", "out", "ws"):
        assert fwd(**{k: None}) == INVALID, k
    assert fwd(ldx=7) == INVALID and fwd(ldo=15) == INVALID
    assert fwd(gate=A) == INVALID and fwd(up=A) == INVALID
    assert fwd(act=3) == INVALID and fwd(act=-1) == INVALID
    assert fwd(rows=-1) == INVALID and fwd(dim=0) == INVALID and fwd(hidden=0) == INVALID
    assert fwd(dim=1 << 20, ldx=1 << 20) == UNSUPPORTED and fwd(rows=1 << 22) == UNSUPPORTED
    assert fwd(ldx=1 << 22) == UNSUPPORTED
    assert fwd(ws=P(4096 + 128)) == INVALID and fwd(n=64) == WORKSPACE
    assert fwd(rows=0, x=None, out=None) == 0

    def bwd(x=A, ldx=8, wg=A, wu=A, gate=A, up=A, dout=A, ldd=16, dx=A, lddx=8, dwg=A, dwu=A, rows=2, act=1, ws=A,
            n=1 << 24):
        return lib.tt_emb_gate_backward(1, x, ldx, wg, wu, gate, up, dout, ldd, dx, lddx, dwg, dwu, rows, 8, 16, act,
                                        ws, n, None)

    for k in ("x", "wg", "wu", "gate", "up", "dout", "dx", "dwg", "dwu", "ws"):
        assert bwd(**{k: None}) == INVALID, k
    assert bwd(ldx=7) == INVALID and bwd(ldd=15) == INVALID and bwd(lddx=7) == INVALID
    assert bwd(act=9) == INVALID and bwd(n=0) == WORKSPACE
    assert lib.tt_emb_gate_workspace_bytes(1, 2, 8, 0) == 0
    assert lib.tt_emb_gate_workspace_bytes(1, 0, 8, 8) > 0


def test_distill_refusals():
    lib = tte.load_library()

    def fwd(dtype=0, z=A, ld=100, ids=A, tl=A, top=4, loss=A, stats=None, rows=2, classes=100, t=1.0, ws=A, n=1 << 20):
        return lib.tt_emb_distill_forward(dtype, z, ld, ids, tl, top, loss, stats, rows, classes, F(t), ws, n, None)

    assert fwd(dtype=5) == INVALID
    for k in ("z", "ids", "tl", "loss", "ws"):
        assert fwd(**{k: None}) == INVALID, k
    assert fwd(ld=99) == INVALID and fwd(top=-1) == INVALID and fwd(top=1025) == UNSUPPORTED
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert fwd(t=t) == INVALID, t
    assert fwd(rows=-1) == INVALID and fwd(classes=0) == INVALID
    assert fwd(classes=(1 << 30) + 1, ld=1 << 31) == UNSUPPORTED
    assert fwd(ws=P(4097)) == INVALID and fwd(n=8) == WORKSPACE
    assert fwd(rows=0, z=None, ids=None, tl=None, loss=None) == 0

    def bwd(z=A, ld=100, ids=A, tl=A, stats=A, w=A, dz=A, ldd=100):
        return lib.tt_emb_distill_backward(0, z, ld, ids, tl, 4, stats, w, dz, ldd, 2, 100, F(1.0), None)

    for k in ("z", "ids", "tl", "stats", "w", "dz"):
        assert bwd(**{k: None}) == INVALID, k
    assert bwd(ldd=99) == INVALID

    def train(w=A, loss=A, dz=A, ldd=100, ws=A, n=1 << 20):
        return lib.tt_emb_distill_train(0, A, 100, A, A, 4, w, loss, dz, ldd, 2, 100, F(1.0), ws, n, None)

    for k in ("w", "loss", "dz", "ws"):
        assert train(**{k: None}) == INVALID, k
    assert train(ldd=1) == INVALID and train(n=1) == WORKSPACE
    assert lib.tt_emb_distill_workspace_bytes(0, 2, 0) == 0


def test_benchmark_counters_outlive_the_dense_sources(tmp_path, monkeypatch):
    """The benchmark's recorded HBM counters belong to the embedding's sources alone."""
    import shutil

    import bench
    assert bench.kernel_source_hash()
    shutil.copytree(bench.CSRC, tmp_path / "csrc")
    monkeypatch.setattr(bench, "CSRC", str(tmp_path / "csrc"))
    first = bench.kernel_source_hash()
    for f in ("gate.hip", "norm.hip", "distill.hip", "tt_dense.h"):
        (tmp_path / "csrc" / f).write_text("changed")
        assert bench.kernel_source_hash() == first, f
    (tmp_path / "csrc" / "plan.hip").write_text("changed")
    assert bench.kernel_source_hash() != first


def test_binding_refuses_what_the_abi_cannot_see():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        tte.tt_emb_norm_forward(x, x[0], None, x)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        tte.tt_emb_norm_workspace_bytes(torch.float64, 4, 8)
    with pytest.raises(ValueError, match="act must be"):
        tte.tt_emb_gate_forward(x, x, x, x, act="tanh")


def _differences(f, x, d, h=1e-5):
    """Derivative of sum(f * d) in every element of x, by central differences."""
    out = torch.empty_like(x)
    for i in range(x.numel()):
        a = x.clone().flatten()
        a[i] += h
        up = float((f(a.view_as(x)) * d).sum())
        a[i] -= 2 * h
        out.view(-1)[i] = (up - float((f(a.view_as(x)) * d).sum())) / (2 * h)
    return out


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_closed_form_gradients_against_differences():
    # central differences with h = 1e-5 are off by about h^2 and 1e-16 / h
    x, w, b, dy = _rand(3, 7), _rand(7, seed=1), _rand(7, seed=2), _rand(3, 7, seed=3)
    dx, dw, db = ref.norm_grads(x, w, dy, 1e-5)
    f = lambda x, w, b: ref.norm(x, w, b, 1e-5)[0]   # noqa: E731
    torch.testing.assert_close(_differences(lambda v: f(v, w, b), x, dy), dx, rtol=1e-7, atol=1e-8)
    torch.testing.assert_close(_differences(lambda v: f(x, v, b), w, dy), dw, rtol=1e-7, atol=1e-8)
    torch.testing.assert_close(_differences(lambda v: f(x, w, v), b, dy), db, rtol=1e-7, atol=1e-8)
    x, wg, wu, d = _rand(3, 5), _rand(4, 5, seed=1), _rand(4, 5, seed=2), _rand(3, 4, seed=3)
    for kind in ("silu", "gelu", "relu"):
        dx, dg, du = ref.gate_grads(x, wg, wu, d, kind)
        g = lambda x, a, b: ref.gate(x, a, b, kind)[0]   # noqa: E731
        torch.testing.assert_close(_differences(lambda v: g(v, wg, wu), x, d), dx, rtol=1e-6, atol=1e-7)
        torch.testing.assert_close(_differences(lambda v: g(x, v, wu), wg, d), dg, rtol=1e-6, atol=1e-7)
        torch.testing.assert_close(_differences(lambda v: g(x, wg, v), wu, d), du, rtol=1e-6, atol=1e-7)
    z = 2 * _rand(4, 9)
    ids = torch.tensor([[0, 3, 8], [2, -1, 9], [-1, -1, -1], [5, 5, 1]])
    tl = _rand(4, 3, seed=5)
    one = torch.ones(4, dtype=torch.float64)
    for t in (1.0, 2.5):
        grad = ref.distill(z, ids, tl, t)[1]
        torch.testing.assert_close(_differences(lambda v: ref.distill(v, ids, tl, t)[0], z, one), grad, rtol=1e-6,
                                   atol=1e-7)

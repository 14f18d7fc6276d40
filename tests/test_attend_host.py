"""Checks of the attention operators that need no GPU: refusals on the host
before any launch, workspace sizes, the binding's checks, and the closed-form
gradients of the 64-bit definitions against differences."""
import ctypes
import math
import random

import pytest

import tensor_train_compressed_amd as tte

torch = pytest.importorskip("torch")
from tests import attend_ref as ref  # noqa: E402
from tests.test_dense_device import Machine, Tensor  # noqa: E402
from tests.test_dense_host import _differences, _rand  # noqa: E402
from tests.test_dense_workspace import rising  # noqa: E402

P = ctypes.c_void_p
A = P(4096)     # an aligned address that no refused call may touch
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
F = ctypes.c_float
BF16, F32 = torch.bfloat16, torch.float32


class Call:
    """A call of the library with named arguments, most of them left as they are good."""

    def __init__(self, name, **good):
        self.f, self.good = getattr(tte.load_library(), name), good

    def __call__(self, **changed):
        assert set(changed) <= set(self.good), set(changed) - set(self.good)
        return self.f(*{**self.good, **changed}.values(), None)

    def refuse(self, status, **one_by_one):
        for k, vs in one_by_one.items():
            for v in vs if isinstance(vs, (list, tuple)) else [vs]:
                assert self(**{k: v}) == status, (k, v)


SIZES = dict(rows=2, heads=4, kv=2, dim=8)


def rotate_head():
    return dict(dtype=0, wdtype=0, q=A, ldq=32, k=A, ldk=16)


def rotate_turn():
    return dict(wq=A, wk=A, positions=A, freq=A, rot=8, pairs=0)


def check_rotate_shared(c):
    c.refuse(INVALID, dtype=[3, -1], wdtype=3, q=None, k=None, wq=None, wk=None, positions=None, freq=None, ldq=31,
             ldk=15, rot=[-2, 3, 10], pairs=[2, -1], rows=-1, heads=0, kv=0, dim=0,
             eps=[F(-1.0), F(math.nan), F(math.inf)])
    c.refuse(UNSUPPORTED, wdtype=1, rows=(1 << 24) + 1)
    assert c(dim=257, ldq=2000, ldk=2000) == UNSUPPORTED
    assert c(heads=4097, ldq=1 << 20) == UNSUPPORTED and c(kv=4097, ldk=1 << 20) == UNSUPPORTED


def test_rotate_forward_refusals():
    c = Call("tt_emb_rotate_forward", **rotate_head(), **rotate_turn(), qo=A, ldqo=32, ko=A, ldko=16, **SIZES, eps=F(1e-6))
    check_rotate_shared(c)
    c.refuse(INVALID, qo=None, ko=None, ldqo=31, ldko=15)
    assert c(rows=0, q=None, k=None, positions=None, qo=None, ko=None) == OK


def test_rotate_append_refusals():
    c = Call("tt_emb_rotate_append", **rotate_head(), v=A, ldv=16, **rotate_turn(), slots=A, qo=A, ldqo=32, kp=A, vp=A,
             nslots=16, **SIZES, eps=F(1e-6))
    check_rotate_shared(c)
    c.refuse(INVALID, v=None, slots=None, qo=None, kp=None, vp=None, ldv=15, ldqo=31, nslots=-1)
    assert c(rows=0, q=None, k=None, v=None, positions=None, slots=None, qo=None, kp=None, vp=None) == OK


def test_rotate_backward_refusals():
    c = Call("tt_emb_rotate_backward", **rotate_head(), **rotate_turn(), dqo=A, lddqo=32, dko=A, lddko=16, dq=A, lddq=32,
             dk=A, lddk=16, dwq=A, dwk=A, **SIZES, eps=F(1e-6), ws=A, n=1 << 20)
    check_rotate_shared(c)
    c.refuse(INVALID, dqo=None, dko=None, dq=None, dk=None, dwq=None, dwk=None, lddqo=31, lddko=15, lddq=31, lddk=15,
             ws=[None, P(4096 + 16)])
    c.refuse(WORKSPACE, n=16)


def check_attend_shared(c):
    c.refuse(INVALID, dtype=[3, -1], q=None, k=None, v=None, offsets=None, ldq=31, ldk=15, ldv=15, seqs=-1, rows=-1,
             heads=[0, 3], kv=0, dim=0, scale=[F(0.0), F(-1.0), F(math.nan), F(math.inf), F(2.5e38)])
    c.refuse(UNSUPPORTED, ldq=1 << 22, ldk=1 << 22, ldv=1 << 22, rows=1 << 31, seqs=1 << 24)
    assert c(dim=129, ldq=2000, ldk=2000, ldv=2000, ldo=2000, **({"lddo": 2000, "lddq": 2000, "lddk": 2000, "lddv": 2000}
                                                                if "lddo" in c.good else {})) == UNSUPPORTED


def test_attend_refusals():
    head = dict(dtype=0, q=A, ldq=32, k=A, ldk=16, v=A, ldv=16, offsets=A, seqs=1)
    c = Call("tt_emb_attend_forward", **head, out=A, ldo=64, lse=None, **SIZES, causal=1, scale=F(1.0))
    check_attend_shared(c)
    c.refuse(INVALID, out=None, ldo=31)
    assert c(rows=1 << 25, heads=8, kv=2, ldq=64) == UNSUPPORTED        # more threads than a launch takes
    assert c(seqs=(1 << 20) + 1) == UNSUPPORTED
    assert c(rows=0, q=None, k=None, v=None, offsets=None, out=None) == OK and c(seqs=0) == OK
    c = Call("tt_emb_attend_backward", **head, out=A, ldo=32, lse=A, dout=A, lddo=32, dq=A, lddq=32, dk=A, lddk=16, dv=A,
             lddv=16, **SIZES, causal=1, scale=F(1.0), ws=A, n=1 << 20)
    check_attend_shared(c)
    c.refuse(INVALID, out=None, lse=None, dout=None, dq=None, dk=None, dv=None, ldo=31, lddo=31, lddq=31, lddk=15,
             lddv=15, ws=[None, P(4096 + 16)])
    c.refuse(UNSUPPORTED, lddo=1 << 22)
    c.refuse(WORKSPACE, n=16)
    assert c(seqs=0) == OK


def test_paged_refusals():
    c = Call("tt_emb_attend_paged", dtype=0, q=A, ldq=32, kp=A, vp=A, pages=10, page=16, table=A, ldt=5, most=5, lengths=A,
             out=A, ldo=32, seqs=2, heads=4, kv=2, dim=8, scale=F(1.0), ws=A, n=1 << 24)
    c.refuse(INVALID, dtype=[3, -1], q=None, kp=None, vp=None, table=None, lengths=None, out=None, ldq=31, ldo=31,
             pages=-1, page=[0, -1], most=[-1, 6], seqs=-1, heads=[0, 3], kv=0, dim=0,
             scale=[F(0.0), F(-1.0), F(math.nan), F(math.inf), F(2.5e38)], ws=[None, P(4096 + 128)])
    assert c(dim=129, ldq=2000, ldo=2000) == UNSUPPORTED and c(heads=514, ldq=1 << 14, ldo=1 << 14) == UNSUPPORTED
    c.refuse(UNSUPPORTED, page=1 << 31, seqs=1 << 19, pages=1 << 31)
    assert c(most=(1 << 26) + 1, ldt=1 << 27) == UNSUPPORTED                  # tokens of a sequence past 2^30
    c.refuse(WORKSPACE, n=64)
    assert c(seqs=0, q=None, lengths=None, out=None, table=None) == OK


def test_workspaces():
    rng = random.Random(1)
    rows = sorted({*range(70), *(rng.randrange(1, 40000) for _ in range(200))})
    for dt in (F32, BF16):
        for h, kv, d in ((4, 4, 32), (32, 8, 128), (7, 1, 33), (256, 1, 64), (80, 2, 128)):
            rising([(m, tte.tt_emb_rotate_workspace_bytes(dt, m, h, kv, d)) for m in rows])
            rising([(m, tte.tt_emb_attend_workspace_bytes(dt, m, h, kv, d)) for m in rows])
            rising([(m, tte.tt_emb_attend_paged_workspace_bytes(dt, m, h, kv, d)) for m in range(0, 3000)])
    lib = tte.load_library()
    assert lib.tt_emb_rotate_workspace_bytes(0, 4, 4, 2, 257) == 0 and lib.tt_emb_rotate_workspace_bytes(9, 4, 4, 2, 8) == 0
    for f in (lib.tt_emb_attend_workspace_bytes, lib.tt_emb_attend_paged_workspace_bytes):
        assert f(0, 4, 4, 2, 129) == 0 and f(0, 4, 5, 2, 8) == 0 and f(0, -1, 4, 2, 8) == 0 and f(0, 0, 4, 2, 8) > 0


# ---------------------------------------------------------------- the binding

def test_binding_refuses_what_the_abi_cannot_see(monkeypatch):
    Machine(monkeypatch, current=1)
    I64, F64, I32 = torch.int64, torch.float64, torch.int32
    q, k, w, pos, freq = Tensor(4, 32), Tensor(4, 16), Tensor(8), Tensor(4, dtype=I64), Tensor(4, dtype=F64)

    def rot(**c):
        a = {**dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, freq=freq, q_out=q, k_out=k), **c}
        tte.tt_emb_rotate_forward(**a)
    rot()
    for bad in (dict(k=Tensor(3, 16)), dict(k=Tensor(4, 15)), dict(q=Tensor(4, 33)), dict(k_weight=Tensor(7)),
                dict(k_weight=Tensor(8, dtype=BF16)), dict(positions=Tensor(5, dtype=I64)), dict(positions=Tensor(4)),
                dict(freq=Tensor(4)), dict(q_out=Tensor(4, 40)), dict(k_out=Tensor(4, 16, dtype=BF16)),
                dict(pairs="thirds"), dict(q=Tensor(4, 32, dtype=F64))):
        with pytest.raises(ValueError):
            rot(**bad)
    kp = Tensor(6, 16, 2, 8)

    def app(**c):
        a = {**dict(q=q, k=k, v=k, q_weight=w, k_weight=w, positions=pos, freq=freq, slots=pos, q_out=q, k_pages=kp,
                    v_pages=kp), **c}
        tte.tt_emb_rotate_append(**a)
    app()
    for bad in (dict(v=Tensor(4, 8)), dict(slots=Tensor(3, dtype=I64)), dict(slots=Tensor(4, dtype=I32)),
                dict(k_pages=Tensor(6, 16, 2, 9)), dict(v_pages=Tensor(6, 16, 2, 7)), dict(k_pages=Tensor(6, 16, 16)),
                dict(k_pages=Tensor(6, 16, 3, 8), v_pages=Tensor(6, 16, 3, 8))):
        with pytest.raises(ValueError):
            app(**bad)
    off, lse = Tensor(3, dtype=I64), Tensor(4, 4)

    def att(**c):
        a = {**dict(q=q, k=k, v=k, offsets=off, out=q, lse=lse, dout=q, dq=q, dk=k, dv=k, heads=4, kv_heads=2), **c}
        tte.tt_emb_attend_backward(**a)
        fwd = {x: a[x] for x in ("q", "k", "v", "offsets", "out", "lse", "heads", "kv_heads")}
        tte.tt_emb_attend_forward(**fwd)
    att()
    for bad in (dict(heads=3), dict(heads=0), dict(kv_heads=1), dict(k=Tensor(5, 16)), dict(offsets=Tensor(3)),
                dict(offsets=Tensor(0, dtype=I64)), dict(lse=Tensor(4, 3)), dict(out=Tensor(4, 16)), dict(dv=Tensor(4, 8)),
                dict(dout=Tensor(4, 32, dtype=BF16))):
        with pytest.raises(ValueError):
            att(**bad)
    table, lengths = Tensor(4, 9, dtype=I32), Tensor(4, dtype=I64)

    def pag(**c):
        tte.tt_emb_attend_paged(**{**dict(q=q, k_pages=kp, v_pages=kp, table=table, lengths=lengths, out=q), **c})
    pag()
    for bad in (dict(q=Tensor(4, 30)), dict(table=Tensor(3, 9, dtype=I32)), dict(table=Tensor(4, 9, dtype=I64)),
                dict(lengths=Tensor(4, dtype=I32)), dict(lengths=Tensor(5, dtype=I64)), dict(out=Tensor(4, 16)),
                dict(v_pages=Tensor(6, 16, 2, 8, dtype=BF16))):
        with pytest.raises(ValueError):
            pag(**bad)


@pytest.mark.parametrize("stream", [None, 77])
def test_calls_run_where_their_tensors_are(monkeypatch, stream):
    m = Machine(monkeypatch)
    I64, F64, I32 = torch.int64, torch.float64, torch.int32
    q, k, w, pos, freq = Tensor(4, 32), Tensor(4, 16), Tensor(8), Tensor(4, dtype=I64), Tensor(4, dtype=F64)
    kp, off, lse, table = Tensor(6, 16, 2, 8), Tensor(3, dtype=I64), Tensor(4, 4), Tensor(4, 9, dtype=I32)
    s = dict(stream=stream)
    tte.tt_emb_rotate_forward(q, k, w, w, pos, freq, q, k, **s)
    tte.tt_emb_rotate_append(q, k, k, w, w, pos, freq, pos, q, kp, kp, **s)
    tte.tt_emb_rotate_backward(q, k, w, w, pos, freq, q, k, q, k, w, w, **s)
    tte.tt_emb_attend_forward(q, k, k, off, q, lse, heads=4, kv_heads=2, **s)
    tte.tt_emb_attend_backward(q, k, k, off, q, lse, q, q, k, k, heads=4, kv_heads=2, **s)
    tte.tt_emb_attend_paged(q, kp, kp, table, pos, q, **s)
    on = stream or 101
    assert m.calls == [("tt_emb_" + n, 1, on) for n in ("rotate_forward", "rotate_append", "rotate_backward",
                                                        "attend_forward", "attend_backward", "attend_paged")]
    assert m.allocated == [(1, on)] * 3


# -------------------------------------------------------------- the formulas

def test_closed_form_gradients_against_differences():
    # central differences with h = 1e-5 are off by about h^2 and 1e-16 / h
    q, w, dy = _rand(3, 2 * 6), _rand(6, seed=1), _rand(3, 12, seed=2)
    pos = torch.tensor([0, 7, 100000])
    for pairs in ("halves", "neighbours"):
        for freq in (torch.tensor([1.0, 0.1], dtype=torch.float64), torch.zeros(0, dtype=torch.float64)):
            f = lambda x, y: ref.rotate(x, y, pos, freq, 6, pairs, 1e-6)[0]   # noqa: E731
            dx, dw = ref.rotate_grads(q, w, pos, freq, 6, pairs, 1e-6, dy)
            torch.testing.assert_close(_differences(lambda v: f(v, w), q, dy), dx, rtol=1e-6, atol=1e-7)
            torch.testing.assert_close(_differences(lambda v: f(q, v), w, dy), dw, rtol=1e-6, atol=1e-7)
    q, k, v, do = _rand(7, 4 * 3), _rand(7, 2 * 3, seed=1), _rand(7, 2 * 3, seed=2), _rand(7, 12, seed=3)
    ref.U[torch.float64], ref.TINY[torch.float64] = ref.U32, ref.TINY[F32]
    for causal in (False, True):
        def f(q, k, v):
            return torch.nan_to_num(ref.attend(q, k, v, [4, 0, 2], 0, 4, 2, causal, 0.7)[0][0])
        want = ref.attend(q, k, v, [4, 0, 2], 0, 4, 2, causal, 0.7, do)[0]
        for i, g in ((2, lambda x: f(x, k, v)), (3, lambda x: f(q, x, v)), (4, lambda x: f(q, k, x))):
            got = _differences(g, (q, k, v)[i - 2], do)
            torch.testing.assert_close(got[:6], want[i][:6], rtol=1e-6, atol=1e-7)
            assert bool((got[6] == 0).all()) and bool(want[i][6].isnan().all())


def test_definitions_against_torch():
    """The rotation against complex numbers, attention against torch's softmax."""
    q, w, pos = _rand(5, 16), _rand(8, seed=1), torch.tensor([0, 1, 5, 1000, 99999])
    freq = 10000.0 ** (-torch.arange(4, dtype=torch.float64) / 4)
    h = q.view(5, 2, 8)
    u = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w
    z = torch.polar(torch.ones(5, 4, dtype=torch.float64), torch.outer(pos.double(), freq))[:, None]
    got = ref.rotate(q, w, pos, freq, 8, "neighbours", 1e-6)[0].view(5, 2, 8)
    torch.testing.assert_close(torch.view_as_real(torch.view_as_complex(u.view(5, 2, 4, 2).contiguous()) * z).flatten(2), got)
    got = ref.rotate(q, w, pos, freq, 8, "halves", 1e-6)[0].view(5, 2, 8)
    both = torch.complex(u[..., :4], u[..., 4:]) * z
    torch.testing.assert_close(torch.cat((both.real, both.imag), -1), got)
    q, k, v = _rand(6, 4 * 3), _rand(6, 2 * 3, seed=1), _rand(6, 2 * 3, seed=2)
    ref.U[torch.float64], ref.TINY[torch.float64] = ref.U32, ref.TINY[F32]
    out, lse = ref.attend(q, k, v, [6], 0, 4, 2, True, 0.5)[0]
    s = torch.einsum("ihd,jhd->hij", q.view(6, 4, 3), k.view(6, 2, 3).repeat_interleave(2, 1)) * 0.5
    s = s.masked_fill(torch.ones(6, 6, dtype=torch.bool).triu(1), -math.inf)
    torch.testing.assert_close(lse, torch.logsumexp(s, -1))
    want = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v.view(6, 2, 3).repeat_interleave(2, 1)).flatten(1)
    torch.testing.assert_close(out, want)
    pages = torch.zeros(4, 2, 2, 3, dtype=torch.float64)
    pages_v = pages.clone()
    table = torch.tensor([[2, 0, 3, -1]], dtype=torch.int32)
    for j in range(6):
        pages[table[0, j // 2], j % 2], pages_v[table[0, j // 2], j % 2] = k[j].view(2, 3), v[j].view(2, 3)
    one, _ = ref.paged(q[5:], pages, pages_v, table, torch.tensor([6]), 0.5)
    torch.testing.assert_close(one[0], out[5])


def test_benchmark_counters_outlive_the_attention_sources(tmp_path, monkeypatch):
    """The benchmark's recorded HBM counters belong to the embedding's sources alone."""
    import shutil

    import bench
    first = bench.kernel_source_hash()
    shutil.copytree(bench.CSRC, tmp_path / "csrc")
    monkeypatch.setattr(bench, "CSRC", str(tmp_path / "csrc"))
    for f in ("rotate.hip", "attend.hip", "attend_dq.hip", "attend_dkv.hip", "paged.hip", "tt_attend.h", "attend.h"):
        (tmp_path / "csrc" / f).write_text("changed")
        assert bench.kernel_source_hash() == first, f

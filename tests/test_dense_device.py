"""The dense operators' binding with tensors that are not on the current device: the
kernel and the workspace the call allocates are on the tensors' device and its stream.
Stand-ins for device tensors, streams and the library: no GPU is touched."""
import contextlib

import pytest

import tensor_train_compressed_amd as tte

torch = pytest.importorskip("torch")
F32 = torch.float32


class Tensor:
    """What the binding asks of a device tensor."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, *shape, dtype=F32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def stride(self):
        return (self.shape[1], 1)

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.device.index


class Machine:
    """Two devices, the current one 0; a current stream each; a library that notes its calls."""

    def __init__(self, monkeypatch, current=0):
        self.device, self.stream, self.calls, self.allocated = current, None, [], []
        c = torch._C
        monkeypatch.setattr(c, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(c, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: ("stream", 100 + torch.device(d).index))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: ("stream", s))
        monkeypatch.setattr(torch.cuda, "device", self.on_device)
        monkeypatch.setattr(torch.cuda, "stream", self.on_stream)
        monkeypatch.setattr(torch, "empty", self.empty)
        monkeypatch.setattr(tte, "load_library", lambda: self)

    @contextlib.contextmanager
    def on_device(self, d):
        was, self.device = self.device, torch.device(d).index if not isinstance(d, int) else d
        yield
        self.device = was

    @contextlib.contextmanager
    def on_stream(self, s):
        was, self.stream = self.stream, s
        yield
        self.stream = was

    def empty(self, n, dtype=None, device=None):
        self.allocated.append((torch.device(device).index, self.stream[1]))
        return Tensor(n, dtype=dtype)

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 256

        def call(*a):
            self.calls.append((name, self.device, a[-1]))
            return 0
        return call


def every_call(stream=None):
    x, w, s, y, h = Tensor(4, 8), Tensor(8), Tensor(4), Tensor(4, 8), Tensor(4, 16)
    wg, ids, tl, st = Tensor(16, 8), Tensor(4, 3, dtype=torch.int64), Tensor(4, 3), Tensor(4, 2)
    k = dict(stream=stream)
    tte.tt_emb_norm_forward(x, w, w, y, s, s, **k)
    tte.tt_emb_norm_backward(x, w, s, s, y, y, w, w, **k)
    tte.tt_emb_gate_forward(x, wg, wg, h, h, h, **k)
    tte.tt_emb_gate_backward(x, wg, wg, h, h, h, y, wg, wg, **k)
    tte.tt_emb_distill_forward(x, ids, tl, s, st, **k)
    tte.tt_emb_distill_backward(x, ids, tl, st, s, y, **k)
    tte.tt_emb_distill_train(x, ids, tl, s, s, y, **k)


NAMES = ["tt_emb_norm_forward", "tt_emb_norm_backward", "tt_emb_gate_forward", "tt_emb_gate_backward",
         "tt_emb_distill_forward", "tt_emb_distill_backward", "tt_emb_distill_train"]


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_where_their_tensors_are(monkeypatch, current):
    m = Machine(monkeypatch, current)
    every_call()
    assert m.calls == [(n, 1, 101) for n in NAMES]          # on device 1 and its current stream
    assert m.allocated == [(1, 101)] * 5                    # and so the workspaces
    assert m.device == current


def test_a_given_stream_is_the_workspaces_too(monkeypatch):
    m = Machine(monkeypatch)
    every_call(stream=77)
    assert m.calls == [(n, 1, 77) for n in NAMES]
    assert m.allocated == [(1, 77)] * 5

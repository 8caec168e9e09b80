"""The bindings without a GPU: CPU tensors that say they are on a CUDA device,
and a library that records what it is called with."""
from __future__ import annotations

import contextlib

import pytest

import linear_attention_recurrence_step_gb300 as gdn
from linear_attention_recurrence_step_gb300 import layer

torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A CPU tensor that reports a CUDA device."""
    index = 0
    device = property(lambda self: torch.device("cuda", self.index))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def cuda(*shape, dtype=torch.float32, index=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


class Side:
    """A stream object."""
    cuda_stream = 0x7000


class Library:
    """Takes every call, with the sizes that the workspace calls are to give."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_size"):
                return 1 << 12
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    """The recorded calls; `lib.made` holds the stream of every allocation (None:
    the current one)."""
    lib, inside = Library(), []
    lib.made, lib.current = [], 0
    real = torch.empty

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        try:
            yield
        finally:
            inside.pop()

    def empty(*shape, dtype=None, device=None, **kw):
        lib.made.append(inside[-1].cuda_stream if inside else None)
        t = real(*shape, dtype=dtype).as_subclass(OnDevice)
        t.index = torch.device(device).index or 0
        return t

    class External:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    monkeypatch.setattr(gdn, "_lib", lib)
    monkeypatch.setattr(layer, "_raw_stream", lambda dev: 0x5000)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: type("S", (), {"cuda_stream": 0x5000}))
    monkeypatch.setattr(gdn, "_one_device", False)
    monkeypatch.setattr(gdn, "_current_device", lambda: lib.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: External(0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype, device=t.device))
    layer._scan_workspace.cache_clear()
    yield lib
    layer._scan_workspace.cache_clear()


def _calls():
    """name -> (the call, how many outputs and workspaces it allocates)."""
    B, T, Hk, Hv, D = 2, 20, 1, 2, 64
    q, v, g, st = cuda(B, T, Hk, D), cuda(B, T, Hv, D), cuda(B, T, Hv), cuda(B, Hv, D, D)
    tape = (v, cuda(B, T, Hv, D), g, st)
    acc = cuda(B, dtype=torch.int32)
    x, w = cuda(B, T, 64), cuda(64, 4)
    bc = cuda(B, T, 1, 64)
    return {
        "step_record": (lambda **kw: gdn.gdn_step_record(q, q, v, g, g, st, capture_tape=True, **kw), 5),
        "step_record_mapped": (lambda **kw: gdn.gdn_step_record_mapped(q, q, v, g, g, st, mapping="tiled", **kw), 3),
        "chunk_prefill": (lambda **kw: gdn.gdn_chunk_prefill(q, q, v, g, g, st, capture_tape=True, **kw), 6),
        "chunk_prefill_noalloc": (lambda **kw: gdn.gdn_chunk_prefill_noalloc(q, q, v, g, g, st, **kw), 3),
        "state_replay": (lambda **kw: gdn.gdn_state_replay(*tape, accepted=3, **kw), 1),
        "state_replay_per_seq": (lambda **kw: gdn.gdn_state_replay_per_seq(*tape, accepted=acc, **kw), 1),
        "chunk_replay": (lambda **kw: gdn.gdn_chunk_replay(*tape, accepted=3, **kw), 2),
        "repeat_tiled": (lambda **kw: gdn.gqa_repeat_tiled(v.reshape(B * T, Hv, D), 4, **kw), 1),
        "causal_conv": (lambda **kw: gdn.gdn_causal_conv(x, w, **kw), 2),
        "selective_scan": (lambda **kw: gdn.gdn_selective_scan(v, g, cuda(Hv), bc, bc, **kw), 3),
        "gated_norm": (lambda **kw: gdn.gdn_gated_norm(x, cuda(64), residual=x, **kw), 2),
        "sample": (lambda **kw: gdn.gdn_sample(x, x, **kw), 2),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_allocations_belong_to_the_calls_stream(lib, name):
    """Outputs and workspaces that a call allocates come from the memory of the
    stream that its kernels run on: a workspace is free again when the call
    returns, and only work behind it in that stream may then have it."""
    call, count = _calls()[name]
    for given, handle, owner in ((None, 0x5000, None), (Side(), 0x7000, 0x7000), (0x7100, 0x7100, 0x7100),
                                 (0, 0, 0), (1, 1, 0)):
        lib.made.clear()
        lib.calls.clear()
        call(stream=given)
        assert lib.made == [owner] * count
        assert [args[-1] for _, args in lib.calls] == [handle]


@pytest.mark.parametrize("name", list(_calls()))
def test_another_device_is_refused(lib, name):
    """Kernels run on the current device: tensors of another one are refused
    before the library is called."""
    call, _ = _calls()[name]
    lib.current = 1
    with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
        call()
    assert not lib.calls
    lib.current = 0
    call()
    assert len(lib.calls) == 1


# a call of the norm, and the M, K, D and token strides of x and gate that the library gets
def _norms():
    kv = cuda(6, 576)                                  # a fused projection
    seq = cuda(2, 5, 200)
    heads = cuda(4, 3 * 64 + 8)
    w = lambda *s: cuda(*s)  # noqa: E731
    return {
        "rows of a projection": (lambda **kw: gdn.gdn_gated_norm(kv[:, :512], w(512), **kw), (6, 1, 512, 576, 576)),
        "three dimensions": (lambda **kw: gdn.gdn_gated_norm(seq[..., 8:72], w(64), **kw), (10, 1, 64, 200, 200)),
        "one row": (lambda **kw: gdn.gdn_gated_norm(kv[0, 3:35], w(32), **kw), (1, 1, 32, 32, 32)),
        "one of many": (lambda **kw: gdn.gdn_gated_norm(kv[2:3, :512], w(512), **kw), (1, 1, 512, 512, 512)),
        "a sliced gate": (lambda **kw: gdn.gdn_gated_norm(cuda(6, 512), w(512), gate=kv[:, 64:], **kw), (6, 1, 512, 512, 576)),
        "a sliced x": (lambda **kw: gdn.gdn_gated_norm(kv[:, 64:], w(512), gate=cuda(6, 512), **kw), (6, 1, 512, 576, 512)),
        "heads of a projection": (lambda **kw: gdn.gdn_gated_norm(heads[:, :192].unflatten(-1, (3, 64)), w(64), **kw),
                                  (4, 3, 64, 200, 200)),
        "heads, x whole": (lambda **kw: gdn.gdn_gated_norm(cuda(4, 3, 64), w(64), gate=heads[:, 8:].unflatten(-1, (3, 64)), **kw),
                           (4, 3, 64, 192, 200)),
        "a weight per head": (lambda **kw: gdn.gdn_gated_norm(heads[:, :192].unflatten(-1, (3, 64)), w(3, 64), **kw),
                              (4, 3, 64, 200, 200)),
        "whole": (lambda **kw: gdn.gdn_gated_norm(cuda(4, 3, 64), w(64), **kw), (12, 1, 64, 64, 64)),
    }


@pytest.mark.parametrize("name", list(_norms()))
def test_norm_takes_slices(lib, name):
    """Rows, and tokens of several heads, of a wider tensor, x and gate each."""
    call, want = _norms()[name]
    call()
    (_, args), = lib.calls
    assert args[6:11] == want


def test_norm_refuses_what_is_not_rows(lib):
    for x in (cuda(64, 6).t(), cuda(4, 5, 64).transpose(0, 1), cuda(4, 64).expand(4, 64)[:, ::2]):
        with pytest.raises(ValueError, match="x's"):
            gdn.gdn_gated_norm(x, cuda(x.shape[-1]))
    with pytest.raises(ValueError, match="gate's"):
        gdn.gdn_gated_norm(cuda(6, 64), cuda(64), gate=cuda(64, 6).t())
    assert not lib.calls


def _wrong_arguments():
    x, w, v, g = cuda(2, 20, 64), cuda(64, 4), cuda(2, 20, 2, 64), cuda(2, 20, 2)
    bc, A = cuda(2, 20, 1, 64), cuda(2)
    conv, scan, norm, sample = gdn.gdn_causal_conv, gdn.gdn_selective_scan, gdn.gdn_gated_norm, gdn.gdn_sample
    calls = {
        "conv x list": lambda: conv([1.0], w), "conv x flat": lambda: conv(x[0], w),
        "conv weight list": lambda: conv(x, [1.0]), "conv weight flat": lambda: conv(x, w[:, 0]),
        "conv weight none": lambda: conv(x, None), "conv bias list": lambda: conv(x, w, bias=[0.0]),
        "conv lengths list": lambda: conv(x, w, lengths=[1, 2]), "conv state list": lambda: conv(x, w, [0.0]),
        "scan x flat": lambda: scan(x, g, A, bc, bc), "scan dt none": lambda: scan(v, None, A, bc, bc),
        "scan B none": lambda: scan(v, g, A, None, bc), "scan B flat": lambda: scan(v, g, A, x, x),
        "scan C list": lambda: scan(v, g, A, bc, [1]), "scan A list": lambda: scan(v, g, [1.0, 2.0], bc, bc),
        "scan D number": lambda: scan(v, g, A, bc, bc, D=1.0), "scan workspace": lambda: scan(v, g, A, bc, bc, workspace=4096),
        "norm x number": lambda: norm(cuda()[()], cuda(1)), "norm weight list": lambda: norm(x, [1.0]),
        "norm gate list": lambda: norm(x, cuda(64), gate=[1.0]), "norm gate number": lambda: norm(x, cuda(64), gate=2.0),
        "norm residual list": lambda: norm(x, cuda(64), residual=[0.0]),
        "norm residual_out": lambda: norm(x, cuda(64), residual=x, residual_out=1),
        "sample logits number": lambda: sample(cuda()[()], cuda()), "sample noise list": lambda: sample(x, [1.0]),
        "sample top_k list": lambda: sample(x, x, top_k=[1]), "sample temperature none": lambda: sample(x, x, temperature=None),
        "sample token list": lambda: sample(x, x, token=[0]),
        "prefill workspace": lambda: gdn.gdn_chunk_prefill(v, v, v, g, g, cuda(2, 2, 64, 64), workspace=4096),
        "replay workspace": lambda: gdn.gdn_chunk_replay(v, v, g, cuda(2, 2, 64, 64), accepted=1, workspace=[0]),
    }
    return calls


@pytest.mark.parametrize("name", list(_wrong_arguments()))
def test_wrong_arguments_are_type_or_value_errors(lib, name):
    with pytest.raises((TypeError, ValueError)):
        _wrong_arguments()[name]()
    assert not lib.calls

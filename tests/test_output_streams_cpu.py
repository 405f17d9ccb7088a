"""Where the binding's outputs come from when a call names a stream: memory of
that stream, which the current one may go on to use.  On the CPU, with the
library and PyTorch's streams replaced by stand-ins; the device's side is in
test_output_streams_gpu.py."""
from __future__ import annotations

import contextlib

import pytest
import torch

import nvfp4_activation_amd as nv
from nvfp4_activation_amd import paged_kv


class Dev(torch.Tensor):
    """A host tensor that passes for a device tensor."""
    is_cuda = True


class Stream:
    cuda_stream = 4711


class Library:
    """Accepts every call; a workspace takes 64 bytes."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith(("_workspace", "_bytes")) else 0


def dev(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Dev)


@pytest.fixture
def allocations(monkeypatch):
    """(stream, tensor) of each torch.empty, and the tensors that the current
    stream was recorded on."""
    made, recorded, on, empty = [], [], [None], torch.empty

    @contextlib.contextmanager
    def stream_context(stream):
        on.append(stream)
        yield
        on.pop()

    def recording_empty(*args, **kwargs):
        t = empty(*args, **{**kwargs, "device": "cpu"}).as_subclass(Dev)
        made.append((on[-1], t))
        return t

    monkeypatch.setattr(torch, "empty", recording_empty)
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    for module in (nv, paged_kv):
        monkeypatch.setattr(module, "lib", Library())
    return made, recorded


def kv_plan(**kw):
    return nv.kv_plan(*(dev(2, dtype=torch.int32) for _ in range(2)), dev(2, 3, dtype=torch.int32),
                      dev(9, dtype=torch.int32), dev(1, dtype=torch.int32), 16, 5, **kw)


def kv_attention(**kw):
    cache = dev(4, 2, 16 * 64 * 9 // 8, dtype=torch.uint8)
    return nv.kv_attention(dev(3, 4, 64), cache, dev(2), dev(1, 3, dtype=torch.int32), dev(2, dtype=torch.int32),
                           dev(1, dtype=torch.int32), **kw)


def named(name, *args):
    def call(**kw):
        return getattr(nv, name)(*args, **kw)
    call.__name__ = name
    return call


class Event:
    cuda_event = 1


u8 = torch.uint8
CALLS = [kv_plan, kv_attention] + [
    named(name, dev(4, 64)) for name in ("rotamax", "rotquant", "rotquant_swizzled", "rotate16", "mx_rotquant",
                                         "stream_calibrate", "stream_calibrate_single")
] + [
    named("quant_from_amax", dev(4, 64), dev(1)),
    named("rotquant_timed", dev(4, 64), [Event(), Event()]),
    named("rotate_matrix", dev(4, 64), dev(16, 16)),
    named("dequant", dev(4, 32, dtype=u8), dev(4, 4, dtype=u8), dev(1)),
    named("dequant_swizzled", dev(4, 32, dtype=u8), dev(512, dtype=u8), dev(1)),
    named("mx_dequant", dev(4, 32, dtype=u8), dev(4, 2, dtype=u8)),
]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_outputs_come_from_the_calls_stream(allocations, call):
    made, recorded = allocations
    stream = Stream()
    result = call(stream=stream)
    assert made and all(on is stream for on, _ in made), "memory of another stream"
    # what the caller gets is recorded on the current stream
    bases = {t.untyped_storage().data_ptr() for t in (result if isinstance(result, tuple) else (result,))
             if isinstance(t, torch.Tensor)}
    assert {(b, "current") for b in bases} <= set(recorded)


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_nothing_is_recorded_on_the_current_stream_alone(allocations, call, monkeypatch):
    made, recorded = allocations
    monkeypatch.setattr(nv, "_stream", lambda device, stream=None: 0)
    monkeypatch.setattr(paged_kv, "_stream", lambda device, stream=None: 0)
    call()
    assert made and all(on is None for on, _ in made) and not recorded


def test_a_backward_pass_through_the_attention_is_refused(allocations):
    q = dev(3, 4, 64).requires_grad_()
    cache = dev(4, 2, 16 * 64 * 9 // 8, dtype=torch.uint8)
    rest = (cache, dev(2), dev(1, 3, dtype=torch.int32), dev(2, dtype=torch.int32), dev(1, dtype=torch.int32))
    got = nv.kv_attention(q, *rest, stream=Stream())
    assert got.requires_grad
    with pytest.raises(RuntimeError, match="no backward pass"):
        got.sum().backward()
    with torch.no_grad():
        assert not nv.kv_attention(q, *rest, stream=Stream()).requires_grad

"""Outputs that the binding allocates for a call on a named stream are that
stream's memory, and stay untouched while the current stream still uses them."""
from __future__ import annotations

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def nv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import nvfp4_activation_amd as nv
    return nv


def stream_of(t):
    """The stream whose memory holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def kv_plan(nv, stream=None):
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    return nv.kv_plan(i32([0, 17]), i32([3, 1]), table, i32(list(range(9))), i32([0]), 16, 5, stream=stream)


def kv_attention(nv, stream=None, tokens=3):
    cache = nv.kv_cache(4, 2, 64, 16)
    q = torch.ones(tokens, 4, 64, device=DEV)
    args = cache, torch.ones(2, device=DEV), i32([[0, 1, 2]]), i32([0, tokens]), i32([tokens])
    torch.cuda.synchronize()
    return nv.kv_attention(q, *args, stream=stream)


def rows():
    x = torch.randn(64, 256, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    torch.cuda.synchronize()
    return x


def named(name, make):
    def call(nv, **kw):
        args = make(nv)
        torch.cuda.synchronize()
        return getattr(nv, name)(*args, **kw)
    call.__name__ = name
    return call


CALLS = [kv_plan, kv_attention] + [
    named(name, lambda nv: (rows(),)) for name in ("rotamax", "rotquant", "rotquant_swizzled", "rotate16",
                                                   "mx_rotquant")
] + [
    named("quant_from_amax", lambda nv: (rows(), nv.rotamax(rows()))),
    named("rotate_matrix", lambda nv: (rows(), torch.eye(16, device=DEV))),
    named("dequant", lambda nv: nv.rotquant(rows())[:3]),
    named("dequant_swizzled", lambda nv: nv.rotquant_swizzled(rows())[:3]),
    named("mx_dequant", lambda nv: nv.mx_rotquant(rows())),
]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_outputs_are_the_streams_memory(nv, call):
    say(call.__name__)
    want = call(nv)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(nv, stream=stream)
    torch.cuda.synchronize()
    got, want = ([t for t in (r if isinstance(r, tuple) else (r,)) if isinstance(t, torch.Tensor)]
                 for r in (got, want))
    for g, w in zip(got, want):
        assert torch.equal(g, w)
        assert stream_of(g) == stream.cuda_stream and stream_of(w) != stream.cuda_stream


def test_memory_in_use_on_the_current_stream_stays(nv):
    """An output dropped while the current stream still reads it is not handed
    out again on its own stream until that is done."""
    say("reuse")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = kv_attention(nv, stream=stream, tokens=48)
    at, shape = out.data_ptr(), out.shape
    torch.cuda.current_stream().wait_stream(stream)
    busy = torch.randn(8192, 8192, device=DEV)
    torch.cuda.synchronize()
    for _ in range(10):  # some 70 ms of work ahead of the read
        busy2 = busy @ busy
    seen = out + busy2[0, 0] * 0
    del out
    with torch.cuda.stream(stream):
        other = torch.empty(shape, device=DEV)
    if not torch.cuda.current_stream().query():  # not done when the memory was asked for
        assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(seen, kv_attention(nv, tokens=48))

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


def test_captured_calls_on_a_forked_stream(nv):
    """A step captured with its calls on a stream that forks off and joins, the
    outputs allocated by the calls; replayed with eager work between."""
    say("capture")
    gen = torch.Generator().manual_seed(9)
    cache = nv.kv_cache(8, 2, 64, 16)
    amax, table = torch.full((2,), 4.0, device=DEV), torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    free, head = i32(list(range(8))), i32([0])
    cached, added = i32([0, 0]), i32([20, 3])
    q, k, v = (torch.randn(32, h, 64, generator=gen).to(DEV) for h in (4, 2, 2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def step(stream):
        p = nv.kv_plan(cached, added, table, free, head, 16, 32, stream=stream)
        nv.kv_append(k, v, p.slots, cache, amax, stream=stream)
        codes = nv.rotquant(q.view(32, 256), stream=stream)
        return nv.kv_attention(q, cache, amax, table, p.cu_q, p.kv_lens, max_kv=1 << 20, stream=stream), p, codes

    want, plan, codes = step(None)
    torch.cuda.synchronize()
    want = want[:23].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out, p, c = step(side)
        dropped = step(side)[0]  # one whose memory is free again before the end
        del dropped
        torch.cuda.current_stream().wait_stream(side)
    for rep in range(4):
        say("replay", rep)
        cache.zero_()
        table.fill_(-1)
        out.fill_(7.0)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        eager = step(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(out[:23], want) and torch.equal(eager[0][:23], want)
        assert torch.equal(p.slots, plan.slots) and all(torch.equal(a, b) for a, b in zip(c, codes))

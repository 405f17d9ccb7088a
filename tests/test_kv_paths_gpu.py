"""kv_attention's kernels, each in every form that it is compiled in: types,
head dimensions, pages of 16 tokens and larger ones, units whole and shared,
against the 64-bit model at the masks, pages and magnitudes where they can go
wrong.  The environment and the estimates send a call to its kernel whatever
the rules for the launch are; whether keys are split is checked by the
workspace."""
from __future__ import annotations

import functools

import numpy as np
import pytest
import torch

import kv_model
from kv_tight_model import Attention, TiledScene
from test_kv_gpu import DEV, DT, Scene, check, nv, say  # noqa: F401

pytestmark = pytest.mark.gpu

FEW, ROWS, TILES = "NVFP4RQ_KV_FEW_ROWS", "NVFP4RQ_KV_ROWS_WGS", "NVFP4RQ_KV_TILE_WGS"
# name: environment, estimates (max_q, max_kv), keys split
PATHS = {
    "rows 16": ({FEW: 100000}, (1, 32), False),
    "rows 32": ({FEW: 100000}, (60, 32), False),
    "rows 16 in 7": ({FEW: 100000, ROWS: 7}, (1, 32), True),
    "rows 32 in 7": ({FEW: 100000, ROWS: 7}, (60, 32), True),
    "rows 16 in 1000": ({FEW: 100000, ROWS: 1000}, (1, 32), True),
    "rows 32 in 1000": ({FEW: 100000, ROWS: 1000}, (60, 32), True),
    "tiles": ({FEW: 1}, (60, 0), False),
    "tiles in 5": ({FEW: 1, TILES: 5}, (60, 0), True),
    "tiles in 900": ({FEW: 1, TILES: 900}, (60, 0), True),
}


@pytest.fixture(params=PATHS)
def path(request, monkeypatch):
    env, estimates, split = PATHS[request.param]
    for name, value in env.items():
        monkeypatch.setenv(name, str(value))
    return request.param, dict(zip(("max_q", "max_kv"), estimates)), split


# ---------------------------------------------------------------- scenes: (scene, arguments, rows to compare)

def causal(dtype, d, page):
    return Scene(81, [3, 1, 0, 20], [60, 700, 40, 130], 6, 2, d, page, dtype=dtype), {}, slice(None)


def window(dtype, d, page):
    return Scene(82, [3, 1, 0, 40], [60, 700, 40, 130], 6, 2, d, page, dtype=dtype), dict(window=45), slice(None)


def not_causal_not_rotated(dtype, d, page):
    s = Scene(83, [5, 40, 1], [50, 0, 333], 6, 2, d, page, dtype=dtype, rotate=False)
    return s, dict(causal=False, scale=0.2), slice(None)


def not_causal(dtype, d, page):
    return Scene(84, [5, 20, 1], [50, 300, 3], 2, 1, d, page, dtype=dtype), dict(causal=False), slice(None)


def without_keys(dtype, d, page):
    s = Scene(85, [5, 3, 40, 1], [0, 0, 0, 0], 6, 2, d, page, dtype=dtype)
    s.lens[:] = [2, 0, 33, -4]
    return s, {}, slice(None)


def without_keys_not_causal(dtype, d, page):
    s, _, rows = without_keys(dtype, d, page)
    return s, dict(causal=False), rows


def missing_pages(dtype, d, page, seen=0):
    s = Scene(86, [30, 1, 1], [20, 400, 90], 6, 2, d, page, dtype=dtype)
    s.table[0, 32 // page] = s.cache.shape[0]  # from key 32 on: seen from position 32 on
    s.table[1, :128 // page] = -1              # dropped, outside a window of 200
    s.table[2, 90 // page] = -(1 << 31)        # the last page
    return s, dict(window=seen), slice(None)


def missing_pages_window(dtype, d, page):
    return missing_pages(dtype, d, page, 200)


def missing_pages_narrow_window(dtype, d, page):
    return missing_pages(dtype, d, page, 16)


def peaked(dtype, d, page):
    return Scene(87, [2, 20], [500, 100], 6, 2, d, page, dtype=dtype, k_gain=20.0), {}, slice(None)


def nan_bytes_in_masked_keys(dtype, d, page):
    s = Scene(88, [24], [10], 6, 2, d, page, dtype=dtype)
    t, blk = 25, np.arange(d // 16)
    for h in range(2):
        p = s.cache[s.table[0, t // page], h]
        p[kv_model.k_scale_at(page, d, t % page, blk)] = 0x7F
        p[kv_model.v_scale_at(page, d, t % page, blk)] = 0x7F
    return s, {}, slice(0, 15)  # the first 15 do not see the key


def magnitudes(dtype, d, page):
    s = Scene(89, [4, 30], [60, 90], 2, 1, d, page, dtype=dtype)
    for i, f in enumerate((1e-30, 1e-8, 0.0, 50.0, 1e-30, 0.0)):
        s.q[i] *= f
    return s, {}, slice(None)


def past_the_table(dtype, d, page):
    s = Scene(90, [1, 20], [40, 33], 2, 1, d, page, dtype=dtype)
    s.lens[0] += page
    return s, {}, slice(None)


SCENES = [causal, window, not_causal_not_rotated, not_causal, without_keys, without_keys_not_causal, missing_pages,
          missing_pages_window, missing_pages_narrow_window, peaked, nan_bytes_in_masked_keys, magnitudes,
          past_the_table]


@functools.lru_cache(maxsize=None)
def case(scene, dtype, d, page):
    s, kw, rows = scene(dtype, d, page)
    want, bound = s.want(**kw)
    return s, kw, rows, want, bound


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_kernel(nv, path, dtype, d, page):  # noqa: F811
    name, estimates, split = path
    for scene in SCENES:
        say(name, dtype, d, page, scene.__name__)
        s, kw, rows, want, bound = case(scene, dtype, d, page)
        args = (s.q.to(DEV), *s.dev())
        need = nv.kv_attention_workspace(*args, **estimates, **kw, rotate=s.rotate)
        assert (need > 0) == split, "another launch than the one meant"
        got = nv.kv_attention(*args, **estimates, **kw, rotate=s.rotate)
        torch.cuda.synchronize()
        check(got[rows], want[rows], bound[rows])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_not_finite_stay_alone(nv, path, dtype, d):  # noqa: F811
    """An infinity or a NaN in a query reaches its own row and no other."""
    name, estimates, _ = path
    say(name, dtype, d)
    s = Scene(91, [4, 30], [60, 90], 2, 1, d, 16, dtype=dtype)
    want, bound = s.want()
    keep = np.ones(want.shape[:2], bool)
    for i, h, e, x in ((1, 0, 3, "inf"), (2, 1, d - 1, "nan"), (9, 0, 17, "-inf"), (33, 1, 0, "nan")):
        s.q[i, h, e] = float(x)
        keep[i, h] = False
    got = nv.kv_attention(s.q.to(DEV), *s.dev(), **estimates)
    torch.cuda.synchronize()
    got = got.cpu()
    assert got[torch.from_numpy(~keep)].isnan().all()
    check(got[torch.from_numpy(keep)], want[keep], bound[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_other_rows(nv, path, dtype):  # noqa: F811
    """Queries out of a wider tensor, outputs head-major; rows in no request
    before, between and after."""
    name, estimates, _ = path
    say(name, dtype)
    s = Scene(92, [9, 1, 20], [30, 700, 0], 4, 2, 64, 16, dtype=dtype, extra_rows=5)
    n = s.q.shape[0]
    wide = torch.zeros(n, 8, 64, dtype=s.q.dtype, device=DEV)
    wide[:, 2:6] = s.q.to(DEV)
    out = torch.full((4, n, 64), 3.0, dtype=s.q.dtype, device=DEV).transpose(0, 1)
    nv.kv_attention(wide[:, 2:6], *s.dev(), out=out, **estimates)
    torch.cuda.synchronize()
    live = int(s.cu[-1])
    want, bound = s.want()
    check(out[:live], want[:live], bound[:live])
    assert (out[live:] == 3.0).all()
    # the first request's rows begin later
    cache, amax, table, cu, lens = s.dev()
    cu[0] += 4
    out.fill_(3.0)
    nv.kv_attention(wide[:, 2:6], cache, amax, table, cu, lens, out=out, **estimates)
    torch.cuda.synchronize()
    s.cu[0] += 4
    want, bound = s.want()
    check(out[4:live], want[4:live], bound[4:live])
    assert (out[:4] == 3.0).all() and (out[live:] == 3.0).all()


# ---------------------------------------------------------------- every key once

LONG = [
    # new, cached, q_heads, kv_heads, d, page, window
    ([1], [3007], 8, 2, 128, 16, 0),
    ([2, 1], [2500, 1100], 8, 1, 128, 32, 0),
    ([1, 3], [2100, 900], 4, 2, 64, 16, 0),
    ([1], [2300], 2, 1, 256, 16, 0),
    ([40], [1800], 4, 2, 64, 64, 0),
    ([90], [1500], 2, 1, 128, 16, 0),
    ([33, 1], [1300, 2000], 2, 1, 256, 32, 0),
    ([2, 60], [3000, 2000], 2, 1, 128, 16, 1200),
]


def whole_tiles(a):
    """The tiles of 32 keys that every row with keys sees in full."""
    live = a.seen[a.seen.any(1)]
    return [lo for lo in range(0, a.seen.shape[1] - 31, 32) if live[:, lo:lo + 32].all()]


@functools.lru_cache(maxsize=None)
def long_case(i):
    *shape, win = LONG[i]
    s = TiledScene(93 + i, *shape)
    parts = [Attention(s, r, window=win) for r in range(len(shape[0]))]
    for a in parts:
        tiles = whole_tiles(a)
        assert len(tiles) >= 20
        # a tile left out or taken twice is past the bounds
        assert min(a.worst_without(lo, lo + 32) for lo in tiles[::7] + tiles[-2:]) > 2
        assert min(a.worst_without(lo, lo + 32, 2) for lo in tiles[::11] + tiles[-2:]) > 2
    results = [a.result() for a in parts]
    return s, win, np.concatenate([r[0] for r in results]), np.concatenate([r[1] for r in results])


@pytest.mark.parametrize("i", range(len(LONG)), ids=lambda i: "-".join(map(str, LONG[i])).replace(" ", ""))
def test_every_key_once(nv, path, i):  # noqa: F811
    name, estimates, _ = path
    say(name, LONG[i])
    s, win, want, bound = long_case(i)
    got = nv.kv_attention(s.q.to(DEV), *s.dev(), window=win, **estimates)
    torch.cuda.synchronize()
    check(got, want, bound)


@pytest.mark.parametrize("i", range(len(LONG)), ids=lambda i: "-".join(map(str, LONG[i])).replace(" ", ""))
def test_every_key_once_as_launched(nv, monkeypatch, i):  # noqa: F811
    """As the rules launch them, without estimates, with the right ones and
    with ones that split everything; and by any number of ranges."""
    s, win, want, bound = long_case(i)
    args = (s.q.to(DEV), *s.dev())
    new, keys = max(LONG[i][0]), int(s.lens.max())
    for estimates in ({}, dict(max_q=new, max_kv=keys), dict(max_q=new, max_kv=1 << 20), dict(max_q=1, max_kv=1)):
        say(LONG[i], estimates)
        got = nv.kv_attention(*args, window=win, **estimates)
        torch.cuda.synchronize()
        check(got, want, bound)
    for wgs in (2, 3, 13, 64, 257):
        say(LONG[i], wgs)
        monkeypatch.setenv(ROWS, str(wgs))
        monkeypatch.setenv(TILES, str(wgs))
        got = nv.kv_attention(*args, window=win)
        torch.cuda.synchronize()
        check(got, want, bound)


# ---------------------------------------------------------------- calls beside each other

SPLIT = [p for p in PATHS if PATHS[p][2]]


def split_scenes(dtype="bf16"):
    return [Scene(95 + i, new, cached, 8, 2, 128, 16, dtype=dtype)
            for i, (new, cached) in enumerate((([1, 20], [1500, 700]), ([30, 2], [300, 900])))]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", SPLIT)
def test_equal_calls_of_shared_units_give_equal_bits(nv, monkeypatch, name, dtype):  # noqa: F811
    env, (max_q, max_kv), _ = PATHS[name]
    for k, v in env.items():
        monkeypatch.setenv(k, str(v))
    for s in split_scenes(dtype):
        args = (s.q.to(DEV), *s.dev(), max_q, max_kv)
        assert nv.kv_attention_workspace(*args) > 0
        first = nv.kv_attention(*args)
        for _ in range(10):
            again = nv.kv_attention(*args)
            torch.cuda.synchronize()
            assert torch.equal(first, again)
        check(first, *s.want())


@pytest.mark.parametrize("name", SPLIT)
def test_shared_units_on_two_streams(nv, monkeypatch, name):  # noqa: F811
    """Calls with workspaces of their own overlap on two streams."""
    env, (max_q, max_kv), _ = PATHS[name]
    for k, v in env.items():
        monkeypatch.setenv(k, str(v))
    scenes = split_scenes()
    args = [(s.q.to(DEV), *s.dev(), max_q, max_kv) for s in scenes]
    assert all(nv.kv_attention_workspace(*a) > 0 for a in args)
    streams = [torch.cuda.Stream() for _ in scenes]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for a, st in zip(args, streams):
            outs.append(nv.kv_attention(*a, stream=st))
    torch.cuda.synchronize()
    wants = [s.want() for s in scenes]
    for i, got in enumerate(outs):
        check(got, *wants[i % 2])


@pytest.mark.parametrize("name", SPLIT)
def test_graphs_of_shared_units_on_one_workspace(nv, monkeypatch, name):  # noqa: F811
    """Two captured calls that share a workspace, replayed in turn on one
    stream, with an eager call on it between them."""
    env, (max_q, max_kv), _ = PATHS[name]
    for k, v in env.items():
        monkeypatch.setenv(k, str(v))
    scenes = split_scenes()
    args = [(s.q.to(DEV), *s.dev(), max_q, max_kv) for s in scenes]
    needs = [nv.kv_attention_workspace(*a) for a in args]
    assert min(needs) > 0
    work = torch.empty(max(needs), dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(a[0]) for a in args]
    graphs = []
    for a, out in zip(args, outs):
        nv.kv_attention(*a, out=out, workspace=work)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv.kv_attention(*a, out=out, workspace=work)
        graphs.append(graph)
    wants = [s.want() for s in scenes]
    for rep in range(4):
        say(name, "replay", rep)
        work.fill_(0xFF)
        for out in outs:
            out.fill_(3.0)
        for graph in graphs:
            graph.replay()
        eager = nv.kv_attention(*args[rep % 2], workspace=work)
        graphs[0].replay()
        torch.cuda.synchronize()
        for out, want in zip(outs, wants):
            check(out, *want)
        check(eager, *wants[rep % 2])


def test_plan_of_more_slots_than_threads(nv):  # noqa: F811
    """More token slots than the launch has threads: each takes several."""
    rng = np.random.default_rng(7)
    n, page, width = 300, 16, 200
    added = rng.integers(900, 1500, n)
    cached = rng.integers(0, 500, n)
    pool = rng.permutation(n * width).astype(np.int32)
    table, at = np.full((n, width), -1, np.int32), 0
    for r in range(n):
        have = -(-int(cached[r]) // page)
        table[r, :have] = pool[at:at + have]
        at += have
    free = pool[at:at + 25000]
    tokens = int(added.sum()) + 1000
    threads = 2 * torch.cuda.get_device_properties(0).multi_processor_count * 512
    assert tokens > threads
    say("plan", tokens, "slots", threads, "threads")
    t = torch.from_numpy(table.copy()).to(DEV)
    p = nv.kv_plan(*(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (cached, added)), t,
                   torch.from_numpy(free).to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV), page, tokens)
    torch.cuda.synchronize()
    slots, cu, lens, head, missing, want = kv_model.plan(cached, added, table, free, 0, page, tokens)
    assert np.array_equal(p.slots.cpu().numpy(), np.array(slots))
    assert p.cu_q.tolist() == cu and p.kv_lens.tolist() == lens
    assert p.head.tolist() == [head] and p.missing.tolist() == missing
    assert np.array_equal(t.cpu().numpy(), want)

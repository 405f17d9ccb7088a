"""kv_attention where lengths and counts are large: lengths past what the block
table has room for, hundreds of millions of keys, many requests in ranges."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_model
from test_kv_gpu import DEV, Scene, check, i32, nv, say  # noqa: F401
from test_kv_paths_gpu import FEW, PATHS, ROWS, TILES, path  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_far_past_the_table(nv, path, dtype, d):  # noqa: F811
    """NaN for the queries that see a key past the table's row, at no cost in
    time; the other requests, and queries before such keys, as ever."""
    name, estimates, _ = path
    for kw in ({}, dict(causal=False), dict(window=20)):
        s = Scene(101, [2, 3, 1, 30], [40, 7, 90, 60], 6, 2, d, 16, dtype=dtype)
        want, bound = s.want(**kw)
        for length in (16 * s.table.shape[1] + 1, 1 << 24, (1 << 31) - (1 << 16), (1 << 31) - 1):
            say(name, dtype, d, kw, length)
            s.lens[1] = length
            got = nv.kv_attention(s.q.to(DEV), *s.dev(), **estimates, **kw)
            torch.cuda.synchronize()
            assert got[4].isnan().all()  # the last query of the request
            if length > 16 * s.table.shape[1] + 40 or kw == dict(causal=False):
                assert got[2:5].isnan().all()
            keep = [0, 1, *range(5, 36)]
            check(got[keep], want[keep], bound[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_before_the_tables_end(nv, path, dtype):  # noqa: F811
    """Of one request's queries those whose keys are all in the table have
    their values, the later ones are NaN; with a window, those that see none in
    it, too."""
    name, estimates, _ = path
    for w in (0, 1, 5, 64):
        say(name, dtype, w)
        s = Scene(102, [40, 2], [100, 30], 6, 2, 64, 16, dtype=dtype)
        s.table = s.table[:, :8].copy()  # keys 0 .. 127 of 140
        want, bound = s.want(window=w)
        assert np.isnan(want[28:40]).all() and not np.isnan(want[:28]).any()
        got = nv.kv_attention(s.q.to(DEV), *s.dev(), **estimates, window=w)
        torch.cuda.synchronize()
        check(got, want, bound)
        # no row of the table at all
        cache, amax, table, cu, lens = s.dev()
        got = nv.kv_attention(s.q.to(DEV), cache, amax, table[:, :0].contiguous(), cu, lens, **estimates, window=w)
        torch.cuda.synchronize()
        assert got.isnan().all()


@pytest.mark.parametrize("heads,requests", [(2, 1), (2, 3)])
def test_half_a_billion_keys(nv, heads, requests):  # noqa: F811
    """Tables that name one page of 65536 tokens thousands of times.  Queries of
    0 weigh all keys alike, by a power of two; V's values are halves up to 6, so
    that a lane's sums are exact below 2^24 halves, and the result is their mean
    to the joining's roundings."""
    say("keys", heads, requests)
    page, d, width = 65536, 64, 8192
    rng = np.random.default_rng(5)
    cache = np.zeros((1, heads, kv_model.page_bytes(page, d)), np.uint8)
    half = page * d * 9 // 16
    cache[:, :, half:half + page * d // 2] = rng.integers(0, 256, (heads, page * d // 2), dtype=np.uint8)
    cache[:, :, half + page * d // 2:] = 0x38  # 1.0
    amax = np.array([4.0, 2688.0], np.float32)  # V's global scale is 1
    lens = [page * width - 1000 * r for r in range(requests)]
    table = torch.zeros(requests, width, dtype=torch.int32, device=DEV)
    q = torch.zeros(requests, heads, d, device=DEV)
    got = nv.kv_attention(q, torch.from_numpy(cache).to(DEV), torch.from_numpy(amax).to(DEV), table,
                          i32(list(range(requests + 1))), i32(lens), rotate=False, max_q=1)
    torch.cuda.synchronize()
    got = got.cpu().double().numpy()
    for h in range(heads):
        v = kv_model.decode(cache[0, h], page, d, 1.0, 1)
        for r, n in enumerate(lens):
            full, rest = divmod(n, page)
            mean = (full * v.sum(0) + v[:rest].sum(0)) / n
            # up to 4 waves' and 384 ranges' parts: as many roundings of mean |v|,
            # of the sums and of the weights' sum
            assert (np.abs(got[r, h] - mean) <= 800 * 2.0 ** -24 * np.abs(v).mean(0)).all(), (h, r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 65, 700])
def test_many_requests_in_ranges(nv, monkeypatch, n, dtype):  # noqa: F811
    """As many requests as a wave has lanes, one more, and more than a
    workgroup has threads, dealt out in few and many ranges by both kernels."""
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 9, 33, 90], n)]
    cached = [int(x) for x in rng.choice([0, 1, 15, 31, 64, 200], n)]
    cached[n // 2], new[n // 2] = 1500, 2
    s = Scene(103, new, cached, 2, 1, 64, 16, dtype=dtype)
    want, bound = s.want()
    args = (s.q.to(DEV), *s.dev())
    for env in ({ROWS: 1, TILES: 1}, {ROWS: 7, TILES: 5}, {ROWS: 768, TILES: 256}, {ROWS: 3000, TILES: 900},
                {FEW: 1, TILES: 64}, {FEW: 100000, ROWS: 300}):
        for k in (FEW, ROWS, TILES):
            monkeypatch.delenv(k, raising=False)
        for k, v in env.items():
            monkeypatch.setenv(k, str(v))
        say(n, dtype, env)
        assert nv.kv_attention_workspace(*args, max_q=90) > 0
        got = nv.kv_attention(*args, max_q=90)
        torch.cuda.synchronize()
        check(got, want, bound)

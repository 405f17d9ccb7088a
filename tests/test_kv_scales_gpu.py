"""kv_attention where the cache's maxima, the queries and the logits' scale are
far from 1: powers of two go through every kernel exactly, so that the results
are those of the ordinary magnitudes, times a power of two, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import kv_model
import oracle
from test_kv_gpu import DEV, Scene, check, nv, say  # noqa: F401

pytestmark = pytest.mark.gpu

# kernel: the environment that sends a call there
PATHS = {
    "rows": {},
    "rows in ranges": {"NVFP4RQ_KV_ROWS_WGS": 7},
    "rows in many ranges": {"NVFP4RQ_KV_ROWS_WGS": 1000},
    "tiles": {"NVFP4RQ_KV_FEW_ROWS": 1},
    "tiles in ranges": {"NVFP4RQ_KV_FEW_ROWS": 1, "NVFP4RQ_KV_TILE_WGS": 5},
}


def scene(dtype, d, seed=61):
    return Scene(seed, [2, 20], [700, 150], 4, 2, d, 32, dtype=dtype)


def run(nv, s, q, amax, scale, rotate=True):
    cache, _, *rest = s.dev()
    got = nv.kv_attention(q.to(DEV), cache, torch.from_numpy(amax).to(DEV), *rest, scale=scale, rotate=rotate)
    torch.cuda.synchronize()
    return got.float().cpu()


@pytest.fixture(params=PATHS)
def path(request, monkeypatch):
    for name, value in PATHS[request.param].items():
        monkeypatch.setenv(name, str(value))
    return request.param


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_and_large_values(nv, path, dtype, d):  # noqa: F811
    """V's maximum times 2^k: so is the result."""
    say("V", path, dtype, d)
    s = scene(dtype, d)
    base = run(nv, s, s.q, s.amax, None)
    for k in (-100, -60, 60, 110):
        got = run(nv, s, s.q, (s.amax * np.float32([1, 2.0 ** k])).astype(np.float32), None)
        want = base.double() * 2.0 ** k
        normal = want.abs() >= 2.0 ** -126
        assert normal.float().mean() > 0.99
        assert torch.equal(got.double()[normal], want[normal]), k


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_keys_and_scales(nv, path, dtype, d):  # noqa: F811
    """K's maximum, the queries and the scale times powers of two that cancel:
    the same bits."""
    say("K", path, dtype, d)
    s = scene(dtype, d)
    base = run(nv, s, s.q, s.amax, 0.09)
    for kq, ka, ks in ((120, -116, -4), (-116, 0, 116), (100, 0, -100), (-60, -60, 120), (0, 110, -110),
                       (30, 90, -120)):
        q = (s.q.double() * 2.0 ** kq).to(s.q.dtype)
        amax = (s.amax * np.float32([2.0 ** ka, 1])).astype(np.float32)
        got = run(nv, s, q, amax, float(np.float32(0.09)) * 2.0 ** ks)
        assert torch.equal(got, base), (kq, ka, ks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_subnormal_global_scales(nv, path, dtype):  # noqa: F811
    """Global scales below 2^-126, as two binary32 divisions leave them."""
    say("subnormal", path, dtype)
    s = scene(dtype, 128)
    s.amax = np.array([1.3e-36, 0.9e-36], np.float32)
    assert all(0 < float(oracle.global_scale(float(a))) < 2.0 ** -126 for a in s.amax)
    s.q = (s.q.double() * 2.0 ** 120).to(s.q.dtype)  # logits of a few units
    scale = 0.05
    got = run(nv, s, s.q, s.amax, scale)
    want, bound = s.want(scale=scale)
    bound = bound - 1e-37 + 2.0 ** -133  # one step of a subnormal bf16 for the model's allowance near 0
    assert np.median(np.abs(want)) > 1e-38
    check(got, want, bound)


def test_zero_queries_and_large_scales(nv, path):  # noqa: F811
    """Logits of 0 stay 0 whatever factor they have."""
    say("zero", path)
    s = scene("f32", 64)
    s.q.zero_()
    for scale, top in ((0.1, 4.0), (3e38, 4.0), (3e38, 1e38), (1e-45, 4.0)):
        got = run(nv, s, s.q, np.array([top, 9.0], np.float32), scale)
        want, bound = s.want()
        check(got, want, bound)


@pytest.mark.parametrize("amax", [1e-36, 3e-38, 1e-42, 1e38])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_with_extreme_maxima(nv, amax, dtype):  # noqa: F811
    gen = torch.Generator().manual_seed(5)
    k, v = ((torch.randn(40, 2, 128, generator=gen) * min(1.0, amax)).to(torch.bfloat16 if dtype == "bf16" else
                                                                        torch.float32) for _ in range(2))
    a = torch.tensor([amax, amax])
    cache = nv.kv_cache(3, 2, 128, 16)
    nv.kv_append(k.to(DEV), v.to(DEV), torch.arange(40, device=DEV), cache, a.to(DEV))
    torch.cuda.synchronize()
    want = np.zeros((3, 2, kv_model.page_bytes(16, 128)), np.uint8)
    kv_model.append(k, v, list(range(40)), want, a, 16)
    assert np.array_equal(cache.cpu().numpy(), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_maxima_that_are_not_finite_show(nv, path, dtype, bad):  # noqa: F811
    """A maximum that is no number leaves no ordinary results."""
    say("not finite", path, dtype, bad)
    s = scene(dtype, 128)
    assert run(nv, s, s.q, np.array([bad, 9.0], np.float32), None).isnan().all()
    assert not run(nv, s, s.q, np.array([4.0, bad], np.float32), None).isfinite().any()

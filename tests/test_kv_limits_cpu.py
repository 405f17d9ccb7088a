"""The K/V cache's entry points at the ends of their arguments' ranges, on the
CPU."""
from __future__ import annotations

import ctypes
import itertools
import os

import pytest

from test_kv_cpu import batch, cache, lib
from test_kv_host_cpu import CSRC, FLAGS, HELPERS, INC, ROCM, hipcc, run

needs_hipcc = pytest.mark.skipif(not os.path.exists(os.path.join(ROCM, "bin", "hipcc")), reason="hipcc not installed")


@needs_hipcc
def test_extremes_under_asan_ubsan(tmp_path):
    """No overflow on the way through the checks, and no buffer whose size
    wraps round."""
    clang = os.path.join(ROCM, "llvm", "bin", "clang")
    lib_o, drv_o, exe = tmp_path / "kv_san.o", tmp_path / "extremes.o", tmp_path / "san_kv"
    host_san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    r = run([hipcc(), *FLAGS, "-O1", "-g", "-fPIC", *host_san, "-c", os.path.join(CSRC, "kv", "kv.hip"), "-o", lib_o])
    assert r.returncode == 0, r.stdout + r.stderr
    r = run([clang, "-std=c11", "-O1", "-g", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{INC}", "-c",
             os.path.join(HELPERS, "sanitize_kv_extremes.c"), "-o", drv_o])
    assert r.returncode == 0, r.stdout + r.stderr
    r = run([clang + "++", "-fsanitize=address,undefined", drv_o, lib_o, f"-L{ROCM}/lib", "-lamdhip64",
             f"-Wl,-rpath,{ROCM}/lib", "-o", exe])
    assert r.returncode == 0, r.stdout + r.stderr
    env = {**os.environ, "ASAN_OPTIONS": "detect_leaks=1:halt_on_error=1",
           "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1", "HIP_VISIBLE_DEVICES": "-1"}
    r = run([exe], env=env, timeout=300)
    if r.returncode == 3:
        pytest.skip("a GPU is visible; the driver only runs without one")
    assert r.returncode == 0, r.stdout + r.stderr
    assert "clean" in r.stdout


def test_most_rows():
    """Row numbers are 32-bit and counted in steps of a unit, also past the
    last one: tokens * query heads is at most 2^31 - 2^16, whatever the
    estimates."""
    top = (1 << 31) - (1 << 16)
    for heads, d, max_q in itertools.product((1, 8, 24, 128), (64, 128, 256), (0, 1)):
        def need(tokens):
            return lib.nvfp4_kv_attention_workspace(
                tokens, heads, ctypes.byref(cache(kv_heads=1, head_dim=d)), ctypes.byref(batch(requests=1, max_q=max_q)))

        assert need(top // heads) >= 0
        assert need(top // heads + 1) == -1
        assert need(((1 << 31) - 1) // heads) == -1


@pytest.mark.skipif(not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                    reason="the HIP headers are not installed")
def test_division_by_launch_constants(tmp_path):
    """FastDiv's own code, compiled for the host: quotients around multiples of
    some 470,000 divisors."""
    exe = tmp_path / "kv_fastdiv"
    r = run(["g++", "-std=c++17", "-O2", "-Wall", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{INC}",
             f"-I{CSRC}", os.path.join(HELPERS, "kv_fastdiv.cpp"), "-o", exe])
    assert r.returncode == 0, r.stdout + r.stderr
    r = run([exe], timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split()[0]) > 10 ** 7

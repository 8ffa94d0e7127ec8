"""The int8 products' workspaces, without a GPU (tests/dispatch_workspace_driver.cpp)."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from gram_memory_layer_engram_amd import build, engram
from tests._dispatch import PKG, ROOT, Dispatch

OK, INV = 0, 1


@pytest.fixture(scope="module")
def dispatch(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("no host C++ compiler or HIP headers")
    if not os.path.exists(engram.LIB_PATH):
        build.build()
    exe = str(tmp_path_factory.mktemp("workspace") / "driver")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-rdynamic",
                    os.path.join(ROOT, "tests", "dispatch_workspace_driver.cpp"), "-o", exe, engram.LIB_PATH,
                    f"-Wl,-rpath,{PKG}", "-Wl,--allow-shlib-undefined", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
    return Dispatch(exe)


@pytest.mark.parametrize("T,K,N", [(1, 2048, 20480), (8, 64, 32), (16, 512, 4096)])
def test_a_workspace_that_is_not_used_may_lie_anywhere(dispatch, T, K, N):
    """Where none is needed the pointer is not looked at: inside x, the weight, its
    scales or kv, aligned or not, of any size."""
    lines = [f"wkvat {T} {K} {N} {p} {ofs} {size}" for p in (0, 2, 3, 4) for ofs in (0, 1, 16) for size in (0, 100, 1 << 30)]
    for line, (status, launches) in zip(lines, dispatch.calls(lines)):
        assert status == OK and len(launches) == 1, line


def test_a_workspace_that_is_used_may_not(dispatch):
    T, K, N = 20, 64, 32
    need = 1280 + 256
    lines = [f"wkvat {T} {K} {N} {p} {ofs} {need}" for p in (0, 2, 3, 4) for ofs in (0, -256)]
    assert [s for s, _ in dispatch.calls(lines)] == [INV] * 8
    assert dispatch.calls([f"wkvat {T} {K} {N} 5 0 {need}"])[0][0] == OK


def test_the_forward_keeps_no_staged_rows_on_int8_weights(dispatch):
    """Its gather writes int8 codes: codes and scales and kv are all it keeps, beside
    the 64 KiB of flags."""
    for T, hc, dim, c, hd in ((1, 4, 4096, 16, 128), (300, 2, 512, 8, 64), (1000, 4, 4096, 16, 128)):
        K, N = c * hd, (hc + 1) * dim
        pad = lambda b: -(-b // 256) * 256   # noqa: E731
        need = 65536 + pad(2 * T * N) + pad(T * K) + pad(4 * T)
        assert dispatch.calls([f"fwdsize {T} {hc} {dim} {c} {hd} 3"])[0][0] == -(-need // 1024)
        # the other formats stage bf16 rows
        assert dispatch.calls([f"fwdsize {T} {hc} {dim} {c} {hd} 2"])[0][0] == -(-(65536 + pad(2 * T * N) + pad(2 * T * K)) // 1024)


def test_noalloc_takes_what_fits_the_scratch(dispatch):
    """32 MiB at hc 4, dim 4096, K 2048: 43012 bytes a token."""
    T = 32 * 2 ** 20 // (2 * 20480 + 2048 + 4) - 1
    assert dispatch.calls([f"noalloc {T} 4 4096 16 128 3"])[0][0] == OK
    assert dispatch.calls([f"noalloc {T + 2} 4 4096 16 128 3"])[0][0] == 4

"""The int8 products' and the norms' around a block argument checks under
AddressSanitizer (CPU only), as tests/test_abi_asan.py does for the other entry
points: the ABI layer's host side is sanitized, its device side built as usual."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from gram_memory_layer_engram_amd import build as BUILD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "gram_memory_layer_engram_amd")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_int8_and_norms_abi_checks_under_asan(tmp_path):
    objs = [os.path.join(PKG, "_build", s.replace(".hip", ".o")) for s in BUILD.SOURCES if s != "abi.hip"]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library's objects are not built (python -m gram_memory_layer_engram_amd.build)")
    if not os.path.exists(HIPCC) or shutil.which("gcc") is None:
        pytest.skip("no hipcc / gcc")
    abi_o, drv_o, exe = (str(tmp_path / n) for n in ("abi.o", "driver.o", "driver"))
    asan = ["-Xarch_host", "-fsanitize=address"]
    for cmd in ([HIPCC, "--offload-arch=gfx950", "-O1", "-fPIC", "-std=c++17", "-g", *asan, "-Wno-unused-result", "-c",
                 os.path.join(PKG, "csrc", "abi.hip"), "-o", abi_o],
                ["gcc", "-std=c11", "-g", "-c", os.path.join(ROOT, "tests", "abi_asan_int8_driver.c"), "-o", drv_o],
                [HIPCC, "--offload-arch=gfx950", *asan, drv_o, abi_o, *objs, "-o", exe]):
        subprocess.run(cmd, check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert " 0 failures" in r.stdout, r.stdout

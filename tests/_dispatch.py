"""tests/dispatch_driver.cpp: what the library launches for a call, on the CPU."""

from __future__ import annotations

import os
import shutil
import subprocess
from typing import NamedTuple

import pytest

from gram_memory_layer_engram_amd import build, engram

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.dirname(engram.LIB_PATH)


class Launch(NamedTuple):
    kernel: str
    grid: tuple
    block: int
    lds: int      # dynamic
    limit: int    # of the kernel's dynamic LDS when it was launched, 0 if never set


class Dispatch:
    def __init__(self, exe):
        self.exe = exe

    def calls(self, lines):
        """One (status, launches) for each line of the driver's input."""
        r = subprocess.run([self.exe], input="".join(f"{line}\n" for line in lines), capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr
        answers = r.stdout.splitlines()
        assert len(answers) == len(lines)
        out = []
        for a in answers:
            _, status, rest = a.split(" ", 2)
            launches = []
            for part in rest.split(";")[:-1]:
                name, *n = part.split()
                gx, gy, gz, block, lds, limit = (int(v) for v in n)
                launches.append(Launch(name, (gx, gy, gz), block, lds, limit))
            out.append((int(status), launches))
        return out

    def kernels(self):
        r = subprocess.run([self.exe], input="kernels\n", capture_output=True, text=True, timeout=60)
        return set(r.stdout.split(" ", 2)[2].strip().split(";")[:-1])


def build_driver(tmp_dir) -> Dispatch:
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("no host C++ compiler or HIP headers")
    if not os.path.exists(engram.LIB_PATH):
        build.build()
    exe = os.path.join(tmp_dir, "dispatch_driver")
    # -rdynamic: the library finds this program's definitions before the runtime's
    subprocess.run([cxx, "-O1", "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-rdynamic",
                    os.path.join(ROOT, "tests", "dispatch_driver.cpp"), "-o", exe, engram.LIB_PATH,
                    f"-Wl,-rpath,{PKG}", "-Wl,--allow-shlib-undefined", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
    return Dispatch(exe)

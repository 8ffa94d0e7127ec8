"""Which kernels the int8 entry points and the norms around a block launch, without a
GPU (tests/dispatch_int8_driver.cpp): every one is reached by a GPU test, grids cover
every row and token, LDS fits."""

from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

from gram_memory_layer_engram_amd import build, engram
from tests import _int8_shapes as S
from tests._dispatch import PKG, ROOT, Dispatch

LDS = 160 * 1024


@pytest.fixture(scope="module")
def dispatch(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime_api.h"):
        pytest.skip("no host C++ compiler or HIP headers")
    if not os.path.exists(engram.LIB_PATH):
        build.build()
    exe = str(tmp_path_factory.mktemp("dispatch") / "driver")
    subprocess.run([cxx, "-O1", "-std=c++17", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-rdynamic",
                    os.path.join(ROOT, "tests", "dispatch_int8_driver.cpp"), "-o", exe, engram.LIB_PATH,
                    f"-Wl,-rpath,{PKG}", "-Wl,--allow-shlib-undefined", "-L/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib"], check=True, capture_output=True)
    return Dispatch(exe)


def _names(launches):
    return [la.kernel for la in launches]


def test_gpu_tests_reach_every_kernel(dispatch):
    from tests import test_gpu_int8_and_block_norm as G

    shapes = [(t, k, n) for t in S.T for k, n in S.KN] + S.SMALL + S.TILES
    lines = [f"i8 {t} {k} {n}" for t, k, n in shapes] + [f"wkv {t} {k} {n} 3" for t, k, n in shapes]
    lines += [f"i8q {t} {k}" for t, k in S.ROWS]
    lines += [f"forward {t} {hc} {dim} {c} {hd} 3 {o}" for t, dim, hc, c, hd in S.FORWARD for o in (0, 1)]
    lines += [f"ppn {t} {hc} {dim} 1" for t, hc, dim in G.SHAPES]
    reached = set()
    for line, (status, launches) in zip(lines, dispatch.calls(lines)):
        assert status == 0, line
        reached.update(_names(launches))
    family = ("gemv_int8", "gemm_int8", "int8_quantize", "post_pre_norm")
    missing = {k for k in dispatch.kernels() if k.startswith(family)} - reached
    # the gather from fp8 tables takes the same shapes as from bf16 ones (the driver's tables are bf16)
    missing = {k for k in missing if not (k.startswith("int8_quantize_kernel<2,") and k.replace("<2,", "<1,") in reached)}
    assert missing == set()


def test_grids_cover_and_lds_fits(dispatch):
    rng = random.Random(3)
    lines = []
    for _ in range(4000):
        T = rng.choice([rng.randint(1, 16), rng.randint(17, 128), rng.randint(129, 6000)])
        K, N = 16 * int(2 ** rng.uniform(0, 12.9)), 4 * int(2 ** rng.uniform(0, 13.5))
        lines.append(f"{rng.choice(['i8', 'wkv'])} {T} {K} {N}" + " 3")
    limits = {}
    for cus in (64, 256, 304):
        for line, (status, launches) in zip(lines, dispatch.calls([f"cus {cus}"] + lines)[1:]):
            assert status == 0, line
            op, T, K, N, _ = line.split()[0], *map(int, line.split()[1:])
            cols = 0
            for la in launches:
                assert la.lds <= LDS and la.lds <= max(la.limit, 65536), (line, la)
                if la.limit:
                    limits.setdefault(la.kernel, set()).add(la.limit)
                args = la.kernel[la.kernel.index("<") + 1:-1].split(",")
                if la.kernel.startswith("gemv_int8"):
                    assert la.grid[0] == -(-N // (16 * int(args[0]))), (line, la)
                    if "slice" in la.kernel:
                        assert 16 * int(args[1]) * la.grid[1] >= T and la.block == 64 * int(args[1]) * int(args[2])
                        assert 16 * int(args[1]) * (la.grid[1] - 1) < T
                    else:
                        assert T <= 16 and la.block == 64 * int(args[1])
                        assert 128 * int(args[1]) * int(args[3]) >= K, (line, la)   # waves x steps
                    cols = N
                elif "mixed" in la.kernel:
                    tt, t1, tn1 = -(-T // 256), -(-T // 128), -(-N // 128)
                    big, rest = divmod(tn1 * t1 - la.grid[0], 2 * t1 - tt)   # columns of 256x256 tiles
                    assert rest == 0 and 1 <= big < -(-N // 256) and -(big * tt) % cus < tt, (line, la)
                    cols = 128 * tn1
                elif la.kernel.startswith("gemm_int8"):
                    t = 128 if "deep" in la.kernel else 64 * int(args[0])
                    assert la.grid[0] % -(-T // t) == 0
                    cols += la.grid[0] // -(-T // t) * t
                else:
                    tpr, bs = int(args[2]), la.block
                    assert la.kernel.startswith("int8_quantize") and 8 * int(args[1]) * tpr >= K
                    assert la.grid[0] * la.grid[1] * (bs // tpr) >= T
            assert cols >= N and cols - N < 256, (line, launches)
    assert {k: v for k, v in limits.items() if len(v) > 1} == {}


def test_bf16_rows_of_a_few_tokens_take_one_launch(dispatch):
    for line, n in (("wkv 8 2048 20480 3", 1), ("wkv 9 2048 20480 3", 2), ("wkv 16 2048 12288 3", 1), ("wkv 17 2048 12288 3", 2),
                    ("wkv 16 4096 4096 3", 1), ("wkv 16 2064 4100 3", 2), ("wkv 8 2064 4100 3", 1),
                    ("wkv 16 512 12292 3", 2), ("wkv 4 4096 28672 3", 2)):
        (status, launches), = dispatch.calls([line])
        assert status == 0 and len(launches) == n, line
        assert launches[0].kernel.startswith("int8_quantize") if n == 2 else launches[0].kernel.endswith("true>"), line


def test_forward_routes(dispatch):
    """The gate's epilogue only where the plain store would take 256x256 tiles as
    well, or kv is past 128 MiB."""
    def route(line):
        (status, launches), = dispatch.calls([line])
        assert status == 0 and len(launches) == 3 and launches[0].kernel.startswith("int8_quantize_kernel<1,")
        return launches[1].kernel, launches[2].kernel.endswith("true>")

    assert route("forward 64 4 4096 16 128 3 0")[0].startswith("gemv_int8_slice") and not route("forward 64 4 4096 16 128 3 0")[1]
    assert route("forward 300 4 4096 16 128 3 0") == ("gemm_int8_kernel<2,false>", False)
    assert route("forward 8192 4 4096 16 128 3 0") == ("gemm_int8_kernel<4,false>", True)
    assert route("forward 8192 4 4096 16 128 3 1") == ("gemm_int8_kernel<4,false>", False)
    for c, hd, tail in ((16, 64, "false"), (9, 112, "true")):      # the epilogue's own GPU test
        assert route(f"forward 1491 4 4096 {c} {hd} 3 0") == (f"gemm_int8_kernel<4,{tail}>", True)


def test_grids_stay_below_what_a_dimension_holds(dispatch):
    """Fewer than 2^32 threads a dimension, up to N 2^28, T 2^30 and 2^31 - 1 rows."""
    lines = [f"i8 {T} {K} {N}" for T in (1, 8, 9, 16, 20, 40, 64, 90, 130) for K in (16, 1040, 2064, 8192, 131056)
             for N in (1 << 24, (1 << 24) + 4, 1 << 27, 1 << 28)]
    lines += [f"i8 {1 << 30} {K} {N}" for K in (16, 2048) for N in (4, 128)]
    lines += [f"i8q {T} {K}" for T in (1 << 20, (1 << 31) - 1) for K in (16, 2048, 8192, 40000)]
    lines += [f"ppn {T} 1 {d} 2" for T in ((1 << 22) + 1, (1 << 31) - 1) for d in (8, 1024, 16384)]
    for line, (status, launches) in zip(lines, dispatch.calls(lines)):
        assert status == 0 and launches, line
        for la in launches:
            assert la.grid[0] * la.block < 1 << 32 and la.grid[1] < 1 << 16, (line, la)

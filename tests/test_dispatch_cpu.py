"""Which kernels the entry points launch, without a GPU (tests/_dispatch.py)."""

from __future__ import annotations

import random

import pytest

from tests._dispatch import build_driver

LDS = 160 * 1024          # of a compute unit
DEFAULT_LIMIT = 64 * 1024


@pytest.fixture(scope="module")
def dispatch(tmp_path_factory):
    return build_driver(str(tmp_path_factory.mktemp("dispatch")))


def _products(n, seed):
    rng = random.Random(seed)
    lines = []
    for _ in range(n):
        T = rng.choice([rng.randint(1, 64), rng.randint(65, 6000)])
        K = 128 * int(2 ** rng.uniform(0, 11))
        N = 4 * int(2 ** rng.uniform(0, 13.5))
        op, f = rng.choice(["wkv", "mx"]), rng.choice([1, 2])
        lines.append(f"{op} {T} {K} {N if f == 2 else (N + 31) // 32 * 32} {f}")
    return lines


def test_a_kernels_lds_limit_does_not_follow_the_call(dispatch):
    """The limit belongs to the kernel: set to a call's own size, another
    thread's call with a smaller K could lower it before the launch."""
    limits = {}
    for status, launches in dispatch.calls(_products(6000, 1)):
        assert status == 0
        for la in launches:
            assert la.lds <= LDS and la.lds <= max(la.limit, DEFAULT_LIMIT), la
            if la.limit:
                limits.setdefault(la.kernel, set()).add(la.limit)
    assert len(limits) > 20
    assert {k: v for k, v in limits.items() if len(v) > 1} == {}


def _shapes(fn, names):
    """The (T, K, N) of a test's own parametrize marks."""
    marks = [m for m in fn.pytestmark if m.name == "parametrize" and m.args[0] == names]
    return marks[0].args[1]


def _names(launches):
    return [la.kernel for la in launches]


def test_many_tiles_run_the_tiles_they_name(dispatch):
    """The GPU tests that say which of their cases run 256x256 tiles, 128x128
    ones or both (template argument 4, 2; the half chunk of k the second)."""
    from tests import test_gpu_norm_and_4bit as G

    for T, K, N in _shapes(G.test_mxfp4_many_tiles, "T,K,N"):
        for op, kernel in (("wkv", "gemm_fp4_bf16_kernel"), ("mx", "gemm_fp4_mx_kernel")):
            (status, launches), = dispatch.calls([f"{op} {T} {K} {N} 2"])
            half = "true" if K % 256 else "false"
            big = T == 515 and K > 1000 or (op == "wkv" and (T, N) == (1500, 20476))
            want = [f"<4,{half},2>"] if big else [f"<2,{half},2>"]
            if K >= 4096:
                want = [f"<4,{half},2>", f"<2,{half},3>"]
            assert status == 0 and _names(launches) == [kernel + w for w in want], (op, T, K, N)
    shapes = _shapes(G.test_wkv_mx_mxfp8_weight_tiles, "T,K,N")
    for i, (T, K, N) in enumerate(shapes):
        (status, launches), = dispatch.calls([f"mx {T} {K} {N} 1"])
        half = "true" if K % 256 else "false"
        tiles = [4, 2] if i == len(shapes) - 1 else [2] if i < 5 else [4]
        assert status == 0 and _names(launches) == [f"gemm_mx_ring_kernel<{t},{half}>" for t in tiles], (T, K, N)


def test_forward_routes(dispatch):
    """MXFP4: the gate epilogue only where 256x256 tiles fill the compute units
    or kv is past 128 MiB; the GEMV up to 64 tokens."""
    def product_and_gate(line):
        (status, launches), = dispatch.calls([line])
        assert status == 0 and len(launches) == 3
        assert launches[0].kernel.startswith("lookup_kernel") and launches[2].kernel.startswith("gate_exact_kernel")
        return launches[1].kernel, launches[2].kernel.endswith("true>")      # the gate from partial sums

    assert product_and_gate("forward 64 4 4096 16 128 2 0") == ("gemv_mxfp4_kernel<false,5,4,8,1,false>", False)
    assert product_and_gate("forward 300 4 4096 16 128 2 0") == ("gemm_fp4_bf16_kernel<2,false,2>", False)
    for C, half in ((8, "false"), (6, "true")):      # the epilogue's own GPU test
        assert product_and_gate(f"forward 1491 4 4096 {C} 64 2 0") == (f"gemm_fp4_bf16_kernel<4,{half},2>", True)
    assert product_and_gate("forward 8192 4 4096 16 128 2 0") == ("gemm_fp4_bf16_kernel<4,false,2>", True)
    assert product_and_gate("forward 8192 4 4096 16 128 2 1") == ("gemm_fp4_bf16_kernel<4,false,2>", False)


@pytest.mark.parametrize("op,T,last", [("mx", 64, 35840), ("mx", 33, 35840), ("mx", 32, 95232), ("mx", 16, 151552),
                                       ("wkv", 64, 180224), ("wkv", 32, 180224), ("wkv", 16, 286720)])
def test_gemv_takes_k_up_to_what_lds_holds(dispatch, op, T, last):
    """A row tile's scale bytes (16 * K/32, up to a KiB more) beside the rings and,
    with MXFP8 x, the token tiles' scale bytes: K 35840 and more. From T 33 on
    MXFP8 x is held to what four token tiles need."""
    for K in (128, 35840, last, last + 128):
        (status, launches), = dispatch.calls([f"{op} {T} {K} 64 2"])
        assert status == 0
        assert launches[0].kernel.startswith("gemv_mxfp4" if K <= last else "gemm_fp4"), K


def test_gpu_tests_reach_every_kernel_of_the_4bit_products(dispatch):
    """Every instantiation in the library has a shape in the GPU tests, on 256
    compute units."""
    from tests import _exact_inputs as X
    from tests import test_gpu_norm_and_4bit as G

    lines = []
    shapes = list(X.LONG_K) + [(T, K, N) for T in X.WIDE_T for K in X.WIDE_K for N in X.WIDE_N]
    shapes += [(T, K, N) for T in _shapes(G.test_mxfp4_products, "T") for K, N in G.KN]
    shapes += list(_shapes(G.test_mxfp4_many_tiles, "T,K,N"))
    for T, K, N in shapes:
        lines += [f"wkv {T} {K} {N} 2", f"mx {T} {K} {N} 2"]
    lines += [f"mx {T} {K} {N} 1" for T, K, N in _shapes(G.test_wkv_mx_mxfp8_weight_tiles, "T,K,N")]
    reached = set()
    for status, launches in dispatch.calls(lines):
        assert status == 0
        reached.update(_names(launches))
    family = ("gemv_mxfp4_kernel", "gemm_fp4_", "gemm_mx_ring_kernel")
    assert {k for k in dispatch.kernels() if k.startswith(family)} - reached == set()


def test_no_product_is_split_or_dropped_by_its_grid(dispatch):
    """Workgroups cover every row of W and every token, on small and large chips."""
    for cus in (64, 256, 304):
        lines = _products(3000, cus)
        answers = dispatch.calls([f"cus {cus}"] + lines)[1:]
        for line, (status, launches) in zip(lines, answers):
            assert status == 0, line
            op, T, K, N, f = line.split()[0], *map(int, line.split()[1:])
            tiles = [la for la in launches if la.kernel.startswith(("gemm_fp4", "gemm_mx_ring"))]
            cols = 0
            for la in tiles:
                t = 64 * int(la.kernel.split("<")[1].split(",")[0].rstrip(">"))
                tt = -(-T // t)
                assert la.grid[0] % tt == 0, (line, la)
                cols += la.grid[0] // tt * t
            if tiles:
                assert cols >= N and cols - N < 256, (line, launches)
            for la in launches:
                if la.kernel.startswith("gemv_mxfp4"):
                    rt = int(la.kernel.split(",")[1])
                    assert la.grid[0] == -(-N // (16 * rt)), (line, la)

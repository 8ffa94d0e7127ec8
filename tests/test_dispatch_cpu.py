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

"""Refusals of the 4-bit entry points at the C ABI that need whole address ranges
(CPU only: answered before any launch)."""

from __future__ import annotations

import os

import pytest

OK, INV = 0, 1
F4 = 2


@pytest.fixture(scope="module")
def lib():
    from gram_memory_layer_engram_amd import build, engram

    if not os.path.exists(engram.LIB_PATH):
        build.build()
    return engram.load_library()


def test_gate_partials_outputs_on_an_operand_or_each_other(lib):
    """MXFP4 weights: other tiles of the launch would read what one has
    written. Sizes in bytes: x 4 * 256 * 2, w 768 * 128, scales 768 * 8, hidden
    4 * 2 * 256 * 2, q and k 2 * 256 * 2, value 4 * 256 * 2, partials 4 * 2 * 8."""
    T, K, hc, dim = 4, 256, 2, 256
    X, W, S, H, Q, KW, V, PA = (i << 24 for i in range(1, 9))

    def call(value, partials, T=T):
        return lib.engram_wkv_gate_partials(X, T, K, W, S, F4, hc, dim, H, Q, KW, value, partials, None, 0, None)

    for base, size in ((X, 2048), (W, 98304), (S, 6144), (H, 4096), (Q, 1024), (KW, 1024)):
        for v in (base, base + size - 16, base - 2048 + 16):
            assert call(v, PA) == INV, hex(v)
        for p in (base, base + size - 8, base - 64 + 8):
            assert call(V, p) == INV, hex(p)
    for p in (V, V + 2048 - 8, V - 64 + 8):
        assert call(V, p) == INV, hex(p)
    assert call(X, V, T=0) == OK

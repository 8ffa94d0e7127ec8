"""Inputs and tolerances of the norm and 4-bit projection tests (no arithmetic
of the operators here: the expected values come from the oracle)."""

from __future__ import annotations

import numpy as np
import torch

F32_U = 2.0 ** -24      # half a step of fp32, relative
BF16_U = 2.0 ** -8      # half a step of bf16, relative to the value


def mxfp4_weight(rng, n, k, lo=118, hi=124):
    """Every e2m1 code, E8M0 bytes around 2^-6: (codes [n, k/2], bytes [n, k/32])."""
    codes = rng.integers(0, 256, size=(n, k // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi, size=(n, k // 32), dtype=np.uint8)
    return codes, scales


def mxfp8_rows(rng, t, k):
    """Finite e4m3 codes of every magnitude, E8M0 bytes around 2^-7."""
    codes = rng.integers(0, 256, size=(t, k), dtype=np.uint8)
    codes = np.where((codes & 0x7F) == 0x7F, codes & 0x80, codes).astype(np.uint8)
    scales = rng.integers(116, 123, size=(t, k // 32), dtype=np.uint8)
    return codes, scales


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale).to(torch.bfloat16)


def product_tolerance(xa, wa, scaled=False):
    """The exact product xa . wa^T and an elementwise bound of its bf16 result
    with fp32 sums: K - 1 fp32 additions, each off by at most one fp32 step of
    the running magnitude (2 * F32_U: the matrix cores may cut instead of
    rounding), then half a bf16 step of the result.

    ``scaled``: MXFP8 activations, on the scaled 8-bit / 4-bit matrix
    instructions. They add the 8 products of a run of 8 consecutive k in a
    window of 14 bits below the run's largest product (measured: of two
    products in one run the smaller vanishes from a ratio of 2^14 on; in
    different runs both count to fp32's last bit), so each of the 7 others
    loses less than 2^-13 of the largest: 7 * 2^-13 * max|x| * max|w| per run
    at most."""
    ref = xa @ wa.T
    acc = 2 * F32_U * xa.shape[1] * (np.abs(xa) @ np.abs(wa).T)
    if scaled:
        runs = [np.abs(a).reshape(a.shape[0], -1, 8).max(axis=2) for a in (xa, wa)]
        acc = acc + 7 * 2.0 ** -13 * (runs[0] @ runs[1].T)
    return ref, acc + BF16_U * (np.abs(ref) + acc) + 2.0 ** -134

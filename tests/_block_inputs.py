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


def product_tolerance(xa, wa):
    """Elementwise bound of bf16(fp32 sums of xa . wa^T) against the exact
    product: K - 1 fp32 additions and the (exact) products' sums, each
    addition off by at most one fp32 step of the running magnitude (2 * F32_U:
    the matrix cores may truncate inside an instruction), then half a bf16
    step of the result, or of the smallest bf16 normal below it."""
    ref = xa @ wa.T
    mass = np.abs(xa) @ np.abs(wa).T
    acc = 2 * F32_U * xa.shape[1] * mass
    return ref, acc + BF16_U * (np.abs(ref) + acc) + 2.0 ** -134

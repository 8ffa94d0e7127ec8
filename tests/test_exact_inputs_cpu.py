"""What the exact product tests can see (CPU only): a reference that lacks one
128-k step, or has one scale byte wrong, is not equal to the whole one."""

from __future__ import annotations

import pytest
import torch

from tests import _exact_inputs as X

# a wide N only repeats what its first rows show
CASES = sorted({(T, K, min(N, 36)) for T, K, N in X.LONG_K} | {(1, 512, 36), (16, 4096, 36)})


@pytest.mark.parametrize("T,K,N", CASES)
def test_a_lost_step_or_a_wrong_scale_byte_shows(T, K, N):
    gen = X.generator(T * 7 + K + N, "cpu")
    w, s = X.mxfp4_weight(N, K, gen)
    wv = X.mxfp4_values(w, s)
    steps = K // 128
    at = {0, steps - 1, steps // 2}
    for waves in (4, 8):       # first and last step of every wave's run
        per = -(-steps // waves)
        at |= {min(v, steps - 1) for i in range(waves) for v in (i * per, i * per + per - 1)}
    for x in (X.bf16_rows(T, K, gen).double(), X.mxfp8_row_values(*X.mxfp8_rows(T, K, gen))):
        whole = X.product(x, wv)
        for i in sorted(at):
            k = slice(128 * i, 128 * i + 128)
            part = (x[:, k] @ wv[:, k].t())
            ref = (x @ wv.t() - part).float().to(torch.bfloat16)
            assert not torch.equal(ref, whole), f"step {i} of {steps}"
            k = slice(128 * i + 96, 128 * i + 128)     # its last block at twice its scale
            ref = (x @ wv.t() + x[:, k] @ wv[:, k].t()).float().to(torch.bfloat16)
            assert not torch.equal(ref, whole), f"scale byte of step {i}"


def test_the_sums_stay_exact():
    for T, K, N in X.LONG_K:
        assert K * 6 * 4 < 2 ** 24 and K * 12 * 8 < 2 ** 24

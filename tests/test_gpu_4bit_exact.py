"""GPU: products on inputs whose sums are exact in fp32 (tests/_exact_inputs.py),
compared for equality: long K, every row tile count of the MXFP4 GEMV, odd scale
rows; and the norm's codes at ties, where they have to be the quantizer's."""

from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from oracle import engram_oracle as o
from tests import _exact_inputs as X
from tests._util import bits, u8

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _E():
    from gram_memory_layer_engram_amd import engram as E
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    E.load_library()
    return E


def _say(msg):
    print(f"[gpu-test] {msg}", flush=True)
    sys.stdout.flush()


def _guarded(T, N):
    """kv [T, N] with 512 elements behind it that a call has to leave alone."""
    guard = torch.full((T * N + 512,), 55, dtype=torch.bfloat16, device=DEV)
    return guard, guard[:T * N].view(T, N)


def _same(kv, ref, guard, what):
    T, N = ref.shape
    bad = kv != ref
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {ref.numel()} differ, first at {bad.nonzero()[0].tolist()}"
    assert bool((guard[T * N:] == 55).all()), what


def _mxfp4_products(E, T, K, N):
    gen = X.generator(T * 7 + K + N, DEV)
    w, s = X.mxfp4_weight(N, K, gen)
    x = X.bf16_rows(T, K, gen)
    xq, xs = X.mxfp8_rows(T, K, gen)
    guard, kv = _guarded(T, N)
    guard8, kv8 = _guarded(T, N)
    E.wkv(x, w, s, kv=kv)
    E.wkv_mx(xq, xs, w, s, kv=kv8)
    wv = X.mxfp4_values(w, s)
    _same(kv, X.product(x.double(), wv), guard, "bf16 x")
    _same(kv8, X.product(X.mxfp8_row_values(xq, xs), wv), guard8, "MXFP8 x")


@pytest.mark.parametrize("T,K,N", X.LONG_K)
def test_mxfp4_long_k_exact(T, K, N):
    _say(f"long K exact {T} {K} {N}")
    _mxfp4_products(_E(), T, K, N)


@pytest.mark.parametrize("N", X.WIDE_N)
@pytest.mark.parametrize("K", X.WIDE_K)
def test_mxfp4_row_tiles_exact(K, N):
    E = _E()
    for T in X.WIDE_T:
        _say(f"row tiles exact {T} {K} {N}")
        _mxfp4_products(E, T, K, N)


@pytest.mark.parametrize("T,K,N", X.ODD_SCALES)
def test_wkv_mx_mxfp8_weights_odd_scale_rows_exact(T, K, N):
    E = _E()
    gen = X.generator(T + N, DEV)
    w, s = X.mxfp8_weight(N, K, gen)
    xq, xs = X.mxfp8_rows(T, K, gen)
    guard, kv = _guarded(T, N)
    E.wkv_mx(xq, xs, w, s, kv=kv)
    _same(kv, X.product(X.mxfp8_row_values(xq, xs), X.mxfp8_weight_values(w, s)), guard, "MXFP8")


@pytest.mark.parametrize("T", [3, 70])
def test_mxfp8_rows_taken_as_bf16_keep_fp32_sums(T):
    """MXFP8 activations are bf16 values exactly; engram_wkv on them sums products
    that cancel in fp32, where the 8-bit matrix instructions of engram_wkv_mx may
    lose what lies 14 bits below the largest of 8."""
    E = _E()
    K, N = 256, 64
    gen = X.generator(T, DEV)
    codes = torch.zeros((T, K), dtype=torch.uint8, device=DEV)
    codes[:, 0], codes[:, 1], codes[:, 2] = 0x7E, 0xFE, 0x01      # 448, -448, 2^-9 in one run of 8
    scales = torch.randint(120, 134, (T, K // 32), generator=gen, device=DEV, dtype=torch.uint8)
    w = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device=DEV)     # 1.0 everywhere
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    x = X.mxfp8_row_values(codes, scales)
    xb = x.to(torch.bfloat16)
    assert torch.equal(xb.double(), x)
    want = (2.0 ** -9 * torch.exp2(scales[:, :1].double() - 127)).expand(T, N)
    assert torch.equal(E.wkv(xb, w, s).double(), want)


def _tie_rows(rows, dim, seed):
    """bf16 rows with mean square 1 and, beside the elements that make it so,
    blocks 2^20 and more below them: every e4m3 midpoint of a block, the
    saturating edge, subnormal codes and blocks below the least scale byte.
    256 of 1024 elements are +-2 (their squares sum to dim exactly in fp32, in any
    order); the others' squares are below 2^-40, so the sum's nearest fp32 values
    give a root of 1 and y is the row itself."""
    rng = np.random.default_rng(seed)
    x = np.zeros((rows, dim // 32, 32))
    big = np.arange(dim // 32) % 4 == 0
    x[:, big] = 2.0 * (1 - 2 * rng.integers(0, 2, size=(rows, int(big.sum()), 32)))
    for r in range(rows):
        for b in np.flatnonzero(~big):
            e = int(rng.choice([-20, -21, -33, -60, -100, -117, -118, -119, -120, -121, -125]))
            top = rng.integers(128, 256) / 128.0                # 8 significant bits: bf16
            v = np.zeros(32)
            v[0] = top
            # midpoints between neighbouring codes (5 significant bits), at every exponent below the top's
            d = rng.integers(0, 18, size=31)
            odd = 2 * rng.integers(8, 16, size=31) + 1           # 17 .. 31: halfway between two of 8 .. 15
            v[1:] = np.minimum(odd / 16.0, top if top > 1 else 1.0) * 2.0 ** -d
            # subnormal codes' midpoints: odd multiples of half the least step, 2^-10 / 2^8 of the scale
            sub = rng.random(31) < 0.3
            v[1:][sub] = (2 * rng.integers(0, 8, size=int(sub.sum())) + 1) * 2.0 ** -18
            v = v * 2.0 ** e * (1 - 2 * rng.integers(0, 2, size=32))
            x[r, b] = v[rng.permutation(32)]
    t = torch.from_numpy(x.reshape(rows, 1, dim).astype(np.float32)).to(torch.bfloat16)
    return t


@pytest.mark.parametrize("rows,dim", [(3, 1024), (300, 1024), (2, 4096), (270, 2048), (2, 16384), (260, 512), (5, 512)])
def test_norm_codes_at_ties_are_the_quantizers(rows, dim):
    """y is bf16 exactly: codes and scale bytes equal engram_mx_quantize's of
    the row, and the oracle's."""
    E = _E()
    x = _tie_rows(rows, dim, dim + rows)
    d = x.to(DEV)
    _, y, q, s = E.add_rms_norm(d, None, None, 0.0, out_format="both")
    assert torch.equal(y.view(torch.int16), d.view(torch.int16))
    q2, s2 = E.mx_quantize(d.view(rows, dim))
    assert torch.equal(s.view(rows, -1), s2) and torch.equal(q.view(rows, dim), q2)
    codes, scale = o.mx_quantize(bits(x.view(rows, dim)))
    assert np.array_equal(u8(s).reshape(rows, -1), scale) and np.array_equal(u8(q).reshape(rows, dim), codes)


@pytest.mark.parametrize("T", [3, 40, 70])
@pytest.mark.parametrize("weights", ["mxfp4", "mxfp8"])
def test_a_nan_scale_makes_a_block_of_zero_codes_nan(T, weights):
    """OCP MX: byte 255 makes its whole block NaN, zero codes too, in a weight's
    scale and in a token's."""
    E = _E()
    K, N = 256, 96
    gen = X.generator(T, DEV)
    w, s = X.mxfp4_weight(N, K, gen) if weights == "mxfp4" else X.mxfp8_weight(N, K, gen)
    xq, xs = X.mxfp8_rows(T, K, gen)
    if weights == "mxfp4":
        w[9, 32:48], s[9, 2] = 0, 255                # k 64 .. 95 of row 9
        rows = torch.zeros(N, dtype=torch.bool, device=DEV)
        rows[9] = True
        got = E.wkv(X.bf16_rows(T, K, gen), w, s)
        assert torch.equal(torch.isnan(got), rows.expand(T, N))
    else:
        w[32:64, 64:96], s[1, 2] = 0, 255
        rows = (torch.arange(N, device=DEV) // 32) == 1
    assert torch.equal(torch.isnan(E.wkv_mx(xq, xs, w, s)), rows.expand(T, N))
    xq[1, 128:160], xs[1, 4] = 0, 255
    want = rows.expand(T, N).clone()
    want[1] = True
    assert torch.equal(torch.isnan(E.wkv_mx(xq, xs, w, s)), want)


@pytest.mark.parametrize("T", [3, 40, 70])
def test_subnormal_bf16_activations_count(T):
    """x of 2^-133 .. 2^-127 against weights near fp32's top: nothing is flushed."""
    E = _E()
    K, N = 256, 64
    gen = X.generator(T, DEV)
    w, s = X.mxfp4_weight(N, K, gen)
    s.fill_(250)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    x[:, ::16] = (torch.randint(1, 128, (T, K // 16), generator=gen, device=DEV).double() * 2.0 ** -133).to(torch.bfloat16)
    ref = X.product(x.double(), X.mxfp4_values(w, s))
    assert torch.equal(E.wkv(x, w, s), ref)


def test_two_threads_with_different_k_at_once():
    """Calls of two host threads, each on its own stream, with K that need
    different LDS from the same kernels: every result is the serial one."""
    import threading

    E = _E()
    T, N = 40, 2048
    jobs = []
    for i, K in enumerate((512, 16384)):
        gen = X.generator(i, DEV)
        w, s = X.mxfp4_weight(N, K, gen)
        x, (xq, xs) = X.bf16_rows(T, K, gen), X.mxfp8_rows(T, K, gen)
        wv = X.mxfp4_values(w, s)
        refs = X.product(x.double(), wv), X.product(X.mxfp8_row_values(xq, xs), wv)
        jobs.append((x, xq, xs, w, s, refs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    start, failed = threading.Barrier(2), []

    def work(x, xq, xs, w, s, refs, stream):
        try:
            with torch.cuda.stream(stream):
                start.wait(30)
                got = [(E.wkv(x, w, s), E.wkv_mx(xq, xs, w, s)) for _ in range(100)]
                stream.synchronize()
                for a, b in got:
                    assert torch.equal(a, refs[0]) and torch.equal(b, refs[1])
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed, failed

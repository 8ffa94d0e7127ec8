"""GPU: the residual RMS norm (bf16 and MXFP8 outputs), products of MXFP4
weights and products of MXFP8 activations, against the oracle in 64 bits.

Tolerances: products as in ``_block_inputs.product_tolerance``. Norm: the fp32
sum of squares of one row is off by at most (dim / 64 + 16) fp32 half steps,
relative (all terms positive; a thread adds at most dim/64 terms, then the
exchanges), the square root halves that, and 4 more roundings make y:
y_rel = (dim / 128 + 16) * 2^-24. bf16 outputs add half a bf16 step; codes add
half an e4m3 step: 2^-4 of the scaled value, at least half the least step 2^-10.
"""

from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from oracle import engram_oracle as o
from tests._block_inputs import BF16_U, F32_U, bf16, mxfp4_weight, mxfp8_rows, product_tolerance
from tests._util import bf16_values, bits, sample_tokens, u8

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


def _inside(got, ref, tol, what):
    bad = np.abs(got - ref) > tol
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - ref) - tol), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance; worst at {i}: "
                             f"got {got[i]!r}, ref {ref[i]!r}, tolerance {tol[i]!r}")


def _y_rel(dim):
    return (dim / 128 + 16) * F32_U


def _check_norm(dim, s, y, res, out, xq, xs):
    if res is not None:
        _inside(bf16_values(bits(res)), s, (BF16_U + 4 * F32_U) * np.abs(s) + 2.0 ** -134, "residual_out")
    yr = _y_rel(dim)
    if out is not None:
        _inside(bf16_values(bits(out)), y, (BF16_U * (1 + yr) + yr) * np.abs(y) + 2.0 ** -134, "out")
    if xq is not None:
        T, hc, _ = y.shape
        yb = y.reshape(T, hc, dim // 32, 32)
        amax = np.abs(yb).max(axis=-1)
        got_byte = u8(xs).astype(np.int64)
        _, e = np.frexp(amax)
        want = np.where(amax == 0, 0, np.clip(e - 1 - 8 + 127, 0, 254))
        # the byte may differ only where the maximum is at a power of two to fp32's rounding
        frac = amax / np.ldexp(1.0, e - 1)
        edge = (frac < 1 + 2 * yr) | (frac > 2 - 4 * yr)
        assert np.all((got_byte == want) | (edge & (np.abs(got_byte - want) <= 1)))
        scale = np.ldexp(1.0, got_byte - 127)[..., None]
        v = yb / scale
        dec = o.e4m3fn_decode(u8(xq)).reshape(yb.shape)
        slack = yr * np.abs(v)
        tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + slack
        sat = np.abs(v) > 448
        tol = np.where(sat, np.abs(v) - 448 + slack, tol)
        assert np.all(np.abs(v) < 512 * (1 + yr))
        _inside(dec, v, tol, "codes")


def _norm_ref(x, r, w, eps):
    c = lambda t: None if t is None else bits(t.contiguous())  # noqa: E731
    return o.add_rms_norm(c(x), c(r), c(w), eps)


@pytest.mark.parametrize("T,hc,dim", [(1, 1, 32), (1, 4, 4096), (3, 2, 64), (5, 3, 544), (17, 1, 1024), (2, 8, 2080),
                                      (33, 4, 2048), (4, 2, 4128), (9, 1, 7168), (3, 4, 8192), (2, 1, 8224), (3, 2, 16384),
                                      (700, 4, 256), (1030, 1, 512), (150, 2, 544), (300, 1, 1024), (131, 3, 2048),
                                      (97, 4, 2080), (70, 4, 4096), (65, 4, 4128), (259, 1, 7168), (90, 3, 8224),
                                      (260, 1, 16384)])
def test_norm_both_outputs(T, hc, dim):
    E = _E()
    rng = np.random.default_rng(dim * 7 + T)
    _say(f"norm {T} {hc} {dim}")
    x, r = bf16(rng, T, hc, dim, scale=3.0), bf16(rng, T, hc, dim)
    x[..., ::17] *= 40
    w = (1 + 0.2 * bf16(rng, hc, dim).float()).to(torch.bfloat16)
    res, out, xq, xs = E.add_rms_norm(x.to(DEV), r.to(DEV), w.to(DEV), 1e-6, out_format="both")
    torch.cuda.synchronize()
    _check_norm(dim, *_norm_ref(x, r, w, 1e-6), res, out, xq, xs)
    # each output alone, and without a residual
    _, o1, _, _ = E.add_rms_norm(x.to(DEV), r.to(DEV), w.to(DEV), 1e-6)
    _, _, q1, s1 = E.add_rms_norm(x.to(DEV), r.to(DEV), w.to(DEV), 1e-6, out_format="mxfp8")
    assert torch.equal(o1, out) and torch.equal(q1, xq) and torch.equal(s1, xs)
    n, o2, q2, s2 = E.add_rms_norm(x.to(DEV), None, None, 1e-3, out_format="both")
    assert n is None
    _check_norm(dim, *_norm_ref(x, None, None, 1e-3), None, o2, q2, s2)


@pytest.mark.parametrize("dim", [8, 24, 40, 1000, 4104, 11000])
def test_norm_bf16_odd_dims(dim):
    E = _E()
    rng = np.random.default_rng(dim)
    x, r, w = bf16(rng, 5, 3, dim), bf16(rng, 5, 3, dim), bf16(rng, dim)
    res, out, _, _ = E.add_rms_norm(x.to(DEV), r.to(DEV), w.to(DEV))
    _check_norm(dim, *_norm_ref(x, r, w, 1e-6), res, out, None, None)


def test_norm_more_rows_than_one_grid_dimension():
    """Rows past what one grid dimension holds (2^20 workgroups of 4 rows)."""
    E = _E()
    T, dim = (1 << 22) + 4099, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, dim), generator=g, device=DEV).to(torch.bfloat16)
    _, out, _, _ = E.add_rms_norm(x, None, None, 1e-6)
    at = torch.cat([torch.arange(0, 9), torch.arange((1 << 22) - 9, T), torch.randint(0, T, (4096,))]).to(DEV)
    s, y = _norm_ref(x[at][:, None].cpu(), None, None, 1e-6)
    _check_norm(dim, s, y, None, out[at][:, None], None, None)
    assert bool(torch.isfinite(out).all())


def test_norm_offsets_past_32_bits():
    """More than 2^32 elements: the last rows, and rows on both sides of the
    2^31- and 2^32-element marks."""
    E = _E()
    T, dim = (1 << 20) + 37, 4096
    g = torch.Generator(device=DEV).manual_seed(2)
    part = torch.randn((4099, dim), generator=g, device=DEV).to(torch.bfloat16)
    x = part.repeat((T + 4098) // 4099, 1)[:T]
    r = part[:1].expand(T, dim)
    w = (1 + 0.1 * torch.randn((dim,), generator=g, device=DEV)).to(torch.bfloat16)
    res, out, xq, xs = E.add_rms_norm(x, r, w, out_format="both")
    at = torch.cat([torch.arange(0, 5), torch.arange((1 << 19) - 3, (1 << 19) + 3),
                    torch.arange((1 << 20) - 3, T)]).to(DEV)
    s, y = _norm_ref(x[at][:, None].cpu(), r[at][:, None].cpu(), w.cpu(), 1e-6)
    _check_norm(dim, s, y, res[at][:, None], out[at][:, None], xq[at][:, None], xs[at][:, None])


def test_norm_strides_broadcast_two_dims_and_in_place():
    E = _E()
    rng = np.random.default_rng(3)
    T, hc, dim = 13, 4, 640
    wide = bf16(rng, T, hc, dim + 96).to(DEV)
    x = wide[..., 32:32 + dim]
    r = bf16(rng, T, 1, dim).to(DEV).expand(T, hc, dim)
    w = bf16(rng, hc, dim).to(DEV)
    before = wide.clone()
    got = E.add_rms_norm(x, r, w, out_format="both")
    _check_norm(dim, *_norm_ref(x.cpu(), r.cpu(), w.cpu(), 1e-6), *got)
    assert torch.equal(wide, before)
    # token-strided view (every second token), two dimensions
    x2 = bf16(rng, 2 * T, dim).to(DEV)[::2]
    _, o2, _, _ = E.add_rms_norm(x2, None, w[:1])
    s, y = _norm_ref(x2.cpu()[:, None], None, w[:1].cpu(), 1e-6)
    _check_norm(dim, s, y, None, o2[:, None], None, None)
    # in place: the residual stream updated where it lies, the norm over x
    xi, ri = x.contiguous(), r.contiguous()
    res, out, xq, xs = E.add_rms_norm(xi, ri, w, out_format="both", residual_out=ri, out=xi)
    assert res.data_ptr() == ri.data_ptr() and out.data_ptr() == xi.data_ptr()
    for a, b in zip((res, out, xq, xs), got):
        assert torch.equal(a, b)


def test_norm_leaves_what_follows_the_rows_alone():
    E = _E()
    rng = np.random.default_rng(4)
    T, hc, dim = 3, 2, 96
    x = bf16(rng, T, hc, dim).to(DEV)
    big = [torch.full((T * hc * dim + 4096,), 77, dtype=dt, device=DEV) for dt in (torch.bfloat16, torch.bfloat16)]
    bq = torch.full((T * hc * dim + 4096,), 77, dtype=torch.uint8, device=DEV)
    bs = torch.full((T * hc * 3 + 4096,), 77, dtype=torch.uint8, device=DEV)
    n = T * hc * dim
    E.add_rms_norm(x, x.clone(), None, out_format="both", residual_out=big[0][:n].view(T, hc, dim),
                   out=big[1][:n].view(T, hc, dim), xq=bq[:n].view(T, hc, dim), xs=bs[:T * hc * 3].view(T, hc, 3))
    assert all(bool((b[n:] == 77).all()) for b in big) and bool((bq[n:] == 77).all())
    assert bool((bs[T * hc * 3:] == 77).all())


def test_norm_zero_tiny_huge_and_non_finite_rows():
    E = _E()
    rng = np.random.default_rng(5)
    dim = 256
    x = bf16(rng, 8, 1, dim)
    x[0] = 0
    x[1] *= 1e-30                # squares vanish in fp32: eps alone
    x[2] *= 1e15                 # squares near fp32's upper range
    x[3, 0, 32:] = 0             # zero blocks beside a live one
    x[4, 0, 5] = float("inf")
    x[5, 0, 200] = float("nan")
    x[6] = x[6].abs() * 1e-3
    _, out, xq, xs = E.add_rms_norm(x.to(DEV), None, None, 1e-6, out_format="both")
    fin = [0, 1, 2, 3, 6, 7]
    s, y = _norm_ref(x[fin], None, None, 1e-6)
    _check_norm(dim, s, y, None, out[fin], None, None)
    _check_norm(dim, s[2:], y[2:], None, None, xq[fin][2:], xs[fin][2:])
    assert np.all(u8(xq[0]) & 0x7F == 0) and np.all(u8(xs[0]) == 0)
    assert np.all(u8(xq[3])[0, 32:] & 0x7F == 0) and np.all(u8(xs[3])[0, 1:] == 0)
    # an infinity makes its row's scale 0: it becomes NaN, the others 0; a NaN takes the row
    assert torch.isnan(out[4, 0, 5]) and u8(xs[4])[0, 0] == 255 and np.all(u8(xq[4])[0, :32] == 0x7F)
    assert bool((out[4, 0, 32:] == 0).all()) and np.all(u8(xs[4])[0, 1:] == 0)
    assert bool(torch.isnan(out[5]).all()) and np.all(u8(xs[5]) == 255) and np.all(u8(xq[5]) == 0x7F)


def test_norm_codes_match_the_quantizer_where_y_is_bf16():
    """Rows whose y is bf16 exactly (mean square 1, weight 1, eps 0): the codes
    are engram_mx_quantize's of that row, for every e4m3 midpoint and edge."""
    E = _E()
    rng = np.random.default_rng(6)
    dim = 4096
    x = torch.from_numpy(rng.integers(-2 ** 7, 2 ** 7, size=(64, dim)).astype(np.float32))
    x = x * torch.exp2(torch.from_numpy(rng.integers(-12, 1, size=(64, dim)).astype(np.float32)))
    x[:, -1] = 0
    # one element completes the row's sum of squares to a mean square that fp32 holds: use the scale of the row
    x = x.to(torch.bfloat16)[:, None]
    _, y, q, s = E.add_rms_norm(x.to(DEV), None, None, 0.0, out_format="both")
    q2, s2 = E.mx_quantize(y.view(64, dim))
    # y is rounded to bf16 there and not here: codes differ by at most one step, bytes at powers of two only
    a, b = o.e4m3fn_decode(u8(q).reshape(64, dim)), o.e4m3fn_decode(u8(q2))
    same = u8(s).reshape(64, -1) == u8(s2)
    assert same.mean() > 0.99
    keep = np.repeat(same, 32, axis=1)
    assert np.all(np.abs(a - b)[keep] <= np.maximum(np.abs(b)[keep] / 8, 2.0 ** -9) + 1e-12)
    assert (a == b)[keep].mean() > 0.95


KN = [(128, 4), (256, 64), (384, 100), (4096, 36), (8192, 20), (2048, 272), (4224, 96), (1024, 20480 // 8), (640, 1284),
      (2560, 5 * 16 * 3 + 36), (512, 20476), (384, 10236)]


@pytest.mark.parametrize("K,N", KN)
@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 33, 48, 50, 64, 65, 130, 300])
def test_mxfp4_products(T, K, N):
    E = _E()
    _say(f"mxfp4 products T {T} K {K} N {N}")
    rng = np.random.default_rng(T * 1000 + K + N)
    wq, ws = mxfp4_weight(rng, N, K)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    wa = o.mxfp4_dequantize_weight(wq, ws)
    x = bf16(rng, T, K)
    guard = torch.full((T * N + 512,), 55, dtype=torch.bfloat16, device=DEV)
    kv = guard[:T * N].view(T, N)
    E.wkv(x.to(DEV), wd, sd, kv=kv)
    ref, tol = product_tolerance(o.bf16_to_f64(bits(x)), wa)
    _inside(bf16_values(bits(kv)), ref, tol, "wkv mxfp4")
    assert bool((guard[T * N:] == 55).all())
    xq, xs = mxfp8_rows(rng, T, K)
    guard.fill_(55)
    E.wkv_mx(torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), wd, sd, kv=kv)
    ref, tol = product_tolerance(o.mx_dequantize_activations(xq, xs), wa, scaled=True)
    _inside(bf16_values(bits(kv)), ref, tol, "wkv_mx mxfp4")
    assert bool((guard[T * N:] == 55).all())


@pytest.mark.parametrize("T", [1, 40, 90])
def test_mxfp4_every_code_and_scale_lands_on_its_place(T):
    """One-hot activations read the weight back exactly: every code, distinct
    scales per row and block, through each route."""
    E = _E()
    K, N = 256, 160
    rng = np.random.default_rng(T)
    wq, ws = mxfp4_weight(rng, N, K, 100, 150)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    wa = o.mxfp4_dequantize_weight(wq, ws)
    one, s127 = 0x38, 127     # e4m3 1.0
    for k0 in range(0, K, T):
        ks = np.arange(k0, min(k0 + T, K))
        x = np.zeros((T, K))
        x[np.arange(len(ks)), ks] = 1.0
        want = np.zeros((T, N))
        want[:len(ks)] = wa[:, ks].T
        xb = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).to(DEV)
        assert np.array_equal(bf16_values(bits(E.wkv(xb, wd, sd))), want)
        xq = np.where(x == 1, one, 0).astype(np.uint8)
        xs = np.full((T, K // 32), s127, dtype=np.uint8)
        xs += (np.arange(K // 32) % 5).astype(np.uint8)     # x's own block scales: 1, 2, 4, 8, 16
        got = E.wkv_mx(torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), wd, sd)
        f = np.ones(T)
        f[:len(ks)] = 2.0 ** (ks // 32 % 5)
        assert np.array_equal(bf16_values(bits(got)), want * f[:, None])


@pytest.mark.parametrize("T", [2, 80])
def test_mxfp4_scale_edges(T):
    """Scale bytes at the ends of E8M0: 0 (2^-127), 1, 254 and NaN (255)."""
    E = _E()
    K, N = 128, 64
    for byte, xval in ((0, 2.0 ** 30), (1, 2.0 ** 30), (60, 1.0), (200, 1.0), (252, 2.0 ** -30), (254, 2.0 ** -30)):
        codes = np.tile(np.arange(16, dtype=np.uint8), K * N // 32)[: N * K // 2]
        wq = (codes | (np.roll(codes, 1) << 4)).reshape(N, K // 2)
        ws = np.full((N, K // 32), byte, dtype=np.uint8)
        x = np.zeros((T, K), dtype=np.float32)
        x[0, 3], x[1, 64] = xval, -xval
        xb = torch.from_numpy(x).to(torch.bfloat16)
        got = bf16_values(bits(E.wkv(xb.to(DEV), torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV))))
        # weights enter a bf16 product as bf16: at byte 254, codes of 2 and more
        # are at or past 2^128 and so infinite (and 0 * inf is NaN)
        wa = o.bf16_to_f64(o.round_to_bf16(o.mxfp4_dequantize_weight(wq, ws)))
        assert np.isfinite(wa).all() == (byte != 254)
        with np.errstate(invalid="ignore"):
            want = np.stack([(row[None] * wa).sum(axis=1) for row in o.bf16_to_f64(bits(xb))])
        assert np.array_equal(got, want, equal_nan=True), (byte, T)
    wq = np.full((N, K // 2), 0x22, dtype=np.uint8)
    ws = np.full((N, K // 32), 127, dtype=np.uint8)
    ws[5, 2] = 255
    x = torch.ones((T, K), dtype=torch.bfloat16, device=DEV)
    got = E.wkv(x, torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV))
    assert bool(torch.isnan(got[:, 5]).all()) and int(torch.isnan(got).sum()) == T
    q, s = E.mx_quantize(x)
    got = E.wkv_mx(q, s, torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV))
    assert bool(torch.isnan(got[:, 5]).all()) and int(torch.isnan(got).sum()) == T


@pytest.mark.parametrize("T", [3, 70])
def test_mxfp4_infinite_and_nan_activations_stay_in_their_token(T):
    E = _E()
    K, N = 256, 96
    rng = np.random.default_rng(T)
    wq, ws = mxfp4_weight(rng, N, K)
    wq[:, 10] = 0x21                # k 20: 0.5, k 21: 1.0 (positive)
    x = bf16(rng, T, K)
    x[1, 20] = float("inf")
    x[2, 7] = float("nan")
    got = E.wkv(x.to(DEV), torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)).cpu().float()
    assert bool((got[1] == float("inf")).all()) and bool(torch.isnan(got[2]).all())
    assert bool(torch.isfinite(got[0]).all()) and bool(torch.isfinite(got[3:]).all())


@pytest.mark.parametrize("T", [4, 40, 70])
def test_wkv_mx_nan_blocks_stay_in_their_token(T):
    """A NaN scale byte or a NaN code in one token's activations."""
    E = _E()
    K, N = 256, 96
    rng = np.random.default_rng(T)
    wq, ws = mxfp4_weight(rng, N, K)
    xq, xs = mxfp8_rows(rng, T, K)
    xs[1, 3], xq[3, 200] = 255, 0x7F
    got = E.wkv_mx(*[torch.from_numpy(a).to(DEV) for a in (xq, xs, wq, ws)]).cpu().float()
    assert bool(torch.isnan(got[[1, 3]]).all()) and bool(torch.isfinite(got[[0, 2]]).all())
    assert bool(torch.isfinite(got[4:]).all())


@pytest.mark.parametrize("T", [1, 9, 16, 40, 64, 65, 300])
@pytest.mark.parametrize("K,N", [(256, 96), (384, 160), (2048, 1280)])
def test_wkv_mx_with_mxfp8_weights_is_wkv_without_its_quantizer(T, K, N):
    E = _E()
    rng = np.random.default_rng(T + K)
    x = bf16(rng, T, K).to(DEV)
    w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    s = torch.from_numpy(rng.integers(119, 128, size=(N // 32, K // 32), dtype=np.uint8)).to(DEV)
    xq, xs = E.mx_quantize(x)
    assert torch.equal(E.wkv_mx(xq, xs, w, s), E.wkv(x, w, s))


@pytest.mark.parametrize("T,dim,hc,C", [(1, 512, 4, 8), (16, 256, 2, 8), (40, 136, 2, 8), (64, 512, 1, 6), (65, 512, 2, 8),
                                        (300, 512, 4, 8), (257, 264, 2, 8), (90, 256, 2, 6), (90, 136, 2, 6)])
@pytest.mark.parametrize("fp8_table", [False, True])
def test_forward_mxfp4(T, dim, hc, C, fp8_table):
    """The layer's forward on a 4-bit wkv weight, every route, against the
    oracle's forward (gate tolerance as the other formats' tests)."""
    E = _E()
    rng = np.random.default_rng(T + dim)
    hd, R = 64, 501      # C 6: K 384, a half chunk at the end
    K, N = C * hd, (hc + 1) * dim
    wq, ws = mxfp4_weight(rng, N, K, 122, 126)
    ids = torch.from_numpy(rng.integers(0, R, size=(T, C)).astype(np.int32)).to(DEV)
    hidden = bf16(rng, T, hc, dim).to(DEV)
    q = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    k = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    mask = torch.from_numpy(rng.random(T) > 0.2).to(DEV)
    if fp8_table:
        codes, scales = mxfp8_rows(rng, R, hd)
        rows, err = o.gather_rows_fp8(codes, scales, ids.cpu().numpy())
        table, ts = torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)
    else:
        table, ts = bf16(rng, R, hd, scale=0.1).to(DEV), None
        rows, err = o.gather_rows(bits(table), ids.cpu().numpy())
    assert not err
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    kv_bits, _ = o.wkv(rows.reshape(T, K), wq, ws)
    outs = []
    for store_kv in (False, True):
        gate = torch.full((T, hc), -1.0, dtype=torch.float32, device=DEV)
        out = E.forward(table, ids, wd, sd, hidden, q, k, mask, gate_out=gate, table_scales=ts, store_kv=store_kv)
        want, g = o.gate(bits(hidden), kv_bits, bits(q), bits(k), mask.cpu().numpy(), 1e-6, 1e-6)
        assert np.abs(gate.cpu().numpy() - g).max() < 2e-2        # kv itself is rounded to bf16 on both sides
        got, ref = bf16_values(bits(out)), o.bf16_to_f64(want)
        assert np.all(np.abs(got - ref) <= 2e-2 + 1e-2 * np.abs(ref))
        assert torch.equal(out[~mask], hidden[~mask])
        outs.append(out)
    plan = E.ForwardPlan(table, ids, wd, sd, hidden, q, k, mask, table_scales=ts)
    for _ in range(2):
        plan.out.zero_()
        assert torch.equal(plan.run(), outs[0])
    if T <= 64:
        a = E.forward_noalloc(table, ids, wd, sd, hidden, q, k, mask, table_scales=ts)
        assert torch.equal(a, outs[0])


@pytest.mark.parametrize("C", [8, 6])
def test_forward_mxfp4_gate_epilogue(C):
    """Enough tokens that the forward's default is the GEMM's gate epilogue (6
    x 80 tiles of 256x256 on 256 compute units), and the route that stores kv:
    sampled tokens against the oracle, the two against each other."""
    E = _E()
    rng = np.random.default_rng(21)
    T, dim, hc, hd, R = 1491, 4096, 4, 64, 301
    K, N = C * hd, (hc + 1) * dim
    wq, ws = mxfp4_weight(rng, N, K, 122, 126)
    table = bf16(rng, R, hd, scale=0.1).to(DEV)
    ids = torch.from_numpy(rng.integers(0, R, size=(T, C)).astype(np.int32)).to(DEV)
    hidden = bf16(rng, T, hc, dim).to(DEV)
    q = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    k = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    mask = torch.from_numpy(rng.random(T) > 0.2).to(DEV)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    gates = [torch.full((T, hc), -1.0, dtype=torch.float32, device=DEV) for _ in range(2)]
    outs = [E.forward(table, ids, wd, sd, hidden, q, k, mask, gate_out=g, store_kv=sk)
            for g, sk in zip(gates, (False, True))]
    assert float((gates[0] - gates[1]).abs().max()) < 1e-3
    toks = sample_tokens(T, 24, seed=2)
    at = torch.from_numpy(toks).to(DEV)
    rows, _ = o.gather_rows(bits(table), ids[at].cpu().numpy())
    kv_bits, _ = o.wkv(rows.reshape(len(toks), K), wq, ws)
    want, g = o.gate(bits(hidden[at]), kv_bits, bits(q), bits(k), mask[at].cpu().numpy(), 1e-6, 1e-6)
    ref = o.bf16_to_f64(want)
    for out, gate in zip(outs, gates):
        assert np.abs(gate[at].cpu().numpy() - g).max() < 2e-2
        assert np.all(np.abs(bf16_values(bits(out[at])) - ref) <= 2e-2 + 1e-2 * np.abs(ref))
        assert torch.equal(out[~mask], hidden[~mask])


def test_a_layer_then_norm_then_projection():
    """The operators as they are used: the layer's forward, its streams added
    to a branch and normalized into MXFP8, and that multiplied with 4-bit and
    8-bit weights; for a decode batch and a prompt."""
    E = _E()
    rng = np.random.default_rng(11)
    hc, dim, N, C, hd, R = 2, 512, 352, 8, 64, 301
    K = C * hd
    wq, ws = mxfp4_weight(rng, (hc + 1) * dim, K, 122, 126)
    w2, s2 = mxfp4_weight(rng, N, dim)
    w8 = rng.integers(0, 256, size=(N, dim), dtype=np.uint8)
    w8 = np.where((w8 & 0x7F) == 0x7F, 0, w8).astype(np.uint8)
    s8 = rng.integers(110, 118, size=(N // 32, dim // 32), dtype=np.uint8)
    table = bf16(rng, R, hd, scale=0.1).to(DEV)
    q, k = bf16(rng, hc, dim).to(DEV), bf16(rng, hc, dim).to(DEV)
    wn = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    for T in (1, 5, 130):
        ids = dev(rng.integers(0, R, size=(T, C)).astype(np.int32))
        hidden, branch = bf16(rng, T, hc, dim).to(DEV), bf16(rng, T, dim).to(DEV)
        stream = E.forward(table, ids, dev(wq), dev(ws), hidden, q, k)
        res, _, xq, xs = E.add_rms_norm(branch[:, None].expand(T, hc, dim), stream, wn, out_format="mxfp8")
        rows = xq.view(T * hc, dim), xs.view(T * hc, dim // 32)
        for w, s, wa in ((w2, s2, o.mxfp4_dequantize_weight(w2, s2)), (w8, s8, o.mx_dequantize_weight(w8, s8))):
            kv = E.wkv_mx(*rows, dev(w), dev(s))
            ref, tol = product_tolerance(o.mx_dequantize_activations(u8(rows[0]), u8(rows[1])), wa, scaled=True)
            _inside(bf16_values(bits(kv)), ref, tol, "projection")
        sref, yref = _norm_ref(branch[:, None].expand(T, hc, dim), stream, wn, 1e-6)
        _check_norm(dim, sref, yref, res, None, xq, xs)


def test_graph_replays_and_side_stream():
    """Captured once and replayed with new inputs between replays, with eager
    work in between; and on a stream of its own."""
    E = _E()
    rng = np.random.default_rng(12)
    hc, dim, N = 2, 1024, 640
    w2, s2 = mxfp4_weight(rng, N, dim)
    w2, s2 = torch.from_numpy(w2).to(DEV), torch.from_numpy(s2).to(DEV)
    wn = bf16(rng, dim).to(DEV)
    for T in (4, 100):
        x, r = bf16(rng, T, hc, dim).to(DEV), bf16(rng, T, hc, dim).to(DEV)
        res, out = torch.empty_like(r), torch.empty_like(x)
        xq = torch.empty((T, hc, dim), dtype=torch.uint8, device=DEV)
        xs = torch.empty((T, hc, dim // 32), dtype=torch.uint8, device=DEV)
        kv, kv2 = (torch.empty((T * hc, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))

        def go():
            E.add_rms_norm(x, r, wn, out_format="both", residual_out=res, out=out, xq=xq, xs=xs)
            E.wkv_mx(xq.view(T * hc, dim), xs.view(T * hc, dim // 32), w2, s2, kv=kv)
            E.wkv(out.view(T * hc, dim), w2, s2, kv=kv2)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            go()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
        for i in range(4):
            x.copy_(bf16(rng, T, hc, dim))
            for t in (res, out, kv, kv2):
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in (res, out, xq, xs, kv, kv2)]
            go()
            torch.cuda.synchronize()
            for a, b in zip(got, (res, out, xq, xs, kv, kv2)):
                assert torch.equal(a, b), (T, i)


def test_results_repeat_bit_for_bit():
    E = _E()
    rng = np.random.default_rng(13)
    wq, ws = mxfp4_weight(rng, 1280, 2048)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    for T in (1, 16, 64, 200):
        x = bf16(rng, T, 2048).to(DEV)
        q, s = E.mx_quantize(x)
        a, b = E.wkv(x, wd, sd), E.wkv_mx(q, s, wd, sd)
        for _ in range(3):
            assert torch.equal(E.wkv(x, wd, sd), a) and torch.equal(E.wkv_mx(q, s, wd, sd), b)
        # a token's result does not depend on the others in its batch, within a route
        if T in (16, 64):
            assert torch.equal(E.wkv(x[:T - 3].contiguous(), wd, sd), a[:T - 3])


def test_empty_batch():
    E = _E()
    x = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=DEV)
    res, out, xq, xs = E.add_rms_norm(x, x, None, out_format="both")
    assert out.shape == (0, 4, 128) and xs.shape == (0, 4, 4)
    wd = torch.zeros((64, 64), dtype=torch.uint8, device=DEV)
    sd = torch.zeros((64, 4), dtype=torch.uint8, device=DEV)
    assert E.wkv(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV), wd, sd).shape == (0, 64)
    e8 = torch.empty((0, 128), dtype=torch.uint8, device=DEV)
    assert E.wkv_mx(e8, torch.empty((0, 4), dtype=torch.uint8, device=DEV), wd, sd).shape == (0, 64)


def test_argument_errors_on_the_device():
    E = _E()
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        E.add_rms_norm(x, x[:, :1])
    with pytest.raises(ValueError):
        E.add_rms_norm(x.transpose(0, 2))
    with pytest.raises(ValueError):
        E.add_rms_norm(x, weight=torch.zeros((3, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        E.add_rms_norm(x.float())
    with pytest.raises(ValueError):
        E.add_rms_norm(x, residual_out=torch.empty_like(x))
    with pytest.raises(ValueError):
        E.add_rms_norm(x, out_format="fp4")
    with pytest.raises(ValueError):
        E.add_rms_norm(torch.zeros((2, 2, 40), dtype=torch.bfloat16, device=DEV), out_format="mxfp8")
    with pytest.raises(ValueError):
        E.add_rms_norm(torch.zeros((2, 2, 64 + 4), dtype=torch.bfloat16, device=DEV)[..., :64])
    with pytest.raises(ValueError):
        E.add_rms_norm(x, out=torch.empty((2, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError, match="one device"):
        E._device_of(x, _FakeOther())
    with pytest.raises(ValueError, match="device tensors"):
        E.add_rms_norm(x, weight=torch.zeros((64,), dtype=torch.bfloat16))


class _FakeOther:
    is_cuda = True

    def get_device(self):
        return 7


@pytest.mark.parametrize("op", ["wkv", "wkv_mx"])
@pytest.mark.parametrize("T,K,N", [(1500, 256, 20480), (1500, 512, 20476), (300, 768, 20480), (515, 256, 10236),
                                   (4096, 512, 5116), (1500, 384, 20476), (1500, 128, 20480), (300, 640, 20480),
                                   (515, 128, 10236), (4096, 384, 5116), (515, 1024, 20480), (515, 1152, 20476),
                                   (4000, 4096, 5116), (4000, 4224, 5120)])
def test_mxfp4_many_tiles(op, T, K, N):
    """Many tiles, ragged in T and N, with and without a half chunk at K's end:
    128x128, on 256 compute units 256x256 in those of 515 tokens and K past 1000
    (and the second with bf16 x), both in the last two; a token from every tile and some more."""
    E = _E()
    rng = np.random.default_rng(K)
    wq, ws = mxfp4_weight(rng, N, K)
    wa = o.mxfp4_dequantize_weight(wq, ws)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    toks = sample_tokens(T, 48, seed=1, tile=128)
    if op == "wkv":
        x = bf16(rng, T, K)
        xa = o.bf16_to_f64(bits(x))
        kv = E.wkv(x.to(DEV), wd, sd)
    else:
        xq, xs = mxfp8_rows(rng, T, K)
        xa = o.mx_dequantize_activations(xq, xs)
        kv = E.wkv_mx(torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), wd, sd)
    ref, tol = product_tolerance(xa[toks], wa, scaled=op == "wkv_mx")
    _inside(bf16_values(bits(kv[torch.from_numpy(toks).to(DEV)])), ref, tol, op)


@pytest.mark.parametrize("T,K,N", [(65, 128, 32), (70, 384, 96), (130, 256, 160), (257, 2048, 2080), (300, 640, 1280),
                                   (515, 512, 20480), (515, 896, 20480), (700, 4224, 20448), (4000, 4224, 5088)])
def test_wkv_mx_mxfp8_weight_tiles(T, K, N):
    """MXFP8 weights past the GEMV: 128x128 tiles in the first five, 256x256 in
    the next three, both in the last (on 256 compute units), with and without a half pair of slices at
    K's end, ragged in T and N."""
    E = _E()
    rng = np.random.default_rng(T + K)
    w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    s = rng.integers(119, 128, size=(N // 32, K // 32), dtype=np.uint8)
    xq, xs = mxfp8_rows(rng, T, K)
    guard = torch.full((T * N + 512,), 55, dtype=torch.bfloat16, device=DEV)
    kv = guard[:T * N].view(T, N)
    E.wkv_mx(*(torch.from_numpy(t).to(DEV) for t in (xq, xs, w, s)), kv=kv)
    assert bool((guard[T * N:] == 55).all())
    toks = sample_tokens(T, 48, seed=1, tile=128)
    ref, tol = product_tolerance(o.mx_dequantize_activations(xq[toks], xs[toks]), o.mx_dequantize_weight(w, s), scaled=True)
    _inside(bf16_values(bits(kv[torch.from_numpy(toks).to(DEV)])), ref, tol, "wkv_mx mxfp8")


@pytest.mark.parametrize("op", ["wkv", "wkv_mx"])
def test_mxfp4_output_offsets_past_32_bits(op):
    """kv of more than 2^32 elements (and x rows past 2^31 bytes of kv)."""
    E = _E()
    T, K, N = 70003, 256, 65536
    rng = np.random.default_rng(5)
    wq, ws = mxfp4_weight(rng, N, K)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    toks = np.concatenate([np.arange(3), [32767, 32768, 65535, 65536], np.arange(T - 5, T)])
    cols = np.concatenate([np.arange(8), np.arange(N // 2 - 4, N // 2 + 4), np.arange(N - 300, N)])
    if op == "wkv":
        x = bf16(rng, T, K)
        xa = o.bf16_to_f64(bits(x[torch.from_numpy(toks)]))
        kv = E.wkv(x.to(DEV), wd, sd)
    else:
        xq, xs = mxfp8_rows(rng, T, K)
        xa = o.mx_dequantize_activations(xq[toks], xs[toks])
        kv = E.wkv_mx(torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), wd, sd)
    ref, tol = product_tolerance(xa, o.mxfp4_dequantize_weight(wq[cols], ws[cols]), scaled=op == "wkv_mx")
    got = kv[torch.from_numpy(toks).to(DEV)][:, torch.from_numpy(cols).to(DEV)]
    _inside(bf16_values(bits(got)), ref, tol, op)


@pytest.mark.parametrize("T,K,N", [(1, 32768, 36), (20, 32768, 36), (50, 36864, 20), (40, 131072, 32), (3, 163840, 8),
                                   (64, 131072 + 128, 4)])
def test_mxfp4_long_k(T, K, N):
    """K past what a compute unit's LDS holds scale bytes for: the tiled GEMM,
    and the GEMV just below that."""
    E = _E()
    rng = np.random.default_rng(K + T)
    wq, ws = mxfp4_weight(rng, N, K)
    wa = o.mxfp4_dequantize_weight(wq, ws)
    wd, sd = torch.from_numpy(wq).to(DEV), torch.from_numpy(ws).to(DEV)
    x = bf16(rng, T, K)
    ref, tol = product_tolerance(o.bf16_to_f64(bits(x)), wa)
    _inside(bf16_values(bits(E.wkv(x.to(DEV), wd, sd))), ref, tol, "wkv")
    xq, xs = mxfp8_rows(rng, T, K)
    got = E.wkv_mx(torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), wd, sd)
    ref, tol = product_tolerance(o.mx_dequantize_activations(xq, xs), wa, scaled=True)
    _inside(bf16_values(bits(got)), ref, tol, "wkv_mx")


@pytest.mark.parametrize("T,dim,hc,K", [(1, 256, 1, 512), (64, 512, 2, 256), (300, 768, 2, 512), (70, 256, 3, 384),
                                         (9, 256, 1, 128), (300, 512, 2, 640)])
def test_mxfp4_gate_partials(T, dim, hc, K):
    """The projection fused with the gate's sums: the value block within the
    product's tolerance, the sums those of the bf16 keys of engram_wkv's tiled
    kernel to the gate tests' tolerance."""
    E = _E()
    rng = np.random.default_rng(T + dim)
    N = (hc + 1) * dim
    wq, ws = mxfp4_weight(rng, N, K, 116, 122)
    wa = o.mxfp4_dequantize_weight(wq, ws)
    x, hidden = bf16(rng, T, K), bf16(rng, T, hc, dim)
    q = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16)
    k = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16)
    args = [t.to(DEV) for t in (x, torch.from_numpy(wq), torch.from_numpy(ws), hidden, q, k)]
    value, parts = E.wkv_gate_partials(*args)
    ref, tol = product_tolerance(o.bf16_to_f64(bits(x)), wa)
    _inside(bf16_values(bits(value)), ref[:, hc * dim:], tol[:, hc * dim:], "value")
    keys = ref[:, :hc * dim].reshape(T, hc, dim // 256, 256)
    kt = tol[:, :hc * dim].reshape(T, hc, dim // 256, 256)
    h = o.bf16_to_f64(bits(hidden)).reshape(T, hc, dim // 256, 256)
    qk = (o.bf16_to_f64(bits(q)) * o.bf16_to_f64(bits(k))).reshape(1, hc, dim // 256, 256)
    got = parts.cpu().numpy().astype(np.float64)
    for i, c in ((0, h * qk), (1, None)):
        if c is None:
            want = (keys ** 2).sum(-1)
            lim = (2 * np.abs(keys) * kt + kt ** 2).sum(-1)
            mass = want
        else:
            want = (c * keys).sum(-1)
            lim = (np.abs(c) * kt).sum(-1)
            mass = (np.abs(c * keys)).sum(-1)
        # each key within its tolerance, then 256 fp32 products (3 roundings) and their sum
        lim = lim + (256 + 4) * F32_U * (mass + lim)
        err = np.abs(got[..., i] - want.transpose(1, 0, 2))
        assert np.all(err <= lim.transpose(1, 0, 2)), (i, float((err - lim.transpose(1, 0, 2)).max()))

"""GPU: rows and products in 8-bit integers and the norms around a block.

Products: the sums are whole numbers and exact, so kv is compared for equality
with the same fp32 steps (sum to fp32, times xs, times ws, to bf16) and against
64 bits within three fp32 half steps and one of bf16. Codes of the quantizer and
its scales: equality with the rule's fp32 steps.

Norms: one fp32 rounding is half a step, u = 2^-24. A row's sum of squares is off
by at most (dim / 64 + 16) u relative (all terms positive, a thread adds at most
dim / 64 of them, then the exchanges), an inverse root by half that and 3 more:
n = dim / 128 + 11. The branch p has that and 6 roundings (weight, gate, scales,
products), a sigmoid 16 more (2^-20); s one more. So
  ds = (n + 24) u * mass,          mass = |residual_scale * r| + |branch|
  dy = |y| (n + 4) u + |w| / rms * ds + |y| * |ds|_2 / |s|_2
(the last: the norm of a vector off by ds), before the output's own rounding:
half a bf16 step (2^-8), half an e4m3 step (2^-4, at least 2^-10 of the block's
scale), half a step of the row's int8 scale.
"""

from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

from oracle import engram_oracle as o
from tests import _int8_shapes as S
from tests._block_inputs import BF16_U, F32_U, bf16, mxfp8_rows
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


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _inside(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.nan_to_num(np.abs(got - ref) - tol, nan=np.inf), -np.inf)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance; worst at {i}: "
                             f"got {got[i]!r}, ref {ref[i]!r}, tolerance {tol[i]!r}")


# --------------------------------------------------------------- products --

def _int8(rng, n, k):
    """Codes of the whole range with -128 among them, scales around 2^-10."""
    return (rng.integers(-128, 128, size=(n, k)).astype(np.int8),
            (rng.uniform(0.5, 2.0, size=n) * 2.0 ** -10).astype(np.float32))


def _check_kv(kv, xq, xs, wq, ws, what):
    want, exact = o.int8_product(xq, xs, wq, ws)
    got = bf16_values(bits(kv))
    _inside(got, exact, (BF16_U * (1 + 4 * F32_U) + 3 * F32_U) * np.abs(exact) + 2.0 ** -134, what)
    assert np.array_equal(bits(kv), want), what


@pytest.mark.parametrize("K,N", S.KN)
@pytest.mark.parametrize("T", S.T)
def test_int8_products(T, K, N):
    E = _E()
    _say(f"int8 {T} {K} {N}")
    rng = np.random.default_rng(T * 1000 + K)
    xq, xs = _int8(rng, T, K)
    wq, ws = _int8(rng, N, K)
    guard = torch.full((T * N + 512,), 55, dtype=torch.bfloat16, device=DEV)
    kv = guard[:T * N].view(T, N)
    E.wkv_int8(_dev(xq), _dev(xs), _dev(wq), _dev(ws), kv=kv)
    assert bool((guard[T * N:] == 55).all())
    _check_kv(kv, xq, xs, wq, ws, "wkv_int8")
    # from bf16 rows
    x = bf16(rng, T, K)
    x[:, ::13] *= 20
    cq, cs = o.int8_quantize(bits(x))
    _check_kv(E.wkv(x.to(DEV), _dev(wq), _dev(ws)), cq, cs, wq, ws, "wkv")


@pytest.mark.parametrize("T,K,N", S.SMALL)
def test_int8_small_batches(T, K, N):
    """Row tiles in each of the ranges that the small-batch kernels are chosen by."""
    E = _E()
    _say(f"int8 small {T} {K} {N}")
    rng = np.random.default_rng(K + N)
    xq, xs = _int8(rng, T, K)
    wq, ws = _int8(rng, N, K)
    wd, sd = _dev(wq), _dev(ws)
    _check_kv(E.wkv_int8(_dev(xq), _dev(xs), wd, sd), xq, xs, wq, ws, "wkv_int8")
    if T <= 16:
        x = bf16(rng, T, K)
        _check_kv(E.wkv(x.to(DEV), wd, sd), *o.int8_quantize(bits(x)), wq, ws, "wkv")


@pytest.mark.parametrize("T,K,N", S.TILES)
def test_int8_many_tiles(T, K, N):
    E = _E()
    _say(f"int8 tiles {T} {K} {N}")
    rng = np.random.default_rng(K)
    xq, xs = _int8(rng, T, K)
    wq, ws = _int8(rng, N, K)
    kv = E.wkv_int8(_dev(xq), _dev(xs), _dev(wq), _dev(ws))
    toks = sample_tokens(T, 48, seed=1, tile=128)
    _check_kv(kv[torch.from_numpy(toks).to(DEV)], xq[toks], xs[toks], wq, ws, "wkv_int8")


@pytest.mark.parametrize("T", [1, 20, 64, 70])
@pytest.mark.parametrize("K", [32768, 131056])
def test_int8_long_k_of_the_largest_codes(T, K):
    """Every product 128 * 128: sums up to 2^31 - 2^18."""
    E = _E()
    N = 36
    xq = np.full((T, K), -128, dtype=np.int8)
    wq = np.full((N, K), -128, dtype=np.int8)
    wq[1::2] = 127
    xq[0, 5] = 3
    xs, ws = np.full(T, 2.0 ** -20, np.float32), np.linspace(0.5, 1, N, dtype=np.float32)
    _check_kv(E.wkv_int8(_dev(xq), _dev(xs), _dev(wq), _dev(ws)), xq, xs, wq, ws, "long")


@pytest.mark.parametrize("T", [3, 70])
def test_int8_scales_that_are_not_ordinary(T):
    """NaN, infinite, zero, negative and subnormal scales stay in their row or column."""
    E = _E()
    K, N = 256, 64
    rng = np.random.default_rng(T)
    xq, xs = _int8(rng, T, K)
    wq, ws = _int8(rng, N, K)
    xq[0], wq[5] = 0, 0
    xs[1], xs[2] = np.nan, -3e-40
    ws[3], ws[5], ws[7], ws[8] = np.inf, np.inf, 0, -1
    kv = E.wkv_int8(_dev(xq), _dev(xs), _dev(wq), _dev(ws)).float().cpu().numpy()
    acc = xq.astype(np.float64) @ wq.astype(np.float64).T
    with np.errstate(all="ignore"):
        want = torch.from_numpy((acc.astype(np.float32) * xs[:, None]) * ws[None]).to(torch.bfloat16).float().numpy()
    assert np.array_equal(np.isnan(kv), np.isnan(want))
    assert np.array_equal(kv[~np.isnan(want)], want[~np.isnan(want)])


def test_int8_output_offsets_past_32_bits():
    """kv of more than 2^32 elements."""
    E = _E()
    T, K, N = 70003, 144, 65536
    rng = np.random.default_rng(5)
    xq, xs = _int8(rng, T, K)
    wq, ws = _int8(rng, N, K)
    toks = np.concatenate([np.arange(3), [32767, 32768, 65535, 65536], np.arange(T - 5, T)])
    cols = np.concatenate([np.arange(8), np.arange(N // 2 - 4, N // 2 + 4), np.arange(N - 300, N)])
    kv = E.wkv_int8(_dev(xq), _dev(xs), _dev(wq), _dev(ws))
    got = kv[torch.from_numpy(toks).to(DEV)][:, torch.from_numpy(cols).to(DEV)]
    _check_kv(got, xq[toks], xs[toks], wq[cols], ws[cols], "past 32 bits")


def test_int8_weight_offsets_past_32_bits():
    """A weight of more than 2^32 bytes, few tokens and a prompt."""
    E = _E()
    K, N = 131056, 36868
    rng = np.random.default_rng(6)
    part = rng.integers(-128, 128, size=(128, K)).astype(np.int8)
    w = _dev(part).repeat((N + 127) // 128, 1)[:N].contiguous()
    ws = rng.uniform(0.5, 2, size=N).astype(np.float32)
    cols = np.concatenate([np.arange(8), np.arange(N // 2 - 4, N // 2 + 4), np.arange(N - 300, N)])
    for T in (3, 66):
        xq, xs = _int8(rng, T, K)
        kv = E.wkv_int8(_dev(xq), _dev(xs), w, _dev(ws))
        _check_kv(kv[:, torch.from_numpy(cols).to(DEV)], xq, xs, part[cols % 128], ws[cols], "weight")


# --------------------------------------------------------------- quantizer --

@pytest.mark.parametrize("T,K", S.ROWS)
def test_int8_quantizer(T, K):
    E = _E()
    _say(f"quantize {T} {K}")
    rng = np.random.default_rng(T + K)
    x = bf16(rng, T, K) * torch.from_numpy(2.0 ** rng.integers(-30, 30, size=(T, 1))).to(torch.bfloat16)
    xq, xs = E.int8_quantize(x.to(DEV))
    want, ws = o.int8_quantize(bits(x))
    assert np.array_equal(xq.cpu().numpy(), want) and np.array_equal(xs.cpu().numpy(), ws)


@pytest.mark.parametrize("K", [64, 1024, 4096])
def test_int8_quantizer_rows_that_are_not_ordinary(K):
    E = _E()
    rng = np.random.default_rng(K)
    x = bf16(rng, 12, K)
    x[0] = 0
    x[1] = 0; x[1, 3] = 2.0 ** -133
    x[2] *= 2.0 ** -125
    x[3] *= 3e37
    x[4, K - 1] = float("inf")
    x[5, 7] = float("-inf")
    x[6, 0] = float("nan")
    x[7] = 1.0
    x[8] = 0; x[8, ::2] = -0.0
    x[9] = 0; x[9, 1], x[9, 2], x[9, 3] = 127, 0.5, 1.5          # ties
    x[10] = 0; x[10, 1], x[10, 2], x[10, 3] = 254, -1, -3
    x[11] *= 2.0 ** -101
    xq, xs = E.int8_quantize(x.to(DEV))
    want, ws = o.int8_quantize(bits(x))
    assert np.array_equal(xq.cpu().numpy(), want)
    assert np.array_equal(xs.cpu().numpy(), ws, equal_nan=True)
    assert np.isnan(ws[4:7]).all() and xq.cpu().numpy()[9, :4].tolist() == [0, 127, 0, 2]


def test_int8_quantizer_offsets_past_32_bits():
    E = _E()
    T, K = 33001, 131056                       # 4.3e9 elements
    g = torch.Generator(device=DEV).manual_seed(3)
    part = torch.randn((67, K), generator=g, device=DEV).to(torch.bfloat16)
    x = part.repeat((T + 66) // 67, 1)[:T]
    xq, xs = E.int8_quantize(x)
    q, s = E.int8_quantize(part)
    for at in (0, 16385, 16386, 32771, 32772, T - 1):
        assert torch.equal(xq[at], q[at % 67]) and float(xs[at]) == float(s[at % 67])


# ------------------------------------------------------------------- norms --

def _norm_case(rng, T, hc, dim, gate, bcast=False, pad=0):
    x = bf16(rng, T, 1 if bcast else hc, dim + pad, scale=0.5)
    x[..., ::17] *= 30
    x = x[..., :dim].expand(T, hc, dim)
    r = bf16(rng, T, hc, dim, scale=2.0)
    w1, w2 = ((1 + 0.2 * bf16(rng, hc, dim).float()).to(torch.bfloat16) for _ in range(2))
    g = None
    if gate == "row":
        g = torch.from_numpy(rng.uniform(-0.2, 1, size=(T, hc)).astype(np.float32))
    elif gate == "channel":
        g = bf16(rng, T, hc, dim, scale=2.0)
    return x, r, w1, w2, g


def _norm_ref(x, r, w1, w2, g, act="none", post_norm=True, rs=1.0, bs=1.0, post_eps=1e-6, eps=1e-6):
    v = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    gv = v(g)
    if gv is not None and gv.ndim == 2:
        gv = gv[..., None]
    if gv is not None and act == "sigmoid":
        gv = 1 / (1 + np.exp(-gv))
    rs, bs, post_eps, eps = (float(np.float32(c)) for c in (rs, bs, post_eps, eps))
    s, y, mass = o.post_pre_norm(v(x), v(r), v(w1), v(w2), gv, post_norm, rs, bs, post_eps, eps)
    dim = x.shape[-1]
    n = dim / 128 + 11
    ds = (n + 24) * F32_U * mass
    norm = np.sqrt((s * s).sum(-1, keepdims=True))
    rms = np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    w = 1.0 if w2 is None else np.abs(v(w2))
    dy = np.abs(y) * (n + 4) * F32_U + w / rms * ds
    with np.errstate(invalid="ignore", divide="ignore"):
        dy = dy + np.abs(y) * np.nan_to_num(np.sqrt((ds * ds).sum(-1, keepdims=True)) / norm)
    return s, y, ds, dy


def _check_norm(ref, res, out=None, xq=None, xs=None, what=""):
    s, y, ds, dy = ref
    if res is not None:
        _inside(bf16_values(bits(res)).reshape(s.shape), s, ds + BF16_U * (np.abs(s) + ds) + 2.0 ** -134, what + "residual")
    if out is not None:
        _inside(bf16_values(bits(out)).reshape(y.shape), y, dy + BF16_U * (np.abs(y) + dy) + 2.0 ** -134, what + "out")
    if xq is not None and xq.dtype == torch.int8:
        scale = xs.cpu().numpy().astype(np.float64).reshape(y.shape[:-1] + (1,))
        amax = np.abs(y).max(-1, keepdims=True)
        top = dy.max(-1, keepdims=True)
        _inside(scale * 127, amax, top + 4 * F32_U * (amax + top) + 2.0 ** -140, what + "scales")
        codes = xq.cpu().numpy().astype(np.float64).reshape(y.shape)
        assert np.abs(codes).max() <= 127
        # half a step, the code's own roundings (3 relative ones of at most 127 steps)
        _inside(codes * scale, y, dy + scale * (0.5 + 127 * 8 * F32_U) + top, what + "int8")
    elif xq is not None:
        yb, db = y.reshape(-1, 32), dy.reshape(-1, 32)
        amax, top = np.abs(yb).max(-1), db.max(-1)
        byte = u8(xs).astype(np.int64).reshape(-1)
        lo, hi = (np.clip(np.frexp(np.maximum(amax + k * top, 1e-300))[1] - 1 - 8 + 127, 0, 254) for k in (-1, 1))
        assert np.all((byte >= lo) & (byte <= hi)), what + "scale bytes"
        scale = np.ldexp(1.0, byte - 127)[:, None]
        v, dv = yb / scale, db / scale
        dec = o.e4m3fn_decode(u8(xq)).reshape(v.shape)
        tol = np.maximum(2.0 ** -4 * (np.abs(v) + dv), 2.0 ** -10) + dv
        tol = np.where(np.abs(v) + dv > 448, np.maximum(tol, np.abs(v) + dv - 448), tol)
        _inside(dec, v, tol, what + "codes")


def _cut(t, rows):
    return None if t is None else t[rows]


SHAPES = [(1, 1, 32), (1, 4, 4096), (3, 2, 64), (5, 3, 544), (17, 1, 1024), (2, 8, 2080), (33, 4, 2048), (4, 2, 4128),
          (9, 1, 7168), (3, 4, 8192), (2, 1, 8224), (3, 2, 16384), (700, 4, 256), (1030, 1, 512), (150, 2, 544),
          (300, 1, 1024), (131, 3, 2048), (97, 4, 2080), (70, 4, 4096), (65, 4, 4128), (259, 1, 7168), (90, 3, 8224),
          (260, 1, 16384), (800, 1, 2048), (200, 4, 4096), (1000, 1, 4096), (100, 8, 8192), (400, 2, 7168),
          (300, 3, 16384)]


@pytest.mark.parametrize("T,hc,dim", SHAPES)
@pytest.mark.parametrize("gate,act", [("none", "none"), ("row", "none"), ("channel", "sigmoid")])
def test_norms_every_output(T, hc, dim, gate, act):
    E = _E()
    _say(f"norms {T} {hc} {dim} {gate}")
    rng = np.random.default_rng(dim * 7 + T)
    case = _norm_case(rng, T, hc, dim, gate)
    ref = _norm_ref(*case, act=act)
    x, r, w1, w2, g = (None if t is None else t.to(DEV) for t in case)
    call = lambda f, **k: E.post_pre_norm(x, r, w1, w2, g, gate_act=act, out_format=f, **k)  # noqa: E731
    res, out, xq, xs = call("both")
    _check_norm(ref, res, out, xq, xs, "mxfp8 ")
    r8, o8, q8, s8 = call("both", q_format="int8")
    assert torch.equal(r8, res) and torch.equal(o8, out)
    _check_norm(ref, None, None, q8, s8, "int8 ")
    # each alone
    r1, o1, n1, n2 = call("bf16")
    assert n1 is None and n2 is None and torch.equal(r1, res) and torch.equal(o1, out)
    _, n1, q1, s1 = call("mxfp8")
    assert n1 is None and torch.equal(q1, xq) and torch.equal(s1, xs)
    _, n1, q1, s1 = call("int8")
    assert n1 is None and torch.equal(q1, q8) and torch.equal(s1, s8)
    r1, n1, n2, n3 = call("none")
    assert torch.equal(r1, res) and n1 is None and n2 is None and n3 is None


@pytest.mark.parametrize("dim", [8, 24, 40, 1000, 4104, 11000])
@pytest.mark.parametrize("T", [2, 140])
def test_norms_odd_dims_and_options(T, dim):
    """No post norm, no weights, no residual, scales, a sigmoid on a row's gate,
    two epsilons."""
    E = _E()
    rng = np.random.default_rng(dim + T)
    x, r, w1, w2, g = _norm_case(rng, T, 2, dim, "row")
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    for args, kw in (((x, r, w1, w2, g), dict(post_norm=False, residual_scale=1.75, branch_scale=0.22)),
                     ((x, r, None, None, g), dict(gate_act="sigmoid", post_eps=1e-2, eps=1e-3)),
                     ((x, None, w1, w2, None), dict(branch_scale=-3.0)),
                     ((x, r, None, w2, None), dict(post_norm=False)),
                     ((x, r, w1, None, g), dict(residual_scale=0.0, branch_scale=1.0))):
        ref_kw = dict(act=kw.get("gate_act", "none"), post_norm=kw.get("post_norm", True), rs=kw.get("residual_scale", 1.0),
                      bs=kw.get("branch_scale", 1.0), eps=kw.get("eps", 1e-6), post_eps=kw.get("post_eps", 1e-6))
        ref = _norm_ref(*args, **ref_kw)
        res, out, xq, xs = E.post_pre_norm(*map(d, args), out_format="both", q_format="int8", **kw)
        _check_norm(ref, res, out, xq, xs, f"{sorted(kw)} ")
    # weights shared by the copies, two dimensions
    ref = _norm_ref(x[:, :1], r[:, :1], w1[:1], w2[:1], g[:, :1])
    res, out, xq, xs = E.post_pre_norm(d(x[:, 0]), d(r[:, 0]), d(w1[0]), d(w2[0]), d(g[:, 0]), out_format="both",
                                       q_format="int8")
    assert out.shape == (T, dim) and xs.shape == (T,)
    _check_norm(ref, res, out, xq, xs, "2d ")
    a = E.post_pre_norm(d(x), d(r), d(w1[0]), d(w2[:1]), d(g))
    b = E.post_pre_norm(d(x), d(r), d(w1[:1].expand(2, dim).contiguous()), d(w2[:1].expand(2, dim).contiguous()), d(g))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [5, 300])
def test_norms_strides_broadcast_and_in_place(T):
    E = _E()
    rng = np.random.default_rng(T)
    hc, dim = 3, 1056
    x, r, w1, w2, g = _norm_case(rng, T, hc, dim, "channel")
    want = E.post_pre_norm(x.to(DEV), r.to(DEV), w1.to(DEV), w2.to(DEV), g.to(DEV), out_format="both", q_format="int8")
    wide = torch.full((T, hc, 3 * dim + 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    views = [wide[..., i * (dim + 8):i * (dim + 8) + dim] for i in range(3)]
    for v, t in zip(views, (x, r, g)):
        v.copy_(t)
    got = E.post_pre_norm(views[0], views[1], w1.to(DEV), w2.to(DEV), views[2], out_format="both", q_format="int8")
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # one branch row and one gate row for every copy; a strided row gate
    xb, gb = x[:, :1].to(DEV).expand(T, hc, dim), g[:, :1].to(DEV).expand(T, hc, dim)
    a = E.post_pre_norm(xb, r.to(DEV), w1.to(DEV), w2.to(DEV), gb)
    b = E.post_pre_norm(xb.contiguous(), r.to(DEV), w1.to(DEV), w2.to(DEV), gb.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    gr = torch.from_numpy(rng.uniform(0, 1, size=(hc, 2 * T)).astype(np.float32)).to(DEV)[:, ::2].t()
    a = E.post_pre_norm(xb, r.to(DEV), w1.to(DEV), w2.to(DEV), gr)
    b = E.post_pre_norm(xb, r.to(DEV), w1.to(DEV), w2.to(DEV), gr.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # in place
    xi, ri = x.contiguous().to(DEV), r.to(DEV).clone()
    res, out, xq, xs = E.post_pre_norm(xi, ri, w1.to(DEV), w2.to(DEV), g.to(DEV), out_format="both", q_format="int8",
                                       residual_out=ri, out=xi)
    assert res is ri and out is xi
    for p, q in zip((res, out, xq, xs), want):
        assert torch.equal(p, q)


def test_norms_leave_what_follows_the_rows_alone():
    E = _E()
    rng = np.random.default_rng(3)
    for T, hc, dim in ((1, 1, 32), (7, 3, 96), (300, 1, 160), (3, 1, 2080), (600, 2, 1056)):
        x, r, w1, w2, _ = _norm_case(rng, T, hc, dim, "none")
        n = T * hc * dim
        for q, size in (("mxfp8", n // 32), ("int8", T * hc)):
            g = [torch.full((n + 256,), 7, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            qt, st = (torch.uint8, torch.uint8) if q == "mxfp8" else (torch.int8, torch.float32)
            gq = torch.full((n + 256,), 7, dtype=qt, device=DEV)
            gs = torch.full((size + 256,), 7, dtype=st, device=DEV)
            sshape = (T, hc, dim // 32) if q == "mxfp8" else (T, hc)
            E.post_pre_norm(x.to(DEV), r.to(DEV), w1.to(DEV), w2.to(DEV), out_format="both", q_format=q,
                            residual_out=g[0][:n].view(T, hc, dim), out=g[1][:n].view(T, hc, dim),
                            xq=gq[:n].view(T, hc, dim), xs=gs[:size].view(sshape))
            for t, m in ((g[0], n), (g[1], n), (gq, n), (gs, size)):
                assert bool((t[m:] == 7).all())


def test_norms_rows_that_are_not_ordinary():
    """Zero rows, infinities and NaN stay in their row; an int8 row with one has scale NaN."""
    E = _E()
    rng = np.random.default_rng(8)
    for dim in (64, 2080):
        x, r, w1, w2, g = _norm_case(rng, 9, 1, dim, "channel")
        x = x.contiguous()
        x[0], r[0] = 0, 0
        x[1, 0, 3] = float("inf")
        r[2, 0, 5] = float("nan")
        r[3, 0, 1] = float("-inf")
        g[4, 0, 2] = float("nan")
        x[5] = 0
        g[6, 0, :8] = torch.tensor([float("inf"), float("-inf"), 200, -200, 88, -88, 0, -0.0])
        x[7] *= 2.0 ** -120
        call = lambda f, **k: [None if t is None else t.float().cpu() for t in E.post_pre_norm(  # noqa: E731
            x.to(DEV), r.to(DEV), w1.to(DEV), w2.to(DEV), g.to(DEV), gate_act="sigmoid", out_format=f, **k)]
        res, out, q8, s8 = call("both", q_format="int8")
        assert bool((res[0] == 0).all()) and bool((out[0] == 0).all()) and float(s8[0, 0]) == 0
        assert bool(torch.isnan(s8[1:5]).all()) and bool((q8[1:5] == 0).all()) and bool((q8[0] == 0).all())
        _, _, qm, sm = call("mxfp8")
        assert bool((sm[2, 0, 0] == 255).all())
        ok = [0, 5, 6, 7, 8]
        ref = _norm_ref(x[ok], r[ok], w1, w2, g[ok], act="sigmoid")
        got = E.post_pre_norm(x.to(DEV), r.to(DEV), w1.to(DEV), w2.to(DEV), g.to(DEV), gate_act="sigmoid",
                              out_format="both", q_format="int8")
        _check_norm(ref, *(t[ok] for t in got))
        # eps 0 on a row of zeros: NaN, as the formula says
        z = torch.zeros((1, dim), dtype=torch.bfloat16, device=DEV)
        _, out, _, s8 = E.post_pre_norm(z, z, post_norm=False, eps=0.0, out_format="both", q_format="int8")
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(s8).all())


def test_norms_offsets_past_32_bits():
    E = _E()
    T, dim = (1 << 20) + 37, 4096
    g = torch.Generator(device=DEV).manual_seed(2)
    part = torch.randn((4099, dim), generator=g, device=DEV).to(torch.bfloat16)
    x = part.repeat((T + 4098) // 4099, 1)[:T]
    w = torch.ones((dim,), dtype=torch.bfloat16, device=DEV)
    res, _, xq, xs = E.post_pre_norm(x, x, w, w, out_format="int8")
    small = E.post_pre_norm(part, part, w, w, out_format="int8")
    for at in (0, 1 << 19, (1 << 20) - 3, 1 << 20, T - 1):
        i = at % 4099
        assert torch.equal(res[at], small[0][i]) and torch.equal(xq[at], small[2][i]) and float(xs[at]) == float(small[3][i])


# ------------------------------------------------------------- as they run --

def _forward_case(rng, T, dim, hc, C, hd, R, fp8_table):
    K, N = C * hd, (hc + 1) * dim
    wq = rng.integers(-127, 128, size=(N, K)).astype(np.int8)
    ws = rng.uniform(0.5, 2.0, size=N).astype(np.float32) * np.float32(2.0 ** -11)
    ids = rng.integers(0, R, size=(T, C)).astype(np.int32)
    hidden = bf16(rng, T, hc, dim).to(DEV)
    q = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    k = (1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16).to(DEV)
    mask = _dev(rng.random(T) > 0.2)
    if fp8_table:
        codes, scales = mxfp8_rows(rng, R, hd)
        table, ts = _dev(codes), _dev(scales)
        rows = lambda i: o.gather_rows_fp8(codes, scales, i)[0]  # noqa: E731
    else:
        table, ts = bf16(rng, R, hd, scale=0.1).to(DEV), None
        rows = lambda i: o.gather_rows(bits(table), i)[0]  # noqa: E731
    return wq, ws, ids, hidden, q, k, mask, table, ts, rows


@pytest.mark.parametrize("T,dim,hc,C,hd", S.FORWARD)
@pytest.mark.parametrize("fp8_table", [False, True])
def test_forward_int8(T, dim, hc, C, hd, fp8_table):
    """The layer's forward on an int8 wkv weight against the oracle's steps, the
    quantized rows and kv bit for bit those of the single calls."""
    E = _E()
    _say(f"forward {T} {dim} {hc} {C} {fp8_table}")
    rng = np.random.default_rng(T + dim)
    wq, ws, ids, hidden, q, k, mask, table, ts, rows = _forward_case(rng, T, dim, hc, C, hd, 501, fp8_table)
    K, N = C * hd, (hc + 1) * dim
    xq, xs = o.int8_quantize(rows(ids).reshape(T, K))
    kv_bits, _ = o.int8_product(xq, xs, wq, ws)
    wd, sd, idd = _dev(wq), _dev(ws), _dev(ids)
    want, g = o.gate(bits(hidden), kv_bits, bits(q), bits(k), mask.cpu().numpy(), 1e-6, 1e-6)
    outs = []
    for store_kv in (False, True):
        gate = torch.full((T, hc), -1.0, dtype=torch.float32, device=DEV)
        out = E.forward(table, idd, wd, sd, hidden, q, k, mask, gate_out=gate, table_scales=ts, store_kv=store_kv)
        assert np.abs(gate.cpu().numpy() - g).max() < 1e-3        # on the same kv, bit for bit
        got, ref = bf16_values(bits(out)), o.bf16_to_f64(want)
        assert np.all(np.abs(got - ref) <= 2e-2 + 1e-2 * np.abs(ref))
        assert torch.equal(out[~mask], hidden[~mask])
        outs.append(out)
    kv = torch.from_numpy(kv_bits.view(np.int16)).view(torch.bfloat16).to(DEV)
    assert torch.equal(outs[1], E.gate(hidden, kv, q, k, mask))
    plan = E.ForwardPlan(table, idd, wd, sd, hidden, q, k, mask, table_scales=ts)
    for _ in range(2):
        plan.out.zero_()
        assert torch.equal(plan.run(), outs[0])
    assert torch.equal(E.forward_noalloc(table, idd, wd, sd, hidden, q, k, mask, table_scales=ts), outs[0])
    with pytest.raises(ValueError):
        E.forward(table, idd, wd, sd, hidden, q, k, mask, table_scales=ts, single_launch=True)


def test_forward_int8_bad_ids():
    E = _E()
    rng = np.random.default_rng(4)
    T, dim, hc, C, hd = 3, 256, 2, 8, 64
    wq, ws, ids, hidden, q, k, mask, table, ts, rows = _forward_case(rng, T, dim, hc, C, hd, 101, False)
    ids[1, 2], ids[2] = 101, -1
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = E.forward(table, _dev(ids), _dev(wq), _dev(ws), hidden, q, k, None, err_flag=flag, store_kv=True)
    assert int(flag) == 1
    xq, xs = o.int8_quantize(rows(ids).reshape(T, C * hd))
    assert xs[2] == 0
    kv = torch.from_numpy(o.int8_product(xq, xs, wq, ws)[0].view(np.int16)).view(torch.bfloat16).to(DEV)
    assert torch.equal(out, E.gate(hidden, kv, q, k))


@pytest.mark.parametrize("C,hd", [(16, 64), (9, 112)])
def test_forward_int8_gate_epilogue(C, hd):
    """Enough tokens that the default is the GEMM's gate epilogue."""
    E = _E()
    rng = np.random.default_rng(21)
    T, dim, hc = 1491, 4096, 4
    wq, ws, ids, hidden, q, k, mask, table, ts, rows = _forward_case(rng, T, dim, hc, C, hd, 301, False)
    wd, sd, idd = _dev(wq), _dev(ws), _dev(ids)
    gates = [torch.full((T, hc), -1.0, dtype=torch.float32, device=DEV) for _ in range(2)]
    outs = [E.forward(table, idd, wd, sd, hidden, q, k, mask, gate_out=g, store_kv=sk) for g, sk in zip(gates, (False, True))]
    assert float((gates[0] - gates[1]).abs().max()) < 1e-3
    toks = sample_tokens(T, 24, seed=2)
    at = torch.from_numpy(toks).to(DEV)
    xq, xs = o.int8_quantize(rows(ids[toks]).reshape(len(toks), C * hd))
    kv_bits, _ = o.int8_product(xq, xs, wq, ws)
    want, g = o.gate(bits(hidden[at]), kv_bits, bits(q), bits(k), mask[at].cpu().numpy(), 1e-6, 1e-6)
    for out, gate in zip(outs, gates):
        assert np.abs(gate[at].cpu().numpy() - g).max() < 1e-3
        assert np.all(np.abs(bf16_values(bits(out[at])) - o.bf16_to_f64(want)) <= 2e-2 + 1e-2 * np.abs(o.bf16_to_f64(want)))
        assert torch.equal(out[~mask], hidden[~mask])


@pytest.mark.parametrize("T,dim,hc,K", [(1, 256, 1, 512), (64, 512, 2, 256), (300, 768, 2, 528), (70, 256, 3, 400)])
def test_int8_gate_partials(T, dim, hc, K):
    E = _E()
    rng = np.random.default_rng(T + dim)
    N = (hc + 1) * dim
    wq, ws = _int8(rng, N, K)
    x, hidden = bf16(rng, T, K), bf16(rng, T, hc, dim)
    q, k = ((1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16) for _ in range(2))
    value, parts = E.wkv_gate_partials(*(t.to(DEV) for t in (x, torch.from_numpy(wq), torch.from_numpy(ws), hidden, q, k)))
    kv_bits, _ = o.int8_product(*o.int8_quantize(bits(x)), wq, ws)
    assert np.array_equal(bits(value), kv_bits[:, hc * dim:])
    keys = o.bf16_to_f64(kv_bits[:, :hc * dim]).reshape(T, hc, dim // 256, 256)
    h = o.bf16_to_f64(bits(hidden)).reshape(T, hc, dim // 256, 256)
    qk = (o.bf16_to_f64(bits(q)) * o.bf16_to_f64(bits(k))).reshape(1, hc, dim // 256, 256)
    got = parts.cpu().numpy().astype(np.float64)
    # 256 fp32 products (3 roundings) and their sum
    for i, terms in ((0, h * qk * keys), (1, keys ** 2)):
        lim = (256 + 4) * F32_U * np.abs(terms).sum(-1)
        assert np.all(np.abs(got[..., i] - terms.sum(-1).transpose(1, 0, 2)) <= lim.transpose(1, 0, 2)), i


def test_a_layer_then_norms_then_projection():
    """The operators as they are used: the layer's forward on int8 weights with
    its gate out, a block's output normed, gated by it and added to the streams,
    normed into int8, and that multiplied."""
    E = _E()
    rng = np.random.default_rng(11)
    hc, dim, N, C, hd = 2, 512, 352, 8, 64
    w2, s2 = _int8(rng, N, dim)
    wn1, wn2 = ((1 + 0.1 * bf16(rng, hc, dim).float()).to(torch.bfloat16) for _ in range(2))
    for T in (1, 5, 130):
        wq, ws, ids, hidden, q, k, mask, table, ts, rows = _forward_case(rng, T, dim, hc, C, hd, 301, False)
        gate = torch.empty((T, hc), dtype=torch.float32, device=DEV)
        stream = E.forward(table, _dev(ids), _dev(wq), _dev(ws), hidden, q, k, gate_out=gate)
        branch = bf16(rng, T, dim)
        res, _, xq, xs = E.post_pre_norm(branch.to(DEV)[:, None].expand(T, hc, dim), stream, wn1.to(DEV), wn2.to(DEV), gate,
                                         out_format="int8")
        kv = E.wkv_int8(xq.view(T * hc, dim), xs.view(T * hc), _dev(w2), _dev(s2))
        _check_norm(_norm_ref(branch[:, None].expand(T, hc, dim), stream.cpu(), wn1, wn2, gate.cpu()), res, None, xq, xs)
        _check_kv(kv, xq.view(T * hc, dim).cpu().numpy(), xs.view(T * hc).cpu().numpy(), w2, s2, "projection")


def test_graph_replays_and_side_stream():
    E = _E()
    rng = np.random.default_rng(12)
    hc, dim, N = 2, 1024, 640
    w2, s2 = (_dev(a) for a in _int8(rng, N, dim))
    wn = bf16(rng, dim).to(DEV)
    for T in (4, 100):
        x, r = bf16(rng, T, hc, dim).to(DEV), bf16(rng, T, hc, dim).to(DEV)
        gate = torch.rand((T, hc), device=DEV)
        res, out = torch.empty_like(r), torch.empty_like(x)
        xq = torch.empty((T, hc, dim), dtype=torch.int8, device=DEV)
        xs = torch.empty((T, hc), dtype=torch.float32, device=DEV)
        kv, kv2 = (torch.empty((T * hc, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ws = torch.empty(E.load_library().engram_wkv_workspace_size(T * hc, dim, N, E.W_INT8), dtype=torch.uint8, device=DEV)
        outs = (res, out, xq, xs, kv, kv2)

        def go():
            E.post_pre_norm(x, r, wn, wn, gate, out_format="both", q_format="int8", residual_out=res, out=out, xq=xq, xs=xs)
            E.wkv_int8(xq.view(T * hc, dim), xs.view(T * hc), w2, s2, kv=kv)
            E.wkv(out.view(T * hc, dim), w2, s2, kv=kv2, workspace=ws)

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
            for t in outs:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs]
            go()
            torch.cuda.synchronize()
            for a, b in zip(got, outs):
                assert torch.equal(a, b), (T, i)


def test_every_route_gives_the_same_kv():
    """Whole-number sums: a token's kv does not depend on the batch it is in."""
    E = _E()
    rng = np.random.default_rng(13)
    K, N = 2048, 20480
    wd, sd = (_dev(a) for a in _int8(rng, N, K))
    x = bf16(rng, 700, K).to(DEV)
    q, s = E.int8_quantize(x)
    full = E.wkv_int8(q, s, wd, sd)
    for T in (1, 5, 8, 9, 16, 17, 40, 64, 65, 96, 100, 128, 129, 300, 600):
        assert torch.equal(E.wkv_int8(q[:T], s[:T], wd, sd), full[:T]), T
        assert torch.equal(E.wkv(x[:T], wd, sd), full[:T]), T


def test_empty_batch():
    E = _E()
    x = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=DEV)
    res, out, xq, xs = E.post_pre_norm(x, x, out_format="both", q_format="int8")
    assert out.shape == (0, 4, 128) and xs.shape == (0, 4) and xq.dtype == torch.int8
    wd = torch.zeros((64, 128), dtype=torch.int8, device=DEV)
    sd = torch.zeros((64,), dtype=torch.float32, device=DEV)
    assert E.wkv(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV), wd, sd).shape == (0, 64)
    q, s = E.int8_quantize(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV))
    assert E.wkv_int8(q, s, wd, sd).shape == (0, 64)


@pytest.mark.parametrize("T", [2, 40, 600])
def test_forward_int8_host_table_and_strided_ids(T):
    """Rows over the host link, and ids laid out column by column: the same output."""
    E = _E()
    rng = np.random.default_rng(T)
    dim, hc, C, hd = 256, 2, 8, 128
    wq, ws, ids, hidden, q, k, mask, table, _, _ = _forward_case(rng, T, dim, hc, C, hd, 301, False)
    wd, sd, idd = _dev(wq), _dev(ws), _dev(ids)
    want = E.forward(table, idd, wd, sd, hidden, q, k, mask)
    assert torch.equal(E.forward(table, idd.t().contiguous().t(), wd, sd, hidden, q, k, mask), want)
    _say(f"int8 host table T={T}")
    ht = E.HostTable(301, hd).copy_from(table)
    try:
        got = E.forward(ht, idd, wd, sd, hidden, q, k, mask)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    finally:
        ht.close()


def test_two_threads_at_once():
    """Calls of two host threads, each on its own stream, of different sizes: every
    result is the serial one."""
    import threading

    E = _E()
    rng = np.random.default_rng(5)
    hc, start, failed, jobs = 2, threading.Barrier(2), [], []
    for T, dim, N in ((3, 1024, 4096), (150, 2064, 1280)):
        x, r, w1, w2, g = (t.contiguous().to(DEV) for t in _norm_case(rng, T, hc, dim, "row"))
        wq, ws = (_dev(a) for a in _int8(rng, N, dim))

        def calls(x=x, r=r, w1=w1, w2=w2, g=g, wq=wq, ws=ws, n=T * hc, dim=dim):
            res, out, xq, xs = E.post_pre_norm(x, r, w1, w2, g, out_format="both", q_format="int8")
            return res, out, xq, xs, E.wkv_int8(xq.view(n, dim), xs.view(n), wq, ws), E.wkv(out.view(n, dim), wq, ws)

        jobs.append((calls, calls(), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(calls, want, stream):
        try:
            with torch.cuda.stream(stream):
                start.wait(30)
                got = [calls() for _ in range(60)]
                stream.synchronize()
                for i in got:
                    for a, b in zip(i, want):
                        assert torch.equal(a, b)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not failed, failed

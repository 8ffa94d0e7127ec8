"""The int8 products and the norms around a block without a GPU: the oracle's
functions against worked values, the argument struct's layout, what the C ABI and
the binding refuse before any launch."""

from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from gram_memory_layer_engram_amd import build, engram as E
from oracle import engram_oracle as o
from tests._block_inputs import bf16
from tests._util import bits

OK, INV, UNS = 0, 1, 2
I8 = 3
BF, I8T, F32, U8 = torch.bfloat16, torch.int8, torch.float32, torch.uint8
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "engram.h")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(E.LIB_PATH):
        build.build()
    return E.load_library()


# ------------------------------------------------------------------ oracle --

def test_quantizer_on_worked_rows():
    x = torch.tensor([[127, 0.5, 1.5, -2.5], [0, 0, -0.0, 0], [-254, 1, 3, 254], [float("inf"), 1, 2, 3],
                      [float("nan"), 1, 2, 3], [2.0 ** -133, 0, -2.0 ** -133, 0]]).to(BF)
    codes, scales = o.int8_quantize(bits(x))
    assert codes.tolist() == [[127, 0, 2, -2], [0] * 4, [-127, 0, 2, 127], [0] * 4, [0] * 4, [127, 0, -127, 0]]
    assert scales[:3].tolist() == [1, 0, 2] and np.isnan(scales[3:5]).all()
    assert scales[5] == np.float32(2.0 ** -133) / np.float32(127)


def test_quantizer_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = bf16(rng, 50, 333) * torch.from_numpy(2.0 ** rng.integers(-90, 90, size=(50, 1))).to(BF)
    codes, scales = o.int8_quantize(bits(x))
    v = x.double().numpy()
    s = scales.astype(np.float64)[:, None]
    # the codes' three fp32 roundings (each 2^-24 of at most 127 steps) and the scale's
    assert np.all(np.abs(codes * s - v) <= s * (0.5 + 4 * 127 * 2.0 ** -24))
    assert np.abs(codes).max(axis=1).tolist() == [127] * 50


def test_product_on_worked_values():
    xq = np.array([[1, -2, 127], [-128, 0, 5]], dtype=np.int8)
    wq = np.array([[3, 4, -1], [-128, 127, 127]], dtype=np.int8)
    got, exact = o.int8_product(xq, np.float32([0.5, 2]), wq, np.float32([1, 0.25]))
    assert exact.tolist() == [[-66.0, 15747 / 8], [-778.0, 17019 / 2]]
    assert o.bf16_to_f64(got).tolist() == [[-66.0, 1968.0], [-776.0, 8512.0]]


def test_norms_with_one_norm_are_the_residual_norm():
    rng = np.random.default_rng(1)
    x, r, w = bf16(rng, 4, 2, 64), bf16(rng, 4, 2, 64), bf16(rng, 2, 64)
    s, y, _ = o.post_pre_norm(x.double().numpy(), r.double().numpy(), None, w.double().numpy(), None, False, 1.0, 1.0, 0, 1e-6)
    s2, y2 = o.add_rms_norm(bits(x), bits(r), bits(w), 1e-6)
    assert np.array_equal(s, s2) and np.allclose(y, y2, rtol=1e-14)


def test_norms_by_hand():
    x = np.array([[[3.0, 4.0]]])          # rms 5 / sqrt(2)
    s, y, _ = o.post_pre_norm(x, np.array([[[1.0, 1.0]]]), np.array([1.0, 2.0]), np.array([2.0, 1.0]), np.array([[[0.5]]]),
                              True, 2.0, 10.0, 0.0, 0.0)
    q = np.sqrt(2) / 5
    want = np.array([2 + 10 * 0.5 * 3 * q, 2 + 10 * 0.5 * 8 * q])
    assert np.allclose(s[0, 0], want, rtol=1e-15)
    assert np.allclose(y[0, 0], want / np.sqrt((want ** 2).mean()) * [2, 1], rtol=1e-15)


# --------------------------------------------------------------------- ABI --

def test_args_layout_matches_c(tmp_path):
    fields = [f for f, _ in E.PostPreNormArgs._fields_]
    src = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{HEADER}"', "int main(void) {",
           'printf("%zu\\n", sizeof(engram_post_pre_norm_args));']
    src += [f'printf("%zu\\n", offsetof(engram_post_pre_norm_args, {f}));' for f in fields] + ["return 0; }"]
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src))
    subprocess.run(["gcc", "-std=c99", str(c), "-o", str(exe)], check=True)
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(E.PostPreNormArgs)
    assert [getattr(E.PostPreNormArgs, f).offset for f in fields] == vals[1:]
    # the binding packs the same bytes
    v = [i + 1 if t not in (ctypes.c_float,) else 0.5 + i for i, (_, t) in enumerate(E.PostPreNormArgs._fields_)]
    assert E._pack_post_pre_norm(*v) == bytes(E.PostPreNormArgs(*v))


X, XS, W, WS, KV, R, G, P1, P2, RO, OUT, XQ = (i << 28 for i in range(1, 13))


def test_quantizer_refusals(lib):
    q = lib.engram_int8_quantize
    assert q(None, 0, 64, None, None, None) == OK
    assert q(X, -1, 64, XQ, XS, None) == INV and q(X, 1, 0, XQ, XS, None) == INV
    for K in (8, 24, 100, 1 << 17):
        assert q(X, 1, K, XQ, XS, None) == UNS, K
    for args in ((None, XQ, XS), (X, None, XS), (X, XQ, None), (X + 8, XQ, XS), (X, XQ + 4, XS), (X, XQ, XS + 2),
                 (X, X + 2 * 3 * 64 - 16, XS), (X, XQ, X + 2 * 3 * 64 - 4), (X, XQ, XQ + 3 * 64 - 4)):
        assert q(args[0], 3, 64, args[1], args[2], None) == INV, args


def test_product_refusals(lib):
    def f(xq=X, xs=XS, T=3, K=64, w=W, ws=WS, N=32, kv=KV):
        return lib.engram_wkv_int8(xq, xs, T, K, w, ws, N, kv, None)

    assert f(None, None, 0, 64, None, None, 32, None) == OK
    assert f(T=-1) == INV and f(K=0) == INV and f(N=0) == INV
    for kw in (dict(K=8), dict(K=100), dict(K=1 << 17), dict(N=30), dict(N=(1 << 28) + 4), dict(T=1 << 31), dict(T=(1 << 30) + 1)):
        assert f(**kw) == UNS, kw
    for name in ("xq", "xs", "w", "ws", "kv"):
        assert f(**{name: None}) == INV
    assert f(xq=X + 8) == INV and f(xs=XS + 2) == INV and f(w=W + 4) == INV and f(ws=WS + 4) == INV and f(kv=KV + 8) == INV
    for base, size in ((X, 192), (XS, 12), (W, 2048), (WS, 128)):
        for kv in (base, base + (size - 1) // 16 * 16, base - 192 + 16):
            assert f(kv=kv) == INV, hex(kv)


def test_wkv_and_partials_with_int8_weights_refuse(lib):
    # a few tokens are quantized in the product's launch
    assert [lib.engram_wkv_workspace_size(T, 64, 32, I8) for T in (0, 1, 16, 17)] == [0, 0, 0, 1280 + 256]
    assert [lib.engram_wkv_workspace_size(8, 4096, 16384, I8), lib.engram_wkv_workspace_size(16, 64, 12288, I8)] == [0, 0]
    assert lib.engram_wkv_workspace_size(9, 64, 12292, I8) == 768 + 256
    assert lib.engram_wkv_workspace_size(8, 4112, 64, I8) == 8 * 4112 + 256 - 8 * 4112 % 256 + 256
    assert lib.engram_wkv_workspace_size(8, 4096, 16388, I8) == 8 * 4096 + 256
    need = lib.engram_wkv_workspace_size(20, 64, 32, I8)
    assert need == 1280 + 256
    WK = 13 << 28

    def f(kv=KV, ws=WK, n=need, x=X, K=64):
        return lib.engram_wkv(x, 20, K, W, WS, I8, 32, kv, ws, n, None)

    assert f(n=need - 1) == INV and f(ws=None) == INV and f(ws=WK + 16) == INV and f(K=72) == UNS
    for base in (X, X + 1280, W, W + 1792, WS, KV, KV + 512):
        assert f(ws=base) == INV, hex(base)
    for kv in (X, W + 2032, WS + 112):
        assert f(kv=kv) == INV
        assert lib.engram_wkv(X, 3, 64, W, WS, I8, 32, kv, None, 0, None) == INV
    assert lib.engram_wkv(X, 3, 64, W, None, I8, 32, KV, WK, need, None) == INV
    assert lib.engram_wkv(None, 0, 64, None, None, I8, 32, None, None, 0, None) == OK

    T, K, hc, dim = 4, 256, 2, 256
    need = lib.engram_wkv_gate_partials_workspace_size(T, K, hc, dim, I8)
    assert need == 1024 + 256 and lib.engram_wkv_gate_partials_workspace_size(T, K, hc, dim, 2) == 0
    assert lib.engram_wkv_gate_partials_workspace_size(T, K, hc, dim, 1) == lib.engram_wkv_workspace_size(T, K, 768, 1)
    H, Q, KW, V, PA = (i << 28 for i in range(14, 19))

    def g(value=V, partials=PA, ws=WK):
        return lib.engram_wkv_gate_partials(X, T, K, W, WS, I8, hc, dim, H, Q, KW, value, partials, ws, need, None)

    for base, size in ((X, 2048), (W, 768 * 256), (WS, 4 * 768), (H, 4096), (Q, 1024), (KW, 1024)):
        assert g(value=base + size - 16) == INV and g(partials=base + size - 8) == INV
        assert g(ws=base + (size - 1) // 256 * 256) == INV, hex(base)
    assert g(partials=V + 2048 - 8) == INV and g(ws=V) == INV and g(ws=PA) == INV


def norms(lib, **kw):
    a = E.PostPreNormArgs(x=X, x_stride_t=128, x_stride_h=64, residual=R, residual_stride_t=128, residual_stride_h=64,
                          gate=None, gate_format=0, post_weight=P1, pre_weight=P2, post_weight_hc=1, pre_weight_hc=2, T=3,
                          hc=2, dim=64, post_norm=1, post_eps=1e-6, eps=1e-6, residual_scale=1, branch_scale=1, q_format=2,
                          residual_out=RO, out=OUT, xq=XQ, xs=XS)
    for k, v in kw.items():
        setattr(a, k, v)
    return lib.engram_post_pre_norm(ctypes.byref(a), None)


def test_norms_refusals(lib):
    assert lib.engram_post_pre_norm(None, None) == INV
    assert norms(lib, T=0) == OK and norms(lib, T=0, x=None, xq=None, xs=None) == OK
    for kw in (dict(T=-1), dict(hc=0), dict(dim=0), dict(eps=-1), dict(post_eps=float("nan")), dict(x_stride_t=-8),
               dict(residual_stride_h=-8), dict(gate_stride_t=-1), dict(gate_format=3), dict(gate_format=-1),
               dict(gate_sigmoid=2), dict(post_norm=2), dict(q_format=3), dict(gate_format=1), dict(gate=G), dict(xq=None),
               dict(xs=None), dict(q_format=0), dict(post_weight_hc=3), dict(pre_weight_hc=0), dict(x=None),
               dict(q_format=0, xq=None, xs=None, out=None, residual_out=None), dict(x=X + 8), dict(residual=R + 2),
               dict(post_weight=P1 + 4), dict(pre_weight=P2 + 8), dict(out=OUT + 8), dict(residual_out=RO + 8),
               dict(xq=XQ + 8), dict(xs=XS + 2), dict(gate=G + 2, gate_format=1), dict(gate=G + 8, gate_format=2)):
        assert norms(lib, **kw) == INV, kw
    for kw in (dict(dim=60), dict(dim=16392), dict(dim=40, q_format=1), dict(x_stride_t=100), dict(residual_stride_h=4),
               dict(gate=G, gate_format=2, gate_stride_t=4), dict(T=1 << 30)):
        assert norms(lib, **kw) == UNS, kw


def test_norms_refuse_outputs_on_other_tensors(lib):
    n = 3 * 2 * 64
    gate = dict(gate=G, gate_format=2, gate_stride_t=128, gate_stride_h=64)
    sizes = dict(x=(X, 2 * n), residual=(R, 2 * n), gate=(G, 2 * n), post=(P1, 128), pre=(P2, 256))
    outs = dict(out=2 * n, residual_out=2 * n, xq=n, xs=24)
    for name, size in outs.items():
        for t, (base, bytes_) in sizes.items():
            whole = (name, t) in (("out", "x"), ("residual_out", "residual"))
            for at in ([] if whole else [base]) + [base + bytes_ - 16, base - (size - 1) // 16 * 16]:
                assert norms(lib, **gate, **{name: at}) == INV, (name, t, hex(at - base))
    for a, size in outs.items():
        for b, base in dict(out=OUT, residual_out=RO, xq=XQ, xs=XS).items():
            if a != b:
                assert norms(lib, **{a: base}) == INV, (a, b)
    # in place only where the rows are whole: a wider tensor's, a row shared by the copies
    for kw in (dict(out=X, x_stride_t=192), dict(out=X, x_stride_h=0), dict(residual_out=R, residual_stride_t=192),
               dict(residual_out=X), dict(out=R)):
        assert norms(lib, **kw) == INV, kw


# ----------------------------------------------------------------- binding --

class OnDevice(torch.Tensor):
    """Host memory that says it is a device tensor's, for calls that are refused."""

    is_cuda = True

    def get_device(self):
        return 0


class Elsewhere(OnDevice):
    def get_device(self):
        return 1


def dev(*shape, dtype=BF, cls=OnDevice):
    return torch.zeros(shape, dtype=dtype).as_subclass(cls)


def test_forward_takes_int8_weights():
    T, HC, DIM, C, HD = 3, 2, 64, 4, 64
    K, N = C * HD, (HC + 1) * DIM

    def args(w, s):
        return E.forward_args(dev(10, HD), dev(T, C, dtype=torch.int32), w, s, dev(T, HC, DIM), dev(HC, DIM), dev(HC, DIM),
                              None, 1e-6, 1e-6, dev(T, HC, DIM))

    assert args(dev(N, K, dtype=I8T), dev(N, dtype=F32)).w_format == E.W_INT8
    for w, s in ((dev(N - 4, K, dtype=I8T), dev(N, dtype=F32)), (dev(N, K, dtype=I8T), dev(N - 1, dtype=F32)),
                 (dev(N, K - 16, dtype=I8T), dev(N, dtype=F32)), (dev(N, K, dtype=U8), dev(N, dtype=F32)),
                 (dev(N, K), dev(N, dtype=F32)), (dev(N, K, dtype=I8T), dev(2 * N, dtype=F32)[::2]),
                 (dev(N, K, dtype=I8T), None), (dev(N, K, dtype=I8T), dev(N, 1, dtype=F32))):
        with pytest.raises(ValueError, match="int8|w must be"):
            args(w, s)


def test_products_refuse():
    xq, xs, w, s = dev(3, 64, dtype=I8T), dev(3, dtype=F32), dev(32, 64, dtype=I8T), dev(32, dtype=F32)
    bad = [(xq.to(U8), xs, w, s), (xq, xs.to(BF), w, s), (xq, xs, w.to(U8), s), (xq, xs, w, s.double()),
           (xq, dev(4, dtype=F32), w, s), (xq, dev(3, 1, dtype=F32), w, s), (xq, xs, dev(32, 48, dtype=I8T), s),
           (xq, xs, w, dev(31, dtype=F32)), (dev(3, 128, dtype=I8T)[:, ::2], xs, w, s), (xq, xs, w.t(), s),
           (xq, dev(3, dtype=F32, cls=Elsewhere), w, s), (xq, xs, dev(32, 64, dtype=I8T, cls=Elsewhere), s),
           (xq, xs, w, dev(32, dtype=F32, cls=Elsewhere)),
           (torch.zeros(3, 64, dtype=I8T), torch.zeros(3), torch.zeros(32, 64, dtype=I8T), torch.zeros(32))]
    for i, args in enumerate(bad):
        with pytest.raises(ValueError):
            E.wkv_int8(*args)
            pytest.fail(f"case {i}")
    for kv in (dev(3, 31), dev(3, 32, dtype=F32), dev(3, 64)[:, ::2], dev(3, 32, cls=Elsewhere)):
        with pytest.raises(ValueError, match="kv"):
            E.wkv_int8(xq, xs, w, s, kv=kv)
    for x, wt, sc in ((dev(3, 64, dtype=F32), w, s), (dev(3, 48), w, s), (dev(3, 64), w, dev(16, dtype=F32)),
                      (dev(3, 64), w.to(U8), s)):
        with pytest.raises(ValueError):
            E.wkv(x, wt, sc)
    with pytest.raises(ValueError, match="workspace"):
        E.wkv(dev(9, 64), w, s, kv=dev(9, 32), workspace=dev(4096, dtype=U8, cls=Elsewhere))


def test_quantizer_binding_refuses():
    x = dev(3, 64)
    for bad in (dev(3, 64, dtype=F32), dev(3, 2, 64), dev(64, 3).t(), torch.zeros((3, 64), dtype=BF)):
        with pytest.raises(ValueError):
            E.int8_quantize(bad)
    good = dict(xq=dev(3, 64, dtype=I8T), xs=dev(3, dtype=F32))
    for kw in (dict(xq=dev(3, 64, dtype=U8)), dict(xq=dev(3, 32, dtype=I8T)), dict(xs=dev(3)), dict(xs=dev(3, 1, dtype=F32)),
               dict(xs=dev(3, dtype=F32, cls=Elsewhere)), dict(xq=dev(3, 64, dtype=I8T, cls=Elsewhere))):
        with pytest.raises(ValueError):
            E.int8_quantize(x, **{**good, **kw})


def test_norms_binding_refuses():
    x = dev(3, 2, 64)
    g = dev(3, 2, dtype=F32)
    outs = dict(residual_out=dev(3, 2, 64), out=dev(3, 2, 64))
    for args, kw in (((dev(64),), {}), ((dev(3, 2, 64, dtype=F32),), {}), ((torch.zeros(3, 2, 64, dtype=BF),), {}),
                     ((dev(3, 2, 128)[..., ::2],), {}), ((x, dev(3, 1, 64)), {}), ((x, dev(3, 2, 64, dtype=F32)), {}),
                     ((x, dev(3, 2, 64, cls=Elsewhere)), {}), ((x, None, dev(32)), {}), ((x, None, dev(3, 64)), {}),
                     ((x, None, None, dev(64, dtype=F32)), {}), ((x, None, None, dev(64, cls=Elsewhere)), {}),
                     ((x, None, None, None, dev(3, dtype=F32)), {}), ((x, None, None, None, dev(3, 2, 64, dtype=F32)), {}),
                     ((x, None, None, None, dev(3, 2)), {}), ((x, None, None, None, dev(3, 2, dtype=F32, cls=Elsewhere)), {}),
                     ((x, None, None, None, g), dict(gate_act="tanh")), ((x,), dict(out_format="fp4")),
                     ((x,), dict(out_format="both", q_format="fp4")), ((x,), dict(out=dev(3, 64))),
                     ((x,), dict(residual_out=dev(3, 2, 64, dtype=F32))), ((x,), dict(xq=dev(3, 2, 64, dtype=I8T))),
                     ((x,), dict(out_format="int8", out=dev(3, 2, 64))),
                     ((x,), dict(out_format="int8", xq=dev(3, 2, 64, dtype=U8))),
                     ((x,), dict(out_format="int8", xq=dev(3, 2, 64, dtype=I8T), xs=dev(3, 2, 2, dtype=U8))),
                     ((x,), dict(out_format="none", out=dev(3, 2, 64))),
                     ((x,), dict(out=dev(3, 2, 64, cls=Elsewhere)))):
        with pytest.raises(ValueError):
            E.post_pre_norm(*args, **{**({} if "out_format" in kw else outs), **kw})

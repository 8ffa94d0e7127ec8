"""The residual RMS norm and the MXFP4 / MXFP8-activation projections without
a GPU: the oracle's new functions against worked values, and every refusal of
the entry points (all answered before any launch)."""

from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import engram_oracle as o

OK, INV, UNS, NOSPACE = 0, 1, 2, 4
P = 0x1000


@pytest.fixture(scope="module")
def lib():
    from gram_memory_layer_engram_amd import build, engram

    if not os.path.exists(engram.LIB_PATH):
        build.build()
    return engram.load_library()


def test_e2m1_values_and_packing():
    assert o.e2m1_decode(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    codes = np.zeros((2, 32), dtype=np.uint8)
    codes[0, 0] = 0x72          # k 0: code 2 (1.0), k 1: code 7 (6.0)
    codes[1, 16] = 0xF1         # k 32: 0.5, k 33: -6.0
    scales = np.array([[128, 127], [127, 125]], dtype=np.uint8)
    w = o.mxfp4_dequantize_weight(codes, scales)
    assert w.shape == (2, 64) and w[0, 0] == 2.0 and w[0, 1] == 12.0
    assert w[1, 32] == 0.125 and w[1, 33] == -1.5 and np.count_nonzero(w) == 4


def test_oracle_norm_closed_forms():
    ones = o.round_to_bf16(np.ones((1, 2, 64)))
    s, y = o.add_rms_norm(ones, ones, None, 0.0)
    assert np.all(s == 2) and np.allclose(y, 1, rtol=1e-15)
    w = o.round_to_bf16(np.array([1.0, 3.0])[:, None] * np.ones((2, 64)))
    _, y = o.add_rms_norm(ones, None, w, 0.0)
    assert np.all(y[0, 0] == 1) and np.all(y[0, 1] == 3)
    _, y = o.add_rms_norm(o.round_to_bf16(np.zeros((1, 1, 8))), None, None, 1e-6)
    assert np.all(y == 0)


def norm(lib, x=P, xst=128, xsh=64, r=2 * P, rst=128, rsh=64, w=3 * P, whc=2, T=4, hc=2, dim=64, eps=1e-6, ro=4 * P,
         out=5 * P, xq=6 * P, xs=7 * P):
    return lib.engram_add_rms_norm(x, xst, xsh, r, rst, rsh, w, whc, T, hc, dim, eps, ro, out, xq, xs, None)


def test_add_rms_norm_refusals(lib):
    assert norm(lib, T=0, x=None, r=None, w=None, ro=None, out=None, xq=None, xs=None) == OK
    for bad in (dict(T=-1), dict(hc=0), dict(dim=0), dict(eps=-1e-6), dict(eps=float("nan")), dict(x=None),
                dict(xst=-8), dict(xsh=-8), dict(rst=-8), dict(rsh=-8), dict(whc=3), dict(whc=0), dict(xq=None),
                dict(xs=None), dict(out=None, xq=None, xs=None), dict(x=P + 2), dict(r=P + 8), dict(w=P + 4),
                dict(ro=P + 2), dict(out=P + 2), dict(xq=P + 8)):
        assert norm(lib, **bad) == INV, bad
    for bad in (dict(dim=60), dict(dim=72), dict(dim=16416), dict(xst=129), dict(rsh=4), dict(T=2**31 // 2)):
        assert norm(lib, **bad) == UNS, bad
    # in place on rows that are not dense, and any other overlap with an output (a tensor is 1 KiB of bf16)
    assert norm(lib, ro=2 * P + 16) == INV and norm(lib, out=P + 512) == INV       # shifted on its own input
    assert norm(lib, ro=P) == INV and norm(lib, out=2 * P) == INV                  # on the other input
    assert norm(lib, out=3 * P) == INV and norm(lib, xs=3 * P + 255) == INV        # on the weight
    assert norm(lib, xq=5 * P + 1008) == INV and norm(lib, xs=6 * P + 511) == INV  # on another output
    assert norm(lib, out=P + 1536, xst=512) == INV                                 # inside a strided input's range
    R, O = 0x20000, 0x30000
    assert norm(lib, r=R, ro=R, rst=256, out=O) == INV
    assert norm(lib, r=R, ro=R, rsh=0, rst=64, out=O) == INV
    assert norm(lib, x=O, out=O, xst=136, ro=None) == INV
    assert norm(lib, x=O, out=O, xsh=0, xst=64, ro=None) == INV
    assert norm(lib, out=O, ro=O) == INV
    assert norm(lib, T=0, dim=72, xq=None, xs=None) == OK   # bf16 output: dim % 8


def test_mxfp4_projection_refusals(lib):
    F4, F8, BF = 2, 1, 0
    big = 1 << 40

    X, W, S, V, Y = (i << 24 for i in range(1, 6))     # apart: x, w, its scales, kv, x's scales

    def wkv(T=4, K=256, N=64, x=X, w=W, s=S, kv=V, ws=P, nbytes=big):
        return lib.engram_wkv(x, T, K, w, s, F4, N, kv, ws, nbytes, None)

    assert wkv(T=0, x=None, w=None, s=None, kv=None, ws=None, nbytes=0) == OK
    for bad in (dict(T=-1), dict(K=0), dict(N=0), dict(x=None), dict(w=None), dict(s=None), dict(kv=None),
                dict(x=X + 2), dict(w=W + 8), dict(s=S + 1), dict(s=S + 4), dict(kv=V + 2),
                # kv (512 bytes) on x (2048), w (8192) or its scales (512)
                dict(kv=X), dict(kv=X + 2032), dict(kv=X - 496), dict(kv=W + 8176), dict(kv=S + 496), dict(kv=S - 496)):
        assert wkv(**bad) == INV, bad
    for bad in (dict(K=192), dict(K=1 << 21), dict(N=66), dict(N=(1 << 28) + 4)):
        assert wkv(**bad) == UNS, bad
    # no workspace: the codes are multiplied as they are
    for T, K in ((0, 256), (64, 384), (300, 256), (300, 384)):
        assert lib.engram_wkv_workspace_size(T, K, 64, F4) == 0

    def mx(T=4, K=256, N=64, xq=X, xs=Y, w=W, s=S, f=F4, kv=V):
        return lib.engram_wkv_mx(xq, xs, T, K, w, s, f, N, kv, None)

    for f in (F4, F8):
        assert mx(f=f, T=0, xq=None, xs=None, w=None, s=None, kv=None) == OK
        for bad in (dict(T=-1), dict(K=0), dict(N=0), dict(xq=None), dict(xs=None), dict(w=None), dict(s=None),
                    dict(kv=None), dict(xq=X + 8), dict(xs=Y + 4), dict(w=W + 8), dict(s=S + 1), dict(kv=V + 2),
                    # kv on the codes (1024 bytes), x's scales (32), w (8192 at least), its scales (16 at least)
                    dict(kv=X + 1008), dict(kv=Y + 16), dict(kv=Y - 496), dict(kv=W + 8176), dict(kv=S)):
            assert mx(f=f, **bad) == INV, (f, bad)
        assert mx(f=f, K=192) == UNS and mx(f=f, N=66) == UNS
    assert mx(f=F8, N=36) == UNS
    assert mx(f=BF, s=None) == UNS
    assert mx(f=7) == INV


def test_forward_mxfp4_refusals_and_workspace(lib):
    from gram_memory_layer_engram_amd import engram

    a = engram.ForwardArgs()
    a.T, a.hc, a.dim, a.n_cols, a.head_dim = 500, 4, 4096, 3, 128
    a.w_format = engram.W_BF16
    plain = lib.engram_forward_workspace_size(ctypes.byref(a))
    a.w_format = engram.W_MXFP4
    assert lib.engram_forward_workspace_size(ctypes.byref(a)) == plain
    # rows and kv of that many tokens do not fit the fixed scratch
    a.table = a.hash_ids = a.w = a.w_scales = a.hidden = a.q_weight = a.k_weight = a.out = P
    a.T, a.num_rows, a.ids_stride_t, a.ids_stride_c = 50000, 10, 16, 1
    assert lib.engram_forward_noalloc(ctypes.byref(a), None) == NOSPACE
    # one launch: MXFP8 weights only
    a.T = 16
    assert lib.engram_forward_single_launch(ctypes.byref(a), P, 1 << 40, None) == UNS
    a.w_scales = None
    assert lib.engram_forward(ctypes.byref(a), P, 1 << 40, None) == INV


def test_binding_refuses_host_tensors_and_wrong_shapes():
    from gram_memory_layer_engram_amd import engram as E

    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        E.add_rms_norm(x)
    with pytest.raises(ValueError, match="device tensors"):
        E.wkv_mx(torch.zeros((2, 128), dtype=torch.uint8), torch.zeros((2, 4), dtype=torch.uint8),
                 torch.zeros((32, 64), dtype=torch.uint8), torch.zeros((32, 4), dtype=torch.uint8))
    with pytest.raises(ValueError):
        E.add_rms_norm(torch.zeros((64,), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="MXFP4"):
        E.wkv(torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((32, 64), dtype=torch.uint8),
              torch.zeros((1, 4), dtype=torch.uint8))

"""What the binding refuses before it calls the library, on stand-in tensors (CPU
only): a weight that is not of the shape the forward will read."""

from __future__ import annotations

import os

import pytest
import torch

from gram_memory_layer_engram_amd import build, engram as E

BF, U8 = torch.bfloat16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(E.LIB_PATH):
        build.build()
    E.load_library()


class OnDevice(torch.Tensor):
    """Host memory that says it is a device tensor's: for calls that have to
    be refused, or that only fill a struct."""

    is_cuda = True

    def get_device(self):
        return 0


def dev(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


T, HC, DIM, C, HD = 3, 2, 64, 4, 64
K, N = C * HD, (HC + 1) * DIM


def forward_args(w, w_scales):
    return E.forward_args(dev(10, HD), dev(T, C, dtype=torch.int32), w, w_scales, dev(T, HC, DIM), dev(HC, DIM),
                          dev(HC, DIM), None, 1e-6, 1e-6, dev(T, HC, DIM))


def test_forward_takes_each_weight_format():
    assert forward_args(dev(N, K), None).w_format == E.W_BF16
    assert forward_args(dev(N, K, dtype=U8), dev(N // 32, K // 32, dtype=U8)).w_format == E.W_MXFP8
    codes = dev(N, K, dtype=U8).view(torch.float8_e4m3fn)
    assert forward_args(codes, dev(N // 32, K // 32, dtype=U8)).w_format == E.W_MXFP8
    assert forward_args(dev(N, K // 2, dtype=U8), dev(N, K // 32, dtype=U8)).w_format == E.W_MXFP4


@pytest.mark.parametrize("w,s", [
    # MXFP4: fewer rows than the forward reads, with scales of its own rows and of all
    ((N - 32, K // 2), (N - 32, K // 32)), ((N - 32, K // 2), (N, K // 32)), ((N, K // 2), (N - 4, K // 32)),
    # packed for another column count: not MXFP8 codes either
    ((N, K // 2 + 64), (N, K // 32)), ((N, K // 4), (N, K // 64)), ((N, K), (N, K // 32)),
    # MXFP8: too few rows, scales of too few blocks
    ((N - 32, K), (N // 32 - 1, K // 32)), ((N - 32, K), (N // 32, K // 32)), ((N, K), (N // 32 - 1, K // 32)),
    ((N, K - 128), (N // 32, (K - 128) // 32)), ((N * K,), (N // 32, K // 32))])
def test_forward_refuses_a_weight_of_another_shape(w, s):
    with pytest.raises(ValueError, match="w must be|scales"):
        forward_args(dev(*w, dtype=U8), dev(*s, dtype=U8))


def test_forward_refuses_other_element_sizes_and_strided_scales():
    with pytest.raises(ValueError, match="w must be"):
        forward_args(dev(N, K, dtype=U8), None)            # codes without scales
    with pytest.raises(ValueError, match="w must be"):
        forward_args(dev(N - 1, K), None)
    with pytest.raises(ValueError, match="scales|w must be"):
        forward_args(dev(N, K), dev(N // 32, K // 32, dtype=U8))
    with pytest.raises(ValueError, match="scales"):
        forward_args(dev(N, K, dtype=U8), dev(N // 32, 2 * K // 32, dtype=U8)[:, ::2])
    with pytest.raises(ValueError, match="scales"):
        forward_args(dev(N, K // 2, dtype=U8), dev(N, 2 * K // 32, dtype=U8)[:, ::2])


def test_gate_partials_refuses_scales_of_another_shape():
    D = 256
    n = (HC + 1) * D
    args = (dev(T, HC, D), dev(HC, D), dev(HC, D))
    for w, s in (((n, K), (n // 32 - 1, K // 32)), ((n, K), (n // 32, K // 32 - 1)), ((n, K // 2), (n - 4, K // 32)),
                 ((n - 32, K // 2), (n - 32, K // 32))):
        with pytest.raises(ValueError, match="w must be|scales"):
            E.wkv_gate_partials(dev(T, K), dev(*w, dtype=U8), dev(*s, dtype=U8), *args)

"""Inputs whose products and sums are exact in fp32 in every order, so that a
kernel's kv has to equal the reference bit for bit whatever K is, and the shapes
that are tested with them.

Weights: every e2m1 code (multiples of 0.5, at most 6) at scales 1/2 and 1;
activations +-1, in MXFP8 at scales 1/2, 1 and 2. A product is a multiple of u
(1/4 with bf16 activations, 1/8 with MXFP8) of at most m (6, 12), so a sum of K is
a multiple of u below K * m, exact where K * m / u < 2^24: K < 699,050 and K <
174,762. The 8-bit matrix instructions' window of 14 bits below the largest of 8
products holds all of them as well (m / u = 96 at most)."""

from __future__ import annotations

import torch

# (T, K, N) with bf16 or MXFP8 activations and MXFP4 weights: K past what LDS holds
# scale bytes for, both sides of that, and a wide N where fewer row tiles fit
LONG_K = [(1, 32768, 36), (20, 32768, 36), (50, 36864, 20), (40, 131072, 32), (3, 163840, 8), (64, 131072 + 128, 4),
          (40, 35840, 36), (40, 35968, 36), (64, 35840, 20), (64, 35968, 20), (16, 65536, 52), (90, 32896, 132),
          (20, 24576, 20476), (48, 30592, 16380), (64, 32768, 20476), (33, 8192, 12292)]
# row tiles of a workgroup: 1 to 5 on 256 compute units, a part tile at the end
WIDE_N = [4100, 6148, 8188, 10236, 12292, 16380, 20476]
WIDE_K = [512, 4096]     # 4096: the swapped scale pieces
WIDE_T = [1, 16, 17, 32, 33, 48, 49, 64]
# MXFP8 activations and weights: scale bytes of an odd number of 8-byte rows
ODD_SCALES = [(T, 256, N) for T in (17, 19, 33, 47, 63) for N in (160, 1280)]


def generator(seed, device):
    return torch.Generator(device=device).manual_seed(seed)


def mxfp4_weight(n, k, gen):
    """(codes [n, k/2], scale bytes [n, k/32])."""
    dev = gen.device
    return (torch.randint(0, 256, (n, k // 2), generator=gen, device=dev, dtype=torch.uint8),
            torch.randint(126, 128, (n, k // 32), generator=gen, device=dev, dtype=torch.uint8))


def mxfp8_weight(n, k, gen):
    """(e4m3 codes of +-1/2, +-1, +-2 and +-3 [n, k], scale bytes [n/32, k/32])."""
    dev = gen.device
    codes = torch.tensor([0x30, 0x38, 0x40, 0x44, 0xB0, 0xB8, 0xC0, 0xC4], dtype=torch.uint8, device=dev)
    return (codes[torch.randint(0, 8, (n, k), generator=gen, device=dev)],
            torch.randint(126, 128, (n // 32, k // 32), generator=gen, device=dev, dtype=torch.uint8))


def bf16_rows(t, k, gen):
    return (1 - 2 * torch.randint(0, 2, (t, k), generator=gen, device=gen.device)).to(torch.bfloat16)


def mxfp8_rows(t, k, gen):
    dev = gen.device
    codes = (0x38 | (torch.randint(0, 2, (t, k), generator=gen, device=dev) << 7)).to(torch.uint8)
    return codes, torch.randint(126, 129, (t, k // 32), generator=gen, device=dev, dtype=torch.uint8)


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def mxfp4_values(codes, scales):
    """In 64 bits, from the formats' definition."""
    lut = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    w = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], dim=-1).view(codes.shape[0], -1)
    return w * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def e4m3_values(codes):
    b = codes.int()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))
    return torch.where(b >= 128, -v, v)


def mxfp8_row_values(codes, scales):
    return e4m3_values(codes) * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def mxfp8_weight_values(codes, scales):
    return e4m3_values(codes) * torch.exp2(scales.double() - 127).repeat_interleave(32, 0).repeat_interleave(32, 1)


def product(x, w):
    """bf16(x . w^T) of 64-bit values whose sums are exact: one rounding (the
    sums are exact in fp32, too)."""
    ref = torch.mm(w, x.t().contiguous()).t()
    assert torch.equal(ref, ref.float().double())
    return ref.float().to(torch.bfloat16).contiguous()

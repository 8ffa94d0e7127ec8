"""Cases for the operators around the memory layer's projections, with their plain forms.

* ``add_rms_norm``: residual addition + root-mean-square norm of the streams
  ``[T, hc, dim]``, output bf16 or MXFP8 (e4m3 codes and one E8M0 byte per 32
  elements).
* ``wkv`` with MXFP4 weights (e2m1 codes, two per byte, low nibble first, one
  E8M0 byte per row and 32 k): products of bf16 activations.
* ``wkv_mx``: products of activations that are MXFP8 already (the norm's 8-bit
  output), with MXFP4 weights or MXFP8 weights (one E8M0 byte per 32x32).

With ``own`` false ``run`` is elementary torch in 32 bits, rounded once at the
end; with ``own`` true it makes the framework's calls. Codes come back as
float8_e4m3fn and scale bytes as float8_e8m0fnu: the values they stand for.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoded token's four residual streams, codes for the next projection: latency only
        {"name": "norm decode T1 mxfp8", "op": "norm", "T": 1, "hc": 4, "dim": 4096, "fmt": "mxfp8",
         "residual": True, "bcast": False, "pad": 0},
        # a ragged batch, one stream, rows cut out of a wider tensor (a slice of a projection's output)
        {"name": "norm ragged T1037 bf16", "op": "norm", "T": 1037, "hc": 1, "dim": 7168, "fmt": "bf16",
         "residual": True, "bcast": False, "pad": 64},
        # prefill: one branch output added to each of the four streams, per-stream weights
        {"name": "norm prefill T8192 mxfp8", "op": "norm", "T": 8192, "hc": 4, "dim": 4096, "fmt": "mxfp8",
         "residual": True, "bcast": True, "pad": 0},
        # 4-bit weights at the decode layer's projection: one token, a small batch, a full small batch
        {"name": "w4 decode T1", "op": "wkv", "T": 1, "N": 20480, "K": 2048},
        {"name": "w4 decode T16", "op": "wkv", "T": 16, "N": 20480, "K": 2048},
        {"name": "w4 decode T61", "op": "wkv", "T": 61, "N": 20480, "K": 2048},
        # a small layer's prompt, ragged
        {"name": "w4 prompt T515", "op": "wkv", "T": 515, "N": 10240, "K": 1024},
        # the prefill projection
        {"name": "w4 prefill T8192", "op": "wkv", "T": 8192, "N": 20480, "K": 2048},
        # products from the norm's codes: decode with 4-bit weights, with 8-bit weights, and prompts
        {"name": "mx w4 decode T4", "op": "wkv_mx", "w": "mxfp4", "T": 4, "N": 20480, "K": 2048},
        {"name": "mx w8 decode T16", "op": "wkv_mx", "w": "mxfp8", "T": 16, "N": 20480, "K": 2048},
        {"name": "mx w4 prompt T1000", "op": "wkv_mx", "w": "mxfp4", "T": 1000, "N": 20480, "K": 4096},
        {"name": "mx w8 prefill T4096", "op": "wkv_mx", "w": "mxfp8", "T": 4096, "N": 20480, "K": 2048},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "wkv", "wkv_mx"])
    if op == "norm":
        fmt = rng.choice(["bf16", "mxfp8"])
        step = 8 if fmt == "bf16" else 32
        dim = step * _log_int(rng, 64 // step, 16384 // step)
        hc = rng.choice([1, 2, 3, 4, 8])
        T = _log_int(rng, 1, max(1, min(8192, (8192 * 4 * 4096) // (hc * dim))))
        return {"op": "norm", "T": T, "hc": hc, "dim": dim, "fmt": fmt, "residual": rng.random() < 0.8,
                "bcast": rng.random() < 0.3, "pad": rng.choice([0, 0, 8, 64])}
    K = 128 * _log_int(rng, 2, 32)
    N = 32 * _log_int(rng, 8, 640)
    T = _log_int(rng, 1, 8192)
    if op == "wkv":
        return {"op": "wkv", "T": T, "N": N, "K": min(K, 2048)}
    return {"op": "wkv_mx", "w": rng.choice(["mxfp4", "mxfp8"]), "T": T, "N": N, "K": min(K, 2048)}


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        hc, dim = case["hc"], case["dim"]
        n = T * hc * dim
        rows_x = T if case["bcast"] else T * hc
        out = 2 * n if case["fmt"] == "bf16" else n + n // 32
        res = 4 * n if case["residual"] else 0          # residual in, residual out
        return {"bytes": 2 * rows_x * dim + res + out + 2 * hc * dim, "flops": 6 * n}
    N, K = case["N"], case["K"]
    w4 = case["op"] == "wkv" or case["w"] == "mxfp4"
    w = N * K // 2 + N * K // 32 if w4 else N * K + (N // 32) * (K // 32)
    x = 2 * T * K if case["op"] == "wkv" else T * K + T * K // 32
    return {"bytes": w + x + 2 * T * N, "flops": 2 * T * N * K}


# ----------------------------------------------------------------- inputs --

def _mx_scale_bytes(amax, top):
    """E8M0 byte of a block with largest magnitude amax, top = floor(log2(format's largest))."""
    e = torch.frexp(amax.float())[1] - 1                # floor(log2), exact
    return torch.where(amax > 0, (e - top + 127).clamp(0, 254), torch.zeros_like(e))


def _pow2(byte):
    """2^(127 - byte), the factor that takes a block to its codes' range, for byte <= 246."""
    return ((254 - byte.to(torch.int32)) << 23).view(torch.float32)


def _make_mxfp4(n, k, gen, std):
    """Weights N(0, std) in MXFP4: (codes [n, k/2], bytes [n, k/32])."""
    w = torch.randn((n, k // 32, 32), generator=gen, device=DEV) * std
    byte = _mx_scale_bytes(w.abs().amax(-1), 2)
    v = w * _pow2(byte).unsqueeze(-1)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(v.abs(), edges).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    code = code.view(n, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte.to(torch.uint8)


def _make_mxfp8_rows(t, k, gen):
    """Activations of unit size with a few large channels, in MXFP8 rows."""
    x = torch.randn((t, k), generator=gen, device=DEV)
    x = x * (1 + 9 * (torch.rand((1, k), generator=gen, device=DEV) < 0.01))
    x = x.view(t, k // 32, 32)
    byte = _mx_scale_bytes(x.abs().amax(-1), 8)
    code = (x * _pow2(byte).unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return code.view(torch.uint8).view(t, k), byte.to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T = case["T"]
    st = {"case": case}
    if case["op"] == "norm":
        hc, dim, pad = case["hc"], case["dim"], case["pad"]
        # a few channels of a residual stream are much larger than the rest
        big = 1 + 29 * (torch.rand((dim,), generator=g, device=DEV) < 0.005)
        xh = 1 if case["bcast"] else hc
        x = torch.randn((T, xh, dim + pad), generator=g, device=DEV)
        x[..., :dim] *= big
        x = x.to(torch.bfloat16)[..., :dim]             # rows of a wider tensor where pad > 0
        st["x"] = x.expand(T, hc, dim)
        st["r"] = None
        if case["residual"]:
            st["r"] = (2 * torch.randn((T, hc, dim), generator=g, device=DEV) * big).to(torch.bfloat16)
        st["w"] = (1 + 0.1 * torch.randn((hc, dim), generator=g, device=DEV)).to(torch.bfloat16)
        return st
    N, K = case["N"], case["K"]
    if case["op"] == "wkv":
        st["x"] = torch.randn((T, K), generator=g, device=DEV).to(torch.bfloat16)
        st["w"], st["s"] = _make_mxfp4(N, K, g, 0.02)
        return st
    st["xq"], st["xs"] = _make_mxfp8_rows(T, K, g)
    if case["w"] == "mxfp4":
        st["w"], st["s"] = _make_mxfp4(N, K, g, 0.02)
    else:
        st["w"] = torch.randn((N, K), generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
        st["s"] = (127 + torch.randint(-8, 1, (N // 32, K // 32), generator=g, device=DEV)).to(torch.uint8)
    return st


# -------------------------------------------------------------- plain form --

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _e8m0(byte):
    return byte.view(torch.float8_e8m0fnu).float()


def _plain_weight(st, N, K):
    w, s = st["w"], st["s"]
    if w.shape[1] == K // 2:
        lut = torch.tensor(_E2M1, device=w.device)
        code = torch.stack([w & 15, w >> 4], -1).view(N, K // 32, 32)
        return (lut[code.int()] * _e8m0(s).unsqueeze(-1)).view(N, K)
    v = w.view(torch.float8_e4m3fn).float().view(N // 32, 32, K // 32, 32)
    return (v * _e8m0(s).view(N // 32, 1, K // 32, 1)).view(N, K)


def _plain_norm(st):
    c, x, r = st["case"], st["x"], st["r"]
    s = x.float() if r is None else x.float() + r.float()
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * st["w"].float()
    out = {} if r is None else {"residual": s.to(torch.bfloat16)}
    if c["fmt"] == "bf16":
        out["out"] = y.to(torch.bfloat16)
        return out
    b = y.view(c["T"], c["hc"], c["dim"] // 32, 32)
    byte = _mx_scale_bytes(b.abs().amax(-1), 8)
    v = (b * _pow2(byte).unsqueeze(-1)).clamp(-448, 448)
    out["codes"] = v.to(torch.float8_e4m3fn).view(y.shape)
    out["scales"] = byte.to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def run(state):
    c = state["case"]
    if own:
        from gram_memory_layer_engram_amd import engram as E
        if c["op"] == "norm":
            res, out, xq, xs = E.add_rms_norm(state["x"], state["r"], state["w"], EPS, out_format=c["fmt"])
            got = {} if res is None else {"residual": res}
            if c["fmt"] == "bf16":
                got["out"] = out
            else:
                got["codes"] = xq.view(torch.float8_e4m3fn)
                got["scales"] = xs.view(torch.float8_e8m0fnu)
            return got
        if c["op"] == "wkv":
            return {"kv": E.wkv(state["x"], state["w"], state["s"])}
        return {"kv": E.wkv_mx(state["xq"], state["xs"], state["w"], state["s"])}
    if c["op"] == "norm":
        return _plain_norm(state)
    N, K, T = c["N"], c["K"], c["T"]
    if c["op"] == "wkv":
        x = state["x"].float()
    else:
        x = state["xq"].view(torch.float8_e4m3fn).float().view(T, K // 32, 32)
        x = (x * _e8m0(state["xs"]).unsqueeze(-1)).view(T, K)
    return {"kv": (x @ _plain_weight(state, N, K).t()).to(torch.bfloat16)}


# ------------------------------------------------------------------- exact --

def _round_to_steps(v, step):
    """v to the nearest multiple of step, ties to even (torch.round's rule)."""
    return torch.round(v / step) * step


def _exact_e8m0(byte):
    return torch.exp2(byte.double() - 127)


def _exact_e4m3(byte):
    b = byte.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e.double() - 7) * (1 + m / 8))
    return torch.where(b >= 128, -v, v)


def _exact_e2m1(nibble):
    b = nibble.long()
    e, m = (b >> 1) & 3, (b & 1).double()
    v = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2))
    return torch.where(b >= 8, -v, v)


def _exact_norm(st):
    """The norm in 64 bits; the MX rule on the exact values: shared exponent
    floor(log2 max) - 8, codes to the nearest e4m3 (3 fraction bits, least
    step 2^-9), ties to even, at most 448."""
    c = st["case"]
    s = st["x"].double()
    out = {}
    if st["r"] is not None:
        s = s + st["r"].double()
        out["residual"] = s
    y = s / torch.sqrt((s * s).sum(-1, keepdim=True) / c["dim"] + EPS) * st["w"].double()
    if c["fmt"] == "bf16":
        out["out"] = y
        return out
    b = y.reshape(-1, 32)
    top = b.abs().amax(-1, keepdim=True)
    shared = torch.where(top > 0, torch.floor(torch.log2(top)) - 8, torch.full_like(top, -127.0)).clamp(-127, 127)
    v = b / torch.exp2(shared)
    mag = v.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(mag)) - 3)
    out["codes"] = _round_to_steps(v, step).clamp(-448, 448).reshape(y.shape)
    out["scales"] = torch.exp2(shared).reshape(c["T"], c["hc"], c["dim"] // 32)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    T, N, K = case["T"], case["N"], case["K"]
    if case["op"] == "wkv":
        x = st["x"].double()
    else:
        x = _exact_e4m3(st["xq"]) * _exact_e8m0(st["xs"]).repeat_interleave(32, 1)
    if st["w"].shape[1] == K // 2:
        w = torch.empty((N, K), dtype=torch.float64, device=DEV)
        w[:, 0::2] = _exact_e2m1(st["w"] & 15)
        w[:, 1::2] = _exact_e2m1(st["w"] >> 4)
        w *= _exact_e8m0(st["s"]).repeat_interleave(32, 1)
    else:
        w = _exact_e4m3(st["w"]) * _exact_e8m0(st["s"]).repeat_interleave(32, 0).repeat_interleave(32, 1)
    return {"kv": torch.matmul(x, w.t())}

"""GPU: calls of the int8 products and of the norms around a block."""

from __future__ import annotations

import sys

import pytest
import torch

from tests._threads import run_together

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


def _int8_weight(g, N, K):
    return (torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8),
            torch.rand((N,), generator=g, device=DEV) * 2.0 ** -10 + 2.0 ** -11)


def _forward_case(T, dim, hc, C, hd, rows=5000, seed=3):
    g = torch.Generator(device=DEV).manual_seed(seed + T)
    bf = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)   # noqa: E731
    w, ws = _int8_weight(g, (hc + 1) * dim, C * hd)
    ids = torch.randint(0, rows, (T, C), generator=g, device=DEV, dtype=torch.int32)
    return bf(rows, hd), ids, w, ws, bf(T, hc, dim), bf(hc, dim), bf(hc, dim)


@pytest.mark.parametrize("T,dim,hc,C,hd", [(1, 512, 4, 8, 64), (70, 512, 2, 8, 64), (300, 512, 2, 9, 112), (770, 4096, 4, 16, 128)])
@pytest.mark.parametrize("store_kv", [False, True])
def test_forward_noalloc_and_a_workspace_of_the_stated_size(T, dim, hc, C, hd, store_kv):
    """A caller's workspace of engram_forward_workspace_size bytes, full of garbage behind
    its flags, and the library's own scratch give what a fresh workspace gives (with kv
    stored: what the single calls give); nothing past the workspace is written."""
    E = _E()
    _say(f"noalloc int8 {T} {dim} {hc} {C} {hd} {store_kv}")
    c = _forward_case(T, dim, hc, C, hd)
    table, ids, w, ws, hidden, q, k = c
    xq, xs = E.int8_quantize(table[ids.long()].reshape(T, C * hd))
    kv = E.wkv_int8(xq, xs, w, ws)
    want = E.gate(hidden, kv, q, k)
    a = E.forward_args(table, ids, w, ws, hidden, q, k, None, 1e-6, 1e-6, hidden, store_kv=store_kv)
    need = E.forward_workspace_size(a)
    room = torch.full((need + 4096,), 0x7f, dtype=torch.uint8, device=DEV)
    room[:65536] = 0
    out = E.forward(*c, workspace=room[:need], store_kv=store_kv)
    assert bool((room[need:] == 0x7f).all()) and not bool(room[:65536].any())
    assert torch.equal(out, E.forward(*c, store_kv=store_kv))
    assert not store_kv or torch.equal(out, want)
    assert torch.equal(E.forward_noalloc(*c, store_kv=store_kv), out)


def test_two_threads_both_end_with_the_serial_results():
    """Norms, both products and the quantizer of two host threads at once, each on its own
    stream and of its own sizes: both threads come to their end, with the serial bits."""
    E = _E()
    work = []
    for T, dim, N in ((3, 1024, 4096), (150, 2064, 1280)):
        _say(f"threads {T} {dim} {N}")
        g = torch.Generator(device=DEV).manual_seed(T)
        x, r = (torch.randn((T, 2, dim), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
        gate = torch.rand((T, 2), generator=g, device=DEV)
        w, ws = _int8_weight(g, N, dim)

        def calls(x=x, r=r, gate=gate, w=w, ws=ws, n=2 * T, dim=dim):
            res, out, xq, xs = E.post_pre_norm(x, r, gate=gate, out_format="both", q_format="int8")
            rows = out.view(n, dim)
            return res, out, xq, xs, E.wkv_int8(xq.view(n, dim), xs.view(n), w, ws), E.wkv(rows, w, ws), *E.int8_quantize(rows)

        def thread(calls=calls, want=calls(), stream=torch.cuda.Stream()):
            with torch.cuda.stream(stream):
                got = [calls() for _ in range(60)]
                stream.synchronize()
                for i in got:
                    for a, b in zip(i, want):
                        assert torch.equal(a, b)

        work.append(thread)
    torch.cuda.synchronize()
    run_together(work)


@pytest.mark.parametrize("dim", [64, 2080, 4096, 16384])
def test_norms_of_rows_as_long_as_fp32_holds(dim):
    """A row's sum of squares is an fp32: up to 2^128 the norm of a row of one magnitude
    is 1 in bf16 (sums and root are off by at most dim / 128 + 11 half steps of 2^-24, far
    below the half step of 2^-9 under 1), past it 0, which is not NaN and reaches no other row."""
    E = _E()
    _say(f"long rows {dim}")
    limit = 2.0 ** 64 / dim ** 0.5
    sign = torch.ones((dim,), device=DEV)
    sign[::3] = -1
    rows = torch.tensor([0.9 * limit, 1.2 * limit, 1.0, -0.98 * limit, 3e38], device=DEV)   # bf16: within 2^-8
    x = (rows.view(-1, 1) * sign).to(torch.bfloat16)
    unit = torch.tensor([1.0, 0.0, 1.0, -1.0, 0.0], device=DEV).view(-1, 1) * sign
    two = torch.full_like(x, 2.0)
    # the norm after the block: the branch
    res, out, _, _ = E.post_pre_norm(x, two)
    assert torch.equal(res.float(), 2 + unit)
    # the norm before the next one, in every format
    kw = dict(post_norm=False)
    res, out, xq, xs = E.post_pre_norm(x, out_format="both", q_format="int8", **kw)
    assert torch.equal(res, x) and torch.equal(out.float(), unit)
    short = torch.tensor([True, False, True, True, False], device=DEV)
    assert bool((xs[~short] == 0).all())
    n = (dim / 128 + 16) * 2.0 ** -24
    assert bool(((xs[short].double() * 127 - 1).abs() <= n).all()) and torch.equal(xq[short].float(), 127 * unit[short])
    _, _, xq, xs = E.post_pre_norm(x, out_format="mxfp8", **kw)
    v = xq.view(torch.float8_e4m3fn).float() * xs.view(torch.float8_e8m0fnu).float().repeat_interleave(32, -1)
    # the MX rule: a largest of just under 1 has the exponent -1, the block scale 2^-9 and, of 512
    # steps, the code's largest, 448: 0.875; at 1 or above the scale is 2^-8, the code 256
    assert bool(((v == unit) | (v == 0.875 * unit)).all())
    _, out, _, _ = E.add_rms_norm(x)
    assert torch.equal(out.float(), unit)


def test_row_gate_sigmoid_error():
    """The sigmoid of a row's gate, read from the int8 rows' fp32 scales: with x = 1 (2^100
    below -40, to stay clear of subnormals) and eps = 2^112, which takes in s^2, the scale is
    sigmoid * x * 2^-56 / 127, the quotient's rounding the only one behind the sigmoid.

    Of a value: fl(z * log2 e) is off by half a step, 2^-21 below 16 and 2^-20 below 32, and
    by |z| * 2^-25.6 for log2 e; times ln 2 (z 11: 0.35 + 0.15, z 16: 0.69 + 0.23 of 2^-20);
    exp and reciprocal one step each (2^-23), the sum half (2^-24): 0.31 of 2^-20."""
    E = _E()
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.cat([(torch.rand((1 << 19,), generator=g, device=DEV) * 2 - 1) * top for top in (1, 11, 16, 80)]
                  + [torch.linspace(-16, -15, 1 << 18, device=DEV), torch.linspace(-11, -10, 1 << 18, device=DEV),
                     torch.arange(-80, 81, device=DEV) * 1.0])
    up = torch.where(z < -40, 2.0 ** 100, 1.0)
    x = up.view(-1, 1).expand(-1, 8).to(torch.bfloat16)
    _, _, _, xs = E.post_pre_norm(x, gate=z, gate_act="sigmoid", post_norm=False, eps=2.0 ** 112, out_format="int8")
    got = xs.double() * 127 * 2.0 ** 56 / up.double()
    want = 1 / (1 + torch.exp(-z.double()))
    err = (got - want).abs() / want
    for lo, hi, tol in ((0, 11, 2.0 ** -20), (11, 16, 2.0 ** -19), (16, 80, 2.0 ** -17)):
        m = (z.abs() >= lo) & (z.abs() <= hi)
        _say(f"sigmoid, |z| {lo} - {hi}: {float(err[m].max() * 2.0 ** 20):.3f} of 2^-20")
        assert float(err[m].max()) <= tol + 2.0 ** -24

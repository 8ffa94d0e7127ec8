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


class OnOther(OnDevice):
    """The same on a second device."""

    def get_device(self):
        return 1


def _layer(cls, fmt):
    d = lambda *shape, dtype=BF: torch.zeros(shape, dtype=dtype).as_subclass(cls)  # noqa: E731
    dim = 256
    n = (HC + 1) * dim
    w, s = {E.W_BF16: (d(n, K), None), E.W_MXFP8: (d(n, K, dtype=U8), d(n // 32, K // 32, dtype=U8)),
            E.W_MXFP4: (d(n, K // 2, dtype=U8), d(n, K // 32, dtype=U8))}[fmt]
    return dict(table=d(10, HD), hash_ids=d(T, C, dtype=torch.int32), w=w, w_scales=s, hidden=d(T, HC, dim),
                q_weight=d(HC, dim), k_weight=d(HC, dim), token_mask=d(T, dtype=torch.bool), out=d(T, HC, dim),
                gate_out=d(T, HC, dtype=torch.float32), err_flag=d(1, dtype=torch.int32))


def _partials(cls, fmt):
    a = _layer(cls, fmt)
    return dict(x=torch.zeros((T, K), dtype=BF).as_subclass(cls),
                value=torch.zeros((T, 256), dtype=BF).as_subclass(cls),
                partials=torch.zeros((HC, T, 1, 2)).as_subclass(cls),
                **{k: a[k] for k in ("w", "w_scales", "hidden", "q_weight", "k_weight")})


class _Recorder:
    """A stand-in for the library and torch's device context: which device was
    current at each call, and the stream it was given."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []
        outer = self

        class device:
            def __init__(self, i):
                self.i = i

            def __enter__(self):
                self.before, outer.current = outer.current, self.i

            def __exit__(self, *exc):
                outer.current = self.before

        class stream:
            def __init__(self, dev):
                self.cuda_stream = 100 + (outer.current if dev is None else dev)

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: stream(dev))
        monkeypatch.setattr(E, "_current_device", lambda: outer.current)
        monkeypatch.setattr(E, "_raw_stream", lambda dev: 100 + dev)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
        monkeypatch.setattr(E, "load_library", lambda: outer)
        monkeypatch.setattr(E, "_lib", outer)
        monkeypatch.setattr(E, "new_forward_workspace", lambda n, device: None)

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 0

        def call(*a):
            self.calls.append((name, self.current, getattr(a[-1], "value", a[-1])))
            return 0
        return call


FORWARDS = [("forward", "engram_forward"), ("forward_noalloc", "engram_forward_noalloc")]


@pytest.mark.parametrize("fmt", [E.W_BF16, E.W_MXFP8, E.W_MXFP4])
def test_forward_and_partials_run_on_their_tensors_device(fmt, monkeypatch):
    for cls, dev_index in ((OnDevice, 0), (OnOther, 1)):
        rec = _Recorder(monkeypatch)
        for fn, entry in FORWARDS:
            getattr(E, fn)(**_layer(cls, fmt))
            assert rec.calls.pop() == (entry, dev_index, 100 + dev_index)
        plan = E.ForwardPlan(**_layer(cls, fmt))
        for _ in range(2):
            plan.run()
            assert rec.calls.pop() == ("engram_forward", dev_index, 100 + dev_index)
        E.wkv_gate_partials(**_partials(cls, fmt))
        assert rec.calls.pop() == ("engram_wkv_gate_partials", dev_index, 100 + dev_index)
        assert rec.current == 0 and not rec.calls


@pytest.mark.parametrize("fmt", [E.W_BF16, E.W_MXFP8, E.W_MXFP4])
def test_forward_and_partials_refuse_tensors_on_two_devices(fmt, monkeypatch):
    rec = _Recorder(monkeypatch)
    for make, fns in ((_layer, [E.forward, E.forward_noalloc, E.ForwardPlan]), (_partials, [E.wkv_gate_partials])):
        for name, t in make(OnDevice, fmt).items():
            if t is None:
                continue
            for fn in fns:
                for other in (t.as_subclass(OnOther), t.as_subclass(torch.Tensor)):     # another device, host memory
                    with pytest.raises(ValueError, match="device"):
                        fn(**{**make(OnDevice, fmt), name: other})
    assert not rec.calls

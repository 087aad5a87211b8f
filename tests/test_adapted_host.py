"""The adapted layer's calls on the host (no GPU needed): the mask generator's
published values, the argument checks of the C calls with stand-in pointers,
and of the binding with CPU tensors."""
import ctypes

import numpy as np
import pytest
import torch

import adapted_ref as ref
import quantized_lora_fine_nf4_amd as q

FAKE = 0x7F0000000000  # 256-aligned stand-in address; no call below reaches the device
NAN = float("nan")


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0x4DFCCABA, 0x190A87F0, 0xC47362BA, 0xB6B5242A]),
], ids=["zeros", "ones", "pi"])
def test_generator_gives_the_published_words(counter, key, words):
    assert ref.philox4x32_7(counter, key) == words


def test_mask_lanes_follow_the_words():
    seed, off = 0x0123456789ABCDEF, 0x1122334455667788
    g = (5 << 32) + 77
    words = ref.philox4x32_7([g & 0xFFFFFFFF, g >> 32, off & 0xFFFFFFFF, off >> 32], [seed & 0xFFFFFFFF, seed >> 32])
    lanes = [h for w in words for h in (w & 0xFFFF, w >> 16)]
    p = sorted(lanes)[4] / 65536
    assert ref.keep(8 * g + np.arange(8), p, seed, off).tolist() == [l >= ref.threshold(p) for l in lanes]


def drop(p=0.0, rng=FAKE):
    return q.nf4_drop(rng, p)


def test_dropout_arguments():
    L = q.lib()

    def call(x=FAKE, n=100, dt=0, d=drop(0.5), out=FAKE):
        return L.nf4_dropout(x, n, dt, d, out, None)
    assert call(x=None) == q.NF4_E_ARG
    assert call(out=None) == q.NF4_E_ARG
    assert call(n=0) == q.NF4_E_ARG
    assert call(n=-1) == q.NF4_E_ARG
    assert call(n=1 << 36) == q.NF4_E_UNSUPPORTED
    assert call(dt=2) == q.NF4_E_UNSUPPORTED
    assert call(x=FAKE + 8) == q.NF4_E_ALIGN
    assert call(out=FAKE + 8) == q.NF4_E_ALIGN
    for p in (-0.1, 1.0, 1.5, NAN, 65535.5 / 65536):
        assert call(d=drop(p)) == q.NF4_E_ARG, p
    assert call(d=drop(0.5, None)) == q.NF4_E_ARG
    assert call(d=drop(0.5, FAKE + 4)) == q.NF4_E_ALIGN


def test_act_grad_arguments():
    L = q.lib()

    def call(dy=FAKE, z=FAKE, act=2, m=100, n=512, dt=0, dz=FAKE, db=FAKE, ws=FAKE, wsb=1 << 24):
        return L.nf4_act_grad(dy, z, act, m, n, dt, dz, db, ws, wsb, None)
    assert call(dy=None) == q.NF4_E_ARG
    assert call(z=None) == q.NF4_E_ARG
    assert call(dz=None) == q.NF4_E_ARG
    assert call(act=0, dz=None, db=None) == q.NF4_E_ARG
    assert call(act=5) == q.NF4_E_ARG
    assert call(act=-1) == q.NF4_E_ARG
    assert call(m=0) == q.NF4_E_ARG
    assert call(m=(1 << 25) + 1) == q.NF4_E_ARG
    assert call(n=0) == q.NF4_E_ARG
    assert call(n=1 << 26) == q.NF4_E_ARG
    assert call(n=12) == q.NF4_E_UNSUPPORTED
    assert call(dt=2) == q.NF4_E_UNSUPPORTED
    for k in ("dy", "z", "dz", "db"):
        assert call(**{k: FAKE + 8}) == q.NF4_E_ALIGN, k
    need = q.nf4_act_grad_workspace_bytes(100, 512)
    assert need > 0 and need % 256 == 0
    assert call(wsb=need - 1) == q.NF4_E_WORKSPACE
    assert call(ws=None) == q.NF4_E_WORKSPACE
    assert call(ws=FAKE + 16) == q.NF4_E_WORKSPACE
    assert q.nf4_act_grad_workspace_bytes(1, 512) == 0     # one block of tokens
    for m, n in ((0, 8), (1, 0), (1, 12), ((1 << 25) + 1, 8), (1, 1 << 26)):
        assert q.nf4_act_grad_workspace_bytes(m, n) == 0


def test_project_arguments():
    L = q.lib()

    def call(x=FAKE, m=10, k=256, w=FAKE, r=16, dt=0, bwd=0, d=drop(), h=FAKE):
        return L.nf4_lora_project(x, m, k, w, r, dt, bwd, 1.0, d, h, None)
    for k in ("x", "w", "h"):
        assert call(**{k: None}) == q.NF4_E_ARG, k
        assert call(**{k: FAKE + 8}) == q.NF4_E_ALIGN, k
    assert call(m=0) == q.NF4_E_ARG
    assert call(m=(1 << 25) + 1) == q.NF4_E_ARG
    assert call(k=0) == q.NF4_E_ARG
    assert call(k=1 << 26) == q.NF4_E_ARG
    assert call(k=100) == q.NF4_E_UNSUPPORTED
    assert call(r=0) == q.NF4_E_ARG
    assert call(r=-1) == q.NF4_E_ARG
    assert call(r=129) == q.NF4_E_UNSUPPORTED
    assert call(dt=2) == q.NF4_E_UNSUPPORTED
    assert call(bwd=2) == q.NF4_E_ARG
    assert call(d=drop(1.0)) == q.NF4_E_ARG
    assert call(d=drop(0.5, None)) == q.NF4_E_ARG
    assert call(d=drop(0.5), bwd=1) == q.NF4_E_UNSUPPORTED


def test_lora_grad_arguments():
    L = q.lib()

    def call(u=FAKE, x=FAKE, m=4000, n=256, r=16, dt=0, side=0, d=drop(), g=FAKE, ws=FAKE, wsb=1 << 26):
        return L.nf4_lora_grad(u, x, m, n, r, dt, side, d, g, ws, wsb, None)
    for k in ("u", "x", "g"):
        assert call(**{k: None}) == q.NF4_E_ARG, k
        assert call(**{k: FAKE + 8}) == q.NF4_E_ALIGN, k
    assert call(m=0) == q.NF4_E_ARG
    assert call(m=(1 << 25) + 1) == q.NF4_E_ARG
    assert call(n=0) == q.NF4_E_ARG
    assert call(n=1 << 26) == q.NF4_E_ARG
    assert call(n=100) == q.NF4_E_UNSUPPORTED
    assert call(r=0) == q.NF4_E_ARG
    assert call(r=129) == q.NF4_E_UNSUPPORTED
    assert call(dt=-1) == q.NF4_E_UNSUPPORTED
    assert call(side=2) == q.NF4_E_ARG
    assert call(d=drop(-1.0)) == q.NF4_E_ARG
    assert call(d=drop(0.5), side=1) == q.NF4_E_UNSUPPORTED
    need = q.nf4_lora_grad_workspace_bytes(4000, 256, 16)
    assert need > 0 and need % 256 == 0
    assert call(wsb=need - 1) == q.NF4_E_WORKSPACE
    assert call(ws=None) == q.NF4_E_WORKSPACE
    assert call(ws=FAKE + 16) == q.NF4_E_WORKSPACE
    assert q.nf4_lora_grad_workspace_bytes(1, 256, 16) == 0
    for m, n, r in ((0, 8, 1), (1, 12, 1), (1, 8, 0), (1, 8, 129)):
        assert q.nf4_lora_grad_workspace_bytes(m, n, r) == 0


def test_linear_arguments():
    L = q.lib()
    rows, cols, f = 256, 384, q.fmt()

    def call(m=10, backward=0, x=FAKE, out=FAKE, fmt=f, ws=FAKE, wsb=1 << 30, n=None, **kw):
        lay = q.nf4_layer(rows * cols if n is None else n, None, FAKE, None, FAKE, FAKE, None)
        a = dict(u=FAKE + 256, v=FAKE + 512, rank=16, act=0, drop=drop(), bias=None, residual=None, preact=None)
        a.update(kw)
        e = q.nf4_epilogue(**a)
        return L.nf4_linear(ctypes.byref(lay), rows, cols, fmt, backward, x, m, ctypes.byref(e), out, 0, ws, wsb, None)
    # nf4_matmul's checks
    assert call(m=0) == q.NF4_E_ARG
    assert call(x=None) == q.NF4_E_ARG
    assert call(out=FAKE + 8) == q.NF4_E_ALIGN
    assert call(n=5) == q.NF4_E_ARG
    assert call(fmt=q.nf4_format(0, 32, 256)) == q.NF4_E_UNSUPPORTED
    # the epilogue's
    assert call(u=None) == q.NF4_E_ARG
    assert call(v=None) == q.NF4_E_ARG
    assert call(rank=0) == q.NF4_E_ARG
    assert call(rank=-3) == q.NF4_E_ARG
    assert call(u=None, v=None, rank=8) == q.NF4_E_ARG
    assert call(rank=129) == q.NF4_E_UNSUPPORTED
    assert call(act=5) == q.NF4_E_ARG
    assert call(act=-1) == q.NF4_E_ARG
    for k in ("u", "v", "bias", "residual", "preact"):
        assert call(**{k: FAKE + 8}) == q.NF4_E_ALIGN, k
    assert call(preact=FAKE) == q.NF4_E_ARG                              # preact is out
    assert call(preact=FAKE + 1024, residual=FAKE + 1024) == q.NF4_E_ARG
    assert call(drop=drop(0.1)) == q.NF4_E_UNSUPPORTED                   # forward
    assert call(backward=1, act=1) == q.NF4_E_UNSUPPORTED
    assert call(backward=1, bias=FAKE + 1024) == q.NF4_E_UNSUPPORTED
    assert call(backward=1, preact=FAKE + 1024) == q.NF4_E_UNSUPPORTED
    assert call(backward=1, drop=drop(0.1, None)) == q.NF4_E_ARG
    assert call(backward=1, drop=drop(1.0)) == q.NF4_E_ARG
    assert call(backward=1, drop=drop(0.1), u=None, v=None, rank=0) == q.NF4_E_ARG
    need = q.nf4_matmul_workspace_bytes(rows, cols, False, 10)
    assert need > 0
    assert call(wsb=need - 1) == q.NF4_E_WORKSPACE
    assert call(ws=None) == q.NF4_E_WORKSPACE
    lay = q.nf4_layer(rows * cols, None, FAKE, None, FAKE, FAKE, None)
    assert L.nf4_linear(ctypes.byref(lay), rows, cols, f, 0, FAKE, 10, None, FAKE, 0, FAKE, 1 << 30,
                        None) == q.NF4_E_ARG


def _bad(fn, *a, **kw):
    with pytest.raises(q.NF4Error) as e:
        fn(*a, **kw)
    assert e.value.status == q.NF4_E_ARG
    return str(e.value)


def test_binding_checks_shapes_types_and_devices():
    """On CPU tensors: every misfit is refused before the library is called, and a call whose tensors all fit is
    refused for not being on the GPU."""
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f32 = lambda *s: torch.zeros(s)
    rng = torch.zeros(2, dtype=torch.int64)
    assert "GPU" in _bad(q.nf4_dropout, b(4, 8), b(4, 8), 0.1, rng)
    assert "out" in _bad(q.nf4_dropout, b(4, 8), b(4, 9), 0.1, rng)
    assert "x" in _bad(q.nf4_dropout, b(8, 4).t(), b(4, 8), 0.1, rng)
    assert "float32" in _bad(q.nf4_dropout, f32(4), f32(4), 0.1, rng)
    assert "rng" in _bad(q.nf4_dropout, b(4), b(4), 0.1, None)
    assert "rng" in _bad(q.nf4_dropout, b(4), b(4), 0.1, torch.zeros(3, dtype=torch.int64))
    assert "rng" in _bad(q.nf4_dropout, b(4), b(4), 0.1, torch.zeros(2, dtype=torch.int32))
    assert "rng" in _bad(q.nf4_dropout, b(4), b(4), 0.1, torch.zeros(2, dtype=torch.complex64))
    assert "rng" in _bad(q.nf4_dropout, b(4), b(4), 0.1, torch.zeros(2, dtype=torch.float64))
    assert "GPU" in _bad(q.nf4_act_grad, b(4, 8), b(4, 8), 1, b(4, 8))
    assert "preact" in _bad(q.nf4_act_grad, b(4, 8), b(4, 7), 1, b(4, 8))
    assert "dz" in _bad(q.nf4_act_grad, b(4, 8), b(4, 8), 1, f32(4, 8))
    assert "dbias" in _bad(q.nf4_act_grad, b(4, 8), b(4, 8), 1, b(4, 8), dbias=b(8))
    assert "dy" in _bad(q.nf4_act_grad, b(8), b(8), 1, b(8))
    assert "GPU" in _bad(q.nf4_lora_project, b(3, 8), b(5, 8), b(3, 5))
    assert "w" in _bad(q.nf4_lora_project, b(3, 8), b(5, 8), b(3, 5), backward=True)
    assert "h" in _bad(q.nf4_lora_project, b(3, 8), b(5, 8), b(5, 3))
    assert "w" in _bad(q.nf4_lora_project, b(3, 8), torch.zeros(5, 8, dtype=torch.float16), b(3, 5))
    assert "GPU" in _bad(q.nf4_lora_grad, b(3, 5), b(3, 8), f32(5, 8))
    assert "grad" in _bad(q.nf4_lora_grad, b(3, 5), b(3, 8), f32(5, 8), side="B")
    assert "u" in _bad(q.nf4_lora_grad, b(4, 5), b(3, 8), f32(5, 8))
    assert "side" in _bad(q.nf4_lora_grad, b(3, 5), b(3, 8), f32(5, 8), side="C")
    lay, f = q.nf4_layer(128 * 256, None, FAKE, None, FAKE, FAKE, None), q.fmt()
    lin = lambda x, out, **kw: _bad(q.nf4_linear, lay, 128, 256, f, x, out, **kw)
    assert "GPU" in lin(b(3, 256), b(3, 128))
    assert "GPU" in lin(b(3, 128), b(3, 256), backward=True)
    assert "x" in lin(b(3, 128), b(3, 128))
    assert "x" in lin(torch.zeros(3, 256, dtype=torch.float16), b(3, 128))
    assert "out" in lin(b(3, 256), b(3, 256))
    assert "out" in lin(b(3, 256), torch.zeros(3, 128, dtype=torch.float64))
    assert "u" in lin(b(3, 256), b(3, 128), lora=(b(4, 16), b(128, 16)))
    assert "v" in lin(b(3, 256), b(3, 128), lora=(b(3, 16), b(16, 128)))
    assert "bias" in lin(b(3, 256), b(3, 128), bias=b(256))
    assert "preact" in lin(b(3, 256), f32(3, 128), preact=f32(3, 128))
    assert "residual" in lin(b(3, 256), f32(3, 128), residual=b(3, 128))


class _Stream:
    """What the binding reads of a torch stream."""

    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


def test_binding_refuses_a_stream_of_another_device(monkeypatch):
    """Before the library is called; a stream of the tensors' device and a bare address pass on to it."""
    calls = []

    class Lib:
        def nf4_status_str(self, st):
            return b"bad argument"

        def nf4_dropout(self, *a):
            calls.append(a)
            return q.NF4_OK
    monkeypatch.setattr(q, "_lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert "device 1" in _bad(q._enqueue, "nf4_dropout", 1, _Stream(0))
    assert not calls
    q._enqueue("nf4_dropout", 1, _Stream(1), 5)
    q._enqueue("nf4_dropout", 1, 77, 6)
    assert calls == [(5, 0), (6, 77)]


def test_binding_finds_the_current_stream_by_torchs_public_call(monkeypatch):
    """A torch without the raw accessor, which is not of its public interface."""
    calls = []

    class Lib:
        def nf4_dropout(self, *a):
            calls.append(a)
            return q.NF4_OK
    monkeypatch.setattr(q, "_lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: _Stream(dev))
    q._enqueue("nf4_dropout", 1, None, 5)
    assert calls == [(5, 0)]

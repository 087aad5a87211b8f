"""The microscaled codec's and the layer norm's calls on the host (no GPU
needed): the header against the binding, argument checks of the C calls with
stand-in pointers, of the binding with CPU tensors, sizes, and the 64-bit forms."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mx4_ref as ref
import quantized_lora_fine_nf4_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # 256-aligned stand-in address; no call below reaches the device
BIG = 1 << 40


def test_binding_covers_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mx4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(mx4_[a-z0-9_]+)\s*\(", text))
    assert names == set(q.MX4_EXPORTS)
    L = ctypes.CDLL(q.LIB_PATH)
    assert all(hasattr(L, n) for n in names)


def test_sizes():
    assert q.mx4_storage_bytes(3, 64) == 96 + 6
    for bad in ((0, 32), (1, 0), (-1, 32), (1, 31), (1 << 30, 1 << 11)):
        assert q.mx4_storage_bytes(*bad) == -1
        assert q.mx4_quantize_workspace_bytes(*bad) == 0
    assert q.mx4_quantize_workspace_bytes(1, 32) == 0          # one workgroup writes the error itself
    assert q.mx4_quantize_workspace_bytes(13824, 5120) % 256 == 0 < q.mx4_quantize_workspace_bytes(13824, 5120)
    for back in (False, True):
        for m in (1, 17, 300, 5000):
            n = q.mx4_matmul_workspace_bytes(264, 2080, back, m)
            assert n >= 0 and n % 256 == 0
    for args in ((0, 32, False, 1), (8, 0, False, 1), (12, 32, False, 1), (8, 48, True, 1), (8, 32, False, 0),
                 (8, 32, False, (1 << 25) + 1), (1 << 26, 32, False, 1)):
        assert q.mx4_matmul_workspace_bytes(*args) == 0
    assert q.lib().mx4_matmul_workspace_bytes(8, 32, 2, 1) == 0
    assert q.mx4_matmul4_workspace_bytes(12, 32, 1) == 0
    assert q.nf4_layer_norm_grad_workspace_bytes(1, 64) == 0
    assert q.nf4_layer_norm_grad_workspace_bytes(100, 5120) > 0
    for m, n in ((0, 8), (1, 0), (1, 7), ((1 << 25) + 1, 8), (1, 1 << 26)):
        assert q.nf4_layer_norm_grad_workspace_bytes(m, n) == 0


def test_quantize_arguments():
    L = q.lib()

    def call(x=FAKE, rows=100, cols=4096, dt=0, codes=FAKE, scales=FAKE + 1, err=FAKE, ws=FAKE, wb=1 << 20):
        return L.mx4_quantize(x, rows, cols, dt, codes, scales, err, ws, wb, None)
    for kw in ({"x": None}, {"codes": None}, {"scales": None}, {"rows": 0}, {"cols": 0}, {"rows": -5},
               {"rows": 1 << 30, "cols": 1 << 10}):
        assert call(**kw) == q.NF4_E_ARG, kw
    assert call(cols=4095) == q.NF4_E_UNSUPPORTED
    assert call(cols=16) == q.NF4_E_UNSUPPORTED
    assert call(dt=2) == q.NF4_E_UNSUPPORTED
    for kw in ({"x": FAKE + 8}, {"codes": FAKE + 4}, {"err": FAKE + 4}):
        assert call(**kw) == q.NF4_E_ALIGN, kw
    for kw in ({"ws": None}, {"ws": FAKE + 128}, {"wb": 8}):
        assert call(**kw) == q.NF4_E_WORKSPACE, kw


def test_dequantize_arguments():
    L = q.lib()

    def call(codes=FAKE, scales=FAKE, rows=100, cols=4096, dt=0, out=FAKE):
        return L.mx4_dequantize(codes, scales, rows, cols, dt, out, None)
    for kw in ({"codes": None}, {"scales": None}, {"out": None}, {"rows": 0}):
        assert call(**kw) == q.NF4_E_ARG, kw
    assert call(cols=33) == q.NF4_E_UNSUPPORTED and call(dt=-1) == q.NF4_E_UNSUPPORTED
    assert call(codes=FAKE + 8) == q.NF4_E_ALIGN and call(out=FAKE + 2) == q.NF4_E_ALIGN


def test_matmul_arguments():
    L = q.lib()

    def call(codes=FAKE, scales=FAKE + 3, rows=4096, cols=2048, dt=0, back=0, x=FAKE, m=4, out=FAKE, f32=0, ws=FAKE,
             wb=BIG):
        return L.mx4_matmul(codes, scales, rows, cols, dt, back, x, m, out, f32, ws, wb, None)

    def call4(codes=FAKE, scales=FAKE + 3, rows=4096, cols=2048, xc=FAKE, xs=FAKE + 1, m=4, dt=0, out=FAKE, f32=0,
              ws=FAKE, wb=BIG):
        return L.mx4_matmul4(codes, scales, rows, cols, xc, xs, m, dt, out, f32, ws, wb, None)
    shared = [({"codes": None}, q.NF4_E_ARG), ({"scales": None}, q.NF4_E_ARG), ({"out": None}, q.NF4_E_ARG),
              ({"rows": 0}, q.NF4_E_ARG), ({"cols": -32}, q.NF4_E_ARG), ({"m": 0}, q.NF4_E_ARG),
              ({"m": (1 << 25) + 1}, q.NF4_E_ARG), ({"rows": 1 << 26}, q.NF4_E_ARG), ({"f32": 2}, q.NF4_E_ARG),
              ({"rows": 1 << 20, "cols": 1 << 20}, q.NF4_E_ARG), ({"rows": 4097}, q.NF4_E_UNSUPPORTED),
              ({"cols": 2032}, q.NF4_E_UNSUPPORTED), ({"dt": 2}, q.NF4_E_UNSUPPORTED),
              ({"codes": FAKE + 8}, q.NF4_E_ALIGN), ({"out": FAKE + 8}, q.NF4_E_ALIGN)]
    for kw, st in shared:
        assert call(**kw) == st, kw
        assert call4(**kw) == st, kw
    assert call(x=None) == q.NF4_E_ARG and call(back=2) == q.NF4_E_ARG
    assert call(x=FAKE + 2) == q.NF4_E_ALIGN
    assert call4(xc=None) == q.NF4_E_ARG and call4(xs=None) == q.NF4_E_ARG
    assert call4(xc=FAKE + 8) == q.NF4_E_ALIGN
    # a side of 2^22 and more, and over 2^38 outputs (of the product or of its gradient)
    for kw in ({"rows": 1 << 22, "cols": 32}, {"rows": 8, "cols": 1 << 22}, {"rows": 8, "cols": (1 << 13) + 32, "m": 1 << 25},
               {"rows": (1 << 13) + 8, "cols": 32, "m": 1 << 25}):
        assert call(**kw) == call(back=1, **kw) == call4(**kw) == q.NF4_E_ARG, kw
        rows, cols, n = kw["rows"], kw["cols"], kw.get("m", 4)
        assert q.mx4_matmul_workspace_bytes(rows, cols, False, n) == q.mx4_matmul4_workspace_bytes(rows, cols, n) == 0
    m = 4
    for back in (0, 1):
        if q.mx4_matmul_workspace_bytes(4096, 2048, back, m):
            for kw in ({"ws": None}, {"ws": FAKE + 16}, {"wb": 16}):
                assert call(back=back, **kw) == q.NF4_E_WORKSPACE, kw


def test_norm_arguments():
    L = q.lib()

    def fwd(x=FAKE, res=None, w=FAKE, b=FAKE, m=10, n=64, dt=0, eps=1e-5, out=FAKE, total=None, stats=FAKE):
        return L.nf4_layer_norm(x, res, w, b, m, n, dt, eps, out, total, stats, None)

    def bwd(dy=FAKE, x=FAKE, w=FAKE, stats=FAKE, res=None, m=10, n=64, dt=0, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, wb=BIG):
        return L.nf4_layer_norm_grad(dy, x, w, stats, res, m, n, dt, dx, dw, db, ws, wb, None)
    for kw in ({"x": None}, {"w": None}, {"b": None}, {"out": None}, {"stats": None}, {"m": 0}, {"n": 0}, {"n": 1 << 26},
               {"m": (1 << 25) + 1}, {"res": FAKE}, {"total": FAKE + 64}, {"res": FAKE, "total": FAKE}, {"eps": -1.0},
               {"eps": float("nan")}, {"eps": float("inf")}):
        assert fwd(**kw) == q.NF4_E_ARG, kw
    assert fwd(n=63) == q.NF4_E_UNSUPPORTED and fwd(dt=3) == q.NF4_E_UNSUPPORTED
    for name in ("x", "w", "b", "out"):
        assert fwd(**{name: FAKE + 8}) == q.NF4_E_ALIGN, name
    assert fwd(stats=FAKE + 4) == q.NF4_E_ALIGN
    assert fwd(res=FAKE + 8, total=FAKE + 64) == q.NF4_E_ALIGN and fwd(res=FAKE, total=FAKE + 8) == q.NF4_E_ALIGN
    for kw in ({"dy": None}, {"x": None}, {"w": None}, {"stats": None}, {"dx": None}, {"dw": None}, {"db": None},
               {"m": 0}, {"n": -8}):
        assert bwd(**kw) == q.NF4_E_ARG, kw
    assert bwd(n=60) == q.NF4_E_UNSUPPORTED and bwd(dt=3) == q.NF4_E_UNSUPPORTED
    for name in ("dy", "x", "w", "dx", "dw", "db", "res"):
        assert bwd(**{name: FAKE + 8}) == q.NF4_E_ALIGN, name
    for kw in ({"ws": None}, {"ws": FAKE + 16}, {"wb": 16}):
        assert bwd(n=5120, **kw) == q.NF4_E_WORKSPACE, kw


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def refused(fn, *a, **kw):
    with pytest.raises(q.NF4Error) as e:
        fn(*a, **kw)
    assert e.value.status == q.NF4_E_ARG, str(e.value)
    return str(e.value)


def test_binding_refuses_what_does_not_fit():
    u8 = torch.uint8
    codes, scales = cpu(64, 64, dtype=u8), cpu(64, 4, dtype=u8)
    x, out = cpu(3, 128), cpu(3, 64)
    # shapes and types first; with everything right, a CPU tensor is refused as such
    assert "GPU" in refused(q.mx4_matmul, codes, scales, x, out)
    assert "x must be" in refused(q.mx4_matmul, codes, scales, cpu(3, 96), out)
    assert "out must be" in refused(q.mx4_matmul, codes, scales, x, cpu(3, 65))
    assert "out must be" in refused(q.mx4_matmul, codes, scales, x, cpu(3, 64, dtype=torch.float16))
    assert "scales must be" in refused(q.mx4_matmul, codes, cpu(64, 8, dtype=u8), x, out)
    assert "codes must be" in refused(q.mx4_matmul, cpu(64, 60, dtype=u8), scales, x, out)
    assert "codes must be" in refused(q.mx4_matmul, cpu(64, 64, dtype=torch.int8), scales, x, out)
    assert "codes must be" in refused(q.mx4_matmul, codes.t().contiguous().t(), scales, x, out)
    assert "two dimensions" in refused(q.mx4_matmul, codes, scales, cpu(128), out)
    assert "expected" in refused(q.mx4_matmul, codes, scales, cpu(3, 128, dtype=torch.float32), out)
    assert "x must be" in refused(q.mx4_matmul, codes, scales, x, out, backward=True)
    xc, xs = cpu(3, 64, dtype=u8), cpu(3, 4, dtype=u8)
    assert "GPU" in refused(q.mx4_matmul4, codes, scales, xc, xs, out)
    assert "columns" in refused(q.mx4_matmul4, codes, scales, cpu(3, 48, dtype=u8), cpu(3, 3, dtype=u8), out)
    assert "out must be" in refused(q.mx4_matmul4, codes, scales, xc, xs, cpu(3, 64, dtype=torch.float64))
    w = cpu(64, 128)
    assert "GPU" in refused(q.mx4_quantize, w, codes, scales)
    assert "x must be" in refused(q.mx4_quantize, cpu(64, 160), codes, scales)
    assert "err must be" in refused(q.mx4_quantize, w, codes, scales, cpu(1, dtype=torch.float32))
    assert "GPU" in refused(q.mx4_dequantize, codes, scales, w)
    assert "out must be" in refused(q.mx4_dequantize, codes, scales, cpu(64, 64))
    assert "expected" in refused(q.mx4_dequantize, codes, scales, cpu(64, 128, dtype=torch.float32))
    v, st = cpu(128), cpu(3, 2, dtype=torch.float32)
    assert "GPU" in refused(q.nf4_layer_norm, x, v, v, x, st)
    assert "weight must be" in refused(q.nf4_layer_norm, x, cpu(64), v, x, st)
    assert "stats must be" in refused(q.nf4_layer_norm, x, v, v, x, cpu(3, 2))
    assert "residual must be" in refused(q.nf4_layer_norm, x, v, v, x, st, residual=cpu(3, 64), total=x)
    assert "[m, n]" in refused(q.nf4_layer_norm, v, v, v, v, st)
    g = cpu(128, dtype=torch.float32)
    assert "GPU" in refused(q.nf4_layer_norm_grad, x, x, v, st, x, g, g)
    assert "dweight must be" in refused(q.nf4_layer_norm_grad, x, x, v, st, x, v, g)
    assert "dx must be" in refused(q.nf4_layer_norm_grad, x, x, v, st, cpu(3, 64), g, g)


# ---- the 64-bit forms themselves -------------------------------------------

def test_reference_codec_on_known_values():
    x = torch.zeros(1, 32, dtype=torch.bfloat16)
    x[0, :9] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0, 7.5])
    c, s = ref.quantize(x)
    assert s.item() == 127   # floor(log2 7.5) - 2 = 0
    nib = torch.stack([c & 15, c >> 4], -1).flatten()[:9].tolist()
    assert nib == [6, 0, 2, 2, 4, 4, 6, 8 + 6, 7]   # ties to the even code, 7.5 to 6
    assert ref.values(c, s)[0, :9].tolist() == [4, 0, 1, 1, 2, 2, 4, -4, 6]
    c, s = ref.quantize(torch.full((1, 32), -0.0, dtype=torch.float16))
    assert s.item() == 0 and (c == 0x88).all()


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    x, w, b, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((2, 16), (16,), (16,), (2, 16)))
    _, mean, _, rstd = ref.layer_norm(x, w, b, 1e-5)
    dx, dw, db = ref.layer_norm_grad(dy, x, w, mean, rstd)
    h = 1e-5
    for i, got in enumerate((dx, dw, db)):
        for k in range(got.numel()):
            v = []
            for sign in (1, -1):
                a = [x.clone(), w.clone(), b.clone()]
                a[i].view(-1)[k] += sign * h
                v.append((dy * ref.layer_norm(*a, 1e-5)[0]).sum().item())
            assert abs(got.view(-1)[k].item() - (v[0] - v[1]) / (2 * h)) < 1e-8

"""MI355X-native NF4 weight codec and AQLoRA layer selector.

Thin Python binding over ``libnf4.so`` (C ABI: ``include/nf4.h``).  The
functions carry the C names and only marshal arguments: every step of the
codec and of the ranking runs in the HIP kernels.  PyTorch provides device
memory and the current stream; nothing here computes on the CPU, and a
missing library raises instead of falling back.

    nf4_quantize, nf4_double_quant, nf4_dequantize, nf4_dequantize_masked,
    nf4_layer_error, aqlora_select_topk     -- enqueue on the current stream
    nf4_linear, nf4_act_grad, nf4_dropout, nf4_lora_project, nf4_lora_grad
                                            -- one adapted layer, on the
                                               tensors' device
    nf4_workspace_bytes, aqlora_workspace_bytes, nf4_storage_bytes,
    aqlora_promote_cost, nf4_levels, nf4_thresholds, nf4_abi_version
                                            -- host-only helpers

``LayerSet`` allocates the per-layer device buffers of a stack of matrices
(one tensor per buffer kind, per-layer slices aligned as the ABI requires)
and keeps the matching ``nf4_layer`` array.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnf4.so")

NF4_OK, NF4_E_ARG, NF4_E_ALIGN, NF4_E_UNSUPPORTED, NF4_E_WORKSPACE, NF4_E_HIP = range(6)
NF4_BF16, NF4_FP16 = 0, 1
AQLORA_PREFIX, AQLORA_FILL = 0, 1
BLOCK, DQ_GROUP = 64, 256


class NF4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib_or_none().nf4_status_str(status).decode() if _lib_or_none() else str(status)
        extra = ""
        if status == NF4_E_HIP and _lib_or_none():
            extra = f" (hipError {_lib_or_none().nf4_last_hip_error()})"
        super().__init__(f"{where}: {msg}{extra}")


class nf4_format(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("blocksize", ctypes.c_int32),
                ("dq_group", ctypes.c_int32)]


class nf4_variant(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("blocksize", ctypes.c_int32),
                ("dq_kind", ctypes.c_int32)]


NF4_DQ_NONE, NF4_DQ_INT8, NF4_DQ_INT8_MEAN, NF4_DQ_E4M3_MEAN = range(4)


NF4_ACT_NONE, NF4_ACT_RELU, NF4_ACT_SILU, NF4_ACT_GELU, NF4_ACT_GELU_TANH = range(5)
NF4_LORA_A, NF4_LORA_B = 0, 1
LORA_MAX_RANK = 128


class nf4_drop(ctypes.Structure):
    _fields_ = [("rng", ctypes.c_void_p), ("p", ctypes.c_float)]


class nf4_epilogue(ctypes.Structure):
    _fields_ = [("u", ctypes.c_void_p), ("v", ctypes.c_void_p), ("rank", ctypes.c_int32),
                ("act", ctypes.c_int32), ("drop", nf4_drop), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("preact", ctypes.c_void_p)]


class nf4_layer(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("w", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("absmax", ctypes.c_void_p), ("qabsmax", ctypes.c_void_p),
                ("scale2", ctypes.c_void_p), ("out", ctypes.c_void_p)]


EXPORTS = {
    # name: (restype, argtypes)
    "nf4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format, ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_double_quant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_dequantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format,
                                      ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_dequantize_masked": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                             ctypes.c_void_p]),
    "nf4_layer_error": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "nf4_layer_error_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format,
                                               ctypes.c_void_p, ctypes.c_void_p]),
    "nf4_noalloc_scratch_bytes": (ctypes.c_size_t, []),
    "nf4_layer_error_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_format,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_size_t, ctypes.c_void_p]),
    "aqlora_select_topk": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                          ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]),
    "aqlora_select": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                     ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_matmul": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, nf4_format,
                                  ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                                  ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "nf4_matmul_ws": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, nf4_format,
                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                                     ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_matmul_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                                     ctypes.c_int64]),
    "nf4_linear": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, nf4_format,
                                  ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                  ctypes.c_void_p]),
    "nf4_act_grad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_dropout": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, nf4_drop,
                                   ctypes.c_void_p, ctypes.c_void_p]),
    "nf4_lora_project": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_float,
                                        nf4_drop, ctypes.c_void_p, ctypes.c_void_p]),
    "nf4_lora_grad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                     ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, nf4_drop,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_act_grad_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "nf4_lora_grad_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32]),
    "nf4_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_void_p, nf4_format]),
    "nf4_layer_error_variant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_variant,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_size_t, ctypes.c_void_p]),
    "nf4_dequantize_variant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, nf4_variant,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                              ctypes.c_void_p]),
    "nf4_workspace_bytes_variant": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_void_p,
                                                      nf4_variant]),
    "nf4_storage_bytes_variant": (ctypes.c_int64, [ctypes.c_int64, nf4_variant]),
    "aqlora_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int32]),
    "nf4_storage_bytes": (ctypes.c_int64, [ctypes.c_int64, nf4_format]),
    "aqlora_promote_cost": (ctypes.c_int64, [ctypes.c_int64, nf4_format]),
    "nf4_levels": (None, [ctypes.c_void_p]),
    "nf4_thresholds": (None, [ctypes.c_void_p]),
    "nf4_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "nf4_abi_version": (ctypes.c_int32, []),
    "nf4_last_hip_error": (ctypes.c_int32, []),
}

_lib = None


def _lib_or_none():
    return _lib


def lib() -> ctypes.CDLL:
    """Load the HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python quantized_lora_fine_nf4_amd/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def fmt(dtype: int = NF4_BF16, dq: bool = True) -> nf4_format:
    return nf4_format(int(dtype), BLOCK, DQ_GROUP if dq else 0)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return int(t.data_ptr())


def _stream(stream) -> int | None:
    if stream is not None:
        return int(stream) if isinstance(stream, int) else int(stream.cuda_stream)
    import torch
    return int(torch.cuda.current_stream().cuda_stream)


def _check(status: int, where: str):
    if status != NF4_OK:
        raise NF4Error(status, where)


def _layers_arg(layers):
    """A LayerSet / LayerSubset, or a sequence of nf4_layer structs."""
    if isinstance(layers, (LayerSet, LayerSubset)):
        return ctypes.byref(layers.c_layers), len(layers)
    arr = (nf4_layer * len(layers))(*layers)
    return arr, len(layers)


# ---- the five calls -------------------------------------------------------

def nf4_quantize(layers, f: nf4_format, ws, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_quantize(arr, nl, f, _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream)), "nf4_quantize")


def nf4_double_quant(layers, f: nf4_format, ws, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_double_quant(arr, nl, f, _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "nf4_double_quant")


def nf4_dequantize(layers, f: nf4_format, ws, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_dequantize(arr, nl, f, _ptr(ws), ws.numel() * ws.element_size(),
                                _stream(stream)), "nf4_dequantize")


def nf4_dequantize_masked(layers, f: nf4_format, skip, ws, stream=None) -> None:
    """nf4_dequantize of the layers whose byte in skip (device uint8[nl], e.g.
    aqlora_select_topk's selected) is 0; the others' outputs are untouched."""
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_dequantize_masked(arr, nl, f, _ptr(skip), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)), "nf4_dequantize_masked")


def nf4_layer_error(layers, f: nf4_format, err, ws, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_layer_error(arr, nl, f, _ptr(err), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)),
           "nf4_layer_error")


def nf4_layer_error_noalloc(layers, f: nf4_format, err, stream=None) -> None:
    """nf4_layer_error with the library's fixed per-device scratch instead of
    a workspace (for callers that cannot allocate)."""
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_layer_error_noalloc(arr, nl, f, _ptr(err), _stream(stream)),
           "nf4_layer_error_noalloc")


def nf4_noalloc_scratch_bytes() -> int:
    return int(lib().nf4_noalloc_scratch_bytes())


def aqlora_select_topk(err, cost, budget_bytes: int, k_cap: int, selected, k_out, ws,
                       stream=None) -> None:
    nl = int(err.numel())
    _check(lib().aqlora_select_topk(_ptr(err), _ptr(cost), nl, int(budget_bytes), int(k_cap),
                                    _ptr(selected), _ptr(k_out), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "aqlora_select_topk")


def nf4_layer_error_norm(layers, f: nf4_format, err, sumsq, ws, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_layer_error_norm(arr, nl, f, _ptr(err), _ptr(sumsq), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "nf4_layer_error_norm")


def aqlora_select(err, cost, budget_bytes: int, k_cap: int, selected, k_out, ws, denom=None,
                  group_end=None, rule: int = AQLORA_PREFIX, stream=None) -> None:
    """group_end: host sequence of group ends (copied before return), or None."""
    nl = int(err.numel())
    ge = None if group_end is None else np.ascontiguousarray(group_end, np.int32)
    _check(lib().aqlora_select(_ptr(err), _ptr(denom), _ptr(cost), nl,
                               None if ge is None else ge.ctypes.data,
                               0 if ge is None else int(ge.size), int(budget_bytes), int(k_cap),
                               int(rule), _ptr(selected), _ptr(k_out), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)),
           "aqlora_select")


def nf4_matmul(layer, rows: int, cols: int, f: nf4_format, x, out, backward: bool = False,
               stream=None) -> None:
    """out = x @ W^T (forward) or x @ W (backward) with W in NF4 form.
    layer: an nf4_layer struct (e.g. ls.c_layers[i]); x, out: device tensors
    (x in the 16-bit type f.dtype names; out float32 or that 16-bit type)."""
    import torch
    m = int(x.shape[0]) if x.dim() > 1 else 1
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    _check(lib().nf4_matmul(ctypes.byref(layer), int(rows), int(cols), f, int(bool(backward)),
                            _ptr(x), m, _ptr(out), out_fp32, _stream(stream)), "nf4_matmul")


def nf4_matmul_workspace_bytes(rows: int, cols: int, backward: bool, m: int) -> int:
    return int(lib().nf4_matmul_workspace_bytes(int(rows), int(cols), int(bool(backward)), int(m)))


def nf4_matmul_ws(layer, rows: int, cols: int, f: nf4_format, x, out, ws, backward: bool = False,
                  stream=None) -> None:
    """nf4_matmul with a workspace (ws: device uint8 tensor of at least
    nf4_matmul_workspace_bytes(...) bytes, or None when that is 0): the
    few-token forward kernel at m <= 32, the split reduction when the output
    tiles alone do not fill the GPU, and the split of the tiles left over
    after whole rounds of large tiles."""
    import torch
    m = int(x.shape[0]) if x.dim() > 1 else 1
    out_fp32 = 1 if out.dtype == torch.float32 else 0
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().nf4_matmul_ws(ctypes.byref(layer), int(rows), int(cols), f, int(bool(backward)),
                               _ptr(x), m, _ptr(out), out_fp32, _ptr(ws), nbytes, _stream(stream)),
           "nf4_matmul_ws")


def variant(dtype: int = NF4_BF16, block: int = BLOCK, kind: int = NF4_DQ_INT8) -> nf4_variant:
    return nf4_variant(int(dtype), int(block), int(kind))


def nf4_layer_error_variant(layers, v: nf4_variant, err, ws, mean=None, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_layer_error_variant(arr, nl, v, _ptr(mean), _ptr(err), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream)),
           "nf4_layer_error_variant")


def nf4_dequantize_variant(layers, v: nf4_variant, ws, mean=None, stream=None) -> None:
    arr, nl = _layers_arg(layers)
    _check(lib().nf4_dequantize_variant(arr, nl, v, _ptr(mean), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)),
           "nf4_dequantize_variant")


def nf4_workspace_bytes_variant(ns, v: nf4_variant) -> int:
    a = np.ascontiguousarray(ns, np.int64)
    return int(lib().nf4_workspace_bytes_variant(a.size, a.ctypes.data if a.size else None, v))


def nf4_storage_bytes_variant(n: int, v: nf4_variant) -> int:
    return int(lib().nf4_storage_bytes_variant(int(n), v))


# ---- the adapted layer ----------------------------------------------------
#
# Unlike the codec calls, these take their shapes from the tensors, so they
# check them: what does not fit raises NF4Error with NF4_E_ARG (or the status
# the C call returns) and enqueues nothing.  Work goes to the current stream of
# the tensors' device, or to `stream`, which must be one of that device's (of a
# torch stream this is checked; an address is taken as it is).

def _misfit(where: str, what: str):
    e = NF4Error(NF4_E_ARG, where)
    e.args = (f"{e.args[0]}: {what}",)
    raise e


def _dtype16(t, where: str) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return NF4_BF16
    if t.dtype is not torch.float16:
        _misfit(where, f"bfloat16 or float16 expected, got {t.dtype}")
    return NF4_FP16


def _fits(t, name: str, where: str, shape: tuple, dtype, dev: int) -> int:
    """The address of a tensor that must have this shape, type and device index."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _misfit(where, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on device {dev}, got "
                       f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


_NO_DROP = nf4_drop(None, 0.0)


def _rng_arg(p: float, rng, where: str, dev: int) -> nf4_drop:
    if not p:
        return _NO_DROP
    if rng is None:
        _misfit(where, "dropout needs rng")
    import torch
    if (rng.numel() != 2 or (rng.dtype is not torch.int64 and rng.dtype is not torch.uint64)
            or rng.get_device() != dev or not rng.is_contiguous()):
        _misfit(where, f"rng must hold {{seed, offset}} as 64-bit integers on device {dev}")
    return nf4_drop(rng.data_ptr(), p)


def _ws_arg(ws, where: str, dev: int):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        _misfit(where, f"the workspace must be a contiguous tensor on device {dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _enqueue(name: str, dev: int, stream, *args) -> None:
    """The C call `name` with these arguments and the stream, the tensors' device current."""
    import torch
    if dev < 0:
        _misfit(name, "tensors must be on the GPU")
    if stream is None:
        # current_stream(dev) without the Stream object, where this torch offers it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        s = raw(dev) if raw else torch.cuda.current_stream(dev).cuda_stream
    else:
        if getattr(stream, "device_index", dev) != dev:
            _misfit(name, f"the stream must be one of device {dev}, got {stream}")
        s = _stream(stream)
    fn = getattr(_lib or lib(), name)
    if dev == torch.cuda.current_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != NF4_OK:
        raise NF4Error(st, name)


def nf4_linear(layer, rows: int, cols: int, f: nf4_format, x, out, ws=None, backward: bool = False, lora=None,
               bias=None, act: int = NF4_ACT_NONE, preact=None, residual=None, p: float = 0.0, rng=None,
               stream=None) -> None:
    """Forward: out = act(z) + residual, z = x W^T + u v^T + bias, preact = z.
    Backward: out = x W + drop(u v) + residual.  W [rows x cols] in NF4 form
    (layer: an nf4_layer struct), lora = (u, v): u [m, rank] and v [rows, rank]
    forward, [rank, cols] backward.  x, u, v, bias, preact in the 16-bit type f
    names; out that type or float32, residual like out (it may be out).  ws:
    device tensor of nf4_matmul_workspace_bytes(rows, cols, backward, m) bytes,
    or None when that is 0."""
    import torch
    w = "nf4_linear"
    dev, t16 = x.get_device(), torch.bfloat16 if f.dtype == NF4_BF16 else torch.float16
    kred, ncol = (rows, cols) if backward else (cols, rows)
    if x.dim() == 2:
        m, xs, os_ = x.shape[0], (x.shape[0], kred), (x.shape[0], ncol)
    else:
        m, xs, os_ = 1, (kred,), (ncol,)
    xp = _fits(x, "x", w, xs, t16, dev)
    f32 = out.dtype is torch.float32
    if out.dim() == 1 and m == 1:
        os_ = (ncol,)
    op = _fits(out, "out", w, os_, torch.float32 if f32 else t16, dev)
    e = nf4_epilogue()
    if lora is not None:
        u, v = lora
        r = u.shape[-1]
        e.u = _fits(u, "u", w, (m, r) if u.dim() == 2 or m > 1 else (r,), t16, dev)
        e.v = _fits(v, "v", w, (r, cols) if backward else (rows, r), t16, dev)
        e.rank = r
    e.act = int(act)
    if p:
        e.drop = _rng_arg(p, rng, w, dev)
    if bias is not None:
        e.bias = _fits(bias, "bias", w, (ncol,), t16, dev)
    if preact is not None:
        e.preact = _fits(preact, "preact", w, os_, t16, dev)
    if residual is not None:
        e.residual = _fits(residual, "residual", w, os_, out.dtype, dev)
    wp, wb = _ws_arg(ws, w, dev)
    _enqueue(w, dev, stream, ctypes.byref(layer), int(rows), int(cols), f, 1 if backward else 0, xp, m, ctypes.byref(e), op,
             1 if f32 else 0, wp, wb)


def nf4_act_grad(dy, preact, act: int, dz=None, dbias=None, ws=None, stream=None) -> None:
    """dz = dy act'(preact) and, with dbias (float32 [n]), its sum over the
    tokens.  dy, preact, dz: [m, n], bfloat16 or float16; dz may be dy.  With
    NF4_ACT_NONE preact and dz may be None.  ws: device tensor of
    nf4_act_grad_workspace_bytes(m, n) bytes with dbias."""
    import torch
    w = "nf4_act_grad"
    dt, dev = _dtype16(dy, w), dy.get_device()
    if dy.dim() != 2:
        _misfit(w, "dy must be [m, n]")
    m, n = shape = dy.shape
    dp = _fits(dy, "dy", w, shape, dy.dtype, dev)
    pp = None if preact is None else _fits(preact, "preact", w, shape, dy.dtype, dev)
    zp = None if dz is None else _fits(dz, "dz", w, shape, dy.dtype, dev)
    bp = None if dbias is None else _fits(dbias, "dbias", w, (n,), torch.float32, dev)
    wp, wb = _ws_arg(ws, w, dev)
    _enqueue(w, dev, stream, dp, pp, int(act), m, n, dt, zp, bp, wp, wb)


def nf4_act_grad_workspace_bytes(m: int, n: int) -> int:
    return int(lib().nf4_act_grad_workspace_bytes(int(m), int(n)))


def nf4_dropout(x, out, p: float, rng, stream=None) -> None:
    """out = drop(x) (bfloat16 or float16, any shape; out may be x): the mask of
    rng (device int64 {seed, offset}) over the flat elements."""
    w = "nf4_dropout"
    dt, dev = _dtype16(x, w), x.get_device()
    xp = _fits(x, "x", w, x.shape, x.dtype, dev)
    op = _fits(out, "out", w, x.shape, x.dtype, dev)
    _enqueue(w, dev, stream, xp, x.numel(), dt, _rng_arg(p, rng, w, dev), op)


def nf4_lora_project(x, w, h, scale: float = 1.0, backward: bool = False, p: float = 0.0, rng=None,
                     stream=None) -> None:
    """h [m, rank] = scale drop(x) w^T (x [m, k], w [rank, k]), or backward
    scale x w (w [k, rank]); bfloat16 or float16."""
    fn = "nf4_lora_project"
    dt, dev, t16 = _dtype16(x, fn), x.get_device(), x.dtype
    if x.dim() != 2 or w.dim() != 2:
        _misfit(fn, "x and w must have two dimensions")
    m, k = x.shape
    r = w.shape[1 if backward else 0]
    xp = _fits(x, "x", fn, (m, k), t16, dev)
    wp = _fits(w, "w", fn, (k, r) if backward else (r, k), t16, dev)
    hp = _fits(h, "h", fn, (m, r), t16, dev)
    _enqueue(fn, dev, stream, xp, m, k, wp, r, dt, 1 if backward else 0, scale, _rng_arg(p, rng, fn, dev), hp)


def nf4_lora_grad(u, x, grad, ws=None, side: str = "A", p: float = 0.0, rng=None, stream=None) -> None:
    """side "A": grad [rank, n] = u^T drop(x); side "B": grad [n, rank] =
    x^T u.  u [m, rank], x [m, n] bfloat16 or float16, grad float32.  ws:
    device tensor of nf4_lora_grad_workspace_bytes(m, n, rank) bytes, or None
    when that is 0."""
    import torch
    fn = "nf4_lora_grad"
    dt, dev, t16 = _dtype16(x, fn), x.get_device(), x.dtype
    if x.dim() != 2 or u.dim() != 2:
        _misfit(fn, "u and x must have two dimensions")
    if side != "A" and side != "B":
        _misfit(fn, "side must be 'A' or 'B'")
    m, n = x.shape
    r = u.shape[1]
    xp = _fits(x, "x", fn, (m, n), t16, dev)
    up = _fits(u, "u", fn, (m, r), t16, dev)
    gp = _fits(grad, "grad", fn, (r, n) if side == "A" else (n, r), torch.float32, dev)
    wp, wb = _ws_arg(ws, fn, dev)
    _enqueue(fn, dev, stream, up, xp, m, n, r, dt, NF4_LORA_A if side == "A" else NF4_LORA_B,
             _rng_arg(p, rng, fn, dev), gp, wp, wb)


def nf4_lora_grad_workspace_bytes(m: int, n: int, rank: int) -> int:
    return int(lib().nf4_lora_grad_workspace_bytes(int(m), int(n), int(rank)))


# ---- host helpers ---------------------------------------------------------

def nf4_workspace_bytes(ns, f: nf4_format) -> int:
    a = np.ascontiguousarray(ns, np.int64)
    return int(lib().nf4_workspace_bytes(a.size, a.ctypes.data, f))


def aqlora_workspace_bytes(nl: int) -> int:
    return int(lib().aqlora_workspace_bytes(nl))


def nf4_storage_bytes(n: int, f: nf4_format) -> int:
    return int(lib().nf4_storage_bytes(n, f))


def aqlora_promote_cost(n: int, f: nf4_format) -> int:
    return int(lib().aqlora_promote_cost(n, f))


def nf4_levels() -> np.ndarray:
    out = np.zeros(16, np.float32)
    lib().nf4_levels(out.ctypes.data)
    return out


def nf4_thresholds() -> np.ndarray:
    out = np.zeros(15, np.float32)
    lib().nf4_thresholds(out.ctypes.data)
    return out


def nf4_abi_version() -> int:
    return int(lib().nf4_abi_version())


# ---- device buffers for a stack of matrices -------------------------------

def _round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


class LayerSet:
    """Device buffers for ``len(ns)`` matrices of ``ns[i]`` elements.

    Each buffer kind is one tensor; layer i's slice starts at an offset that
    keeps the ABI's alignment (weights, codes and outputs 16 B).
    Attributes: ``w`` (int16 bits), ``codes`` (uint8), ``absmax`` (float32),
    ``qabsmax`` (int8), ``scale2`` (float32), ``out`` (int16 bits), the offset
    lists ``*_off``, and ``c_layers`` (the nf4_layer array).  ``w``, ``codes``
    and ``out`` may be given (e.g. another LayerSet's, whose offsets do not
    depend on the block size) instead of allocated.
    """

    def __init__(self, ns, f: nf4_format, device="cuda", with_out: bool = True,
                 with_absmax: bool = True, w=None, block: int = BLOCK, codes=None, out=None):
        import torch
        self.ns = [int(n) for n in ns]
        self.fmt = f
        dq = f.dq_group != 0
        self.block = int(block)
        nb = [(n + self.block - 1) // self.block for n in self.ns]
        ng = [(b + DQ_GROUP - 1) // DQ_GROUP for b in nb]

        def offsets(sizes, align):
            offs, run = [], 0
            for s in sizes:
                offs.append(run)
                run += _round_up(max(s, 1), align)
            return offs, run

        self.w_off, wtot = offsets(self.ns, 64)
        self.c_off, ctot = offsets([(n + 1) // 2 for n in self.ns], 64)
        self.a_off, atot = offsets(nb, 64)
        self.s_off, stot = offsets(ng, 64)
        if w is None:
            self.w = torch.empty(wtot, dtype=torch.int16, device=device)
        else:
            assert w.dtype == torch.int16 and w.numel() >= wtot
            self.w = w
        if codes is None:
            self.codes = torch.empty(ctot, dtype=torch.uint8, device=device)
        else:
            assert codes.dtype == torch.uint8 and codes.numel() >= ctot
            self.codes = codes
        self.absmax = torch.empty(atot, dtype=torch.float32, device=device) if (with_absmax or not dq) else None
        self.qabsmax = torch.empty(atot, dtype=torch.int8, device=device) if dq else None
        self.scale2 = torch.empty(stot, dtype=torch.float32, device=device) if dq else None
        if out is not None:
            assert out.dtype == torch.int16 and out.numel() >= wtot
            self.out = out
        else:
            self.out = torch.empty(wtot, dtype=torch.int16, device=device) if with_out else None
        self._build()

    def _build(self):
        L = []
        for i, n in enumerate(self.ns):
            def at(t, off, esz):
                return None if t is None else int(t.data_ptr()) + off * esz
            L.append(nf4_layer(n, at(self.w, self.w_off[i], 2), at(self.codes, self.c_off[i], 1),
                               at(self.absmax, self.a_off[i], 4), at(self.qabsmax, self.a_off[i], 1),
                               at(self.scale2, self.s_off[i], 4), at(self.out, self.w_off[i], 2)))
        self.c_layers = (nf4_layer * len(L))(*L)

    def subset(self, idx) -> "LayerSubset":
        return LayerSubset(self, list(idx))

    def __len__(self):
        return len(self.ns)

    # per-layer views
    def w_of(self, i):
        return self.w[self.w_off[i]: self.w_off[i] + self.ns[i]]

    def out_of(self, i):
        return self.out[self.w_off[i]: self.w_off[i] + self.ns[i]]

    def codes_of(self, i):
        return self.codes[self.c_off[i]: self.c_off[i] + (self.ns[i] + 1) // 2]

    def absmax_of(self, i):
        nb = (self.ns[i] + self.block - 1) // self.block
        return self.absmax[self.a_off[i]: self.a_off[i] + nb]

    def qabsmax_of(self, i):
        nb = (self.ns[i] + self.block - 1) // self.block
        return self.qabsmax[self.a_off[i]: self.a_off[i] + nb]

    def scale2_of(self, i):
        ng = ((self.ns[i] + self.block - 1) // self.block + DQ_GROUP - 1) // DQ_GROUP
        return self.scale2[self.s_off[i]: self.s_off[i] + ng]


class LayerSubset:
    """Some layers of a LayerSet, e.g. the ones left in NF4 after promotion."""

    def __init__(self, parent: LayerSet, idx):
        self.parent = parent
        self.idx = idx
        self.c_layers = (nf4_layer * len(idx))(*[parent.c_layers[i] for i in idx])

    def __len__(self):
        return len(self.idx)


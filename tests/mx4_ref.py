"""Plain 64-bit forms of the microscaled 4-bit codec, its products and the layer
norm, for the tests, written from the formats' fields."""
from __future__ import annotations

import numpy as np
import torch

U16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}    # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half a subnormal step
U32 = 2.0 ** -24
VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x: torch.Tensor):
    """codes [rows, cols / 2], scales [rows, cols / 32] of x [rows, cols], by the distances to all eight magnitudes."""
    a = x.double().cpu().numpy().reshape(-1, 32)
    top = np.abs(a).max(1)
    bad = ~np.isfinite(top)
    top[bad] = 1.0
    _, e = np.frexp(top)
    e = np.where(top > 0, np.clip(e - 1 - 2, -127, 127), -127)
    with np.errstate(invalid="ignore"):
        v = np.abs(np.ldexp(a, -e[:, None]))
    v = np.where(np.isfinite(v), v, 0.0)
    d = np.abs(v[..., None] - VALUES)
    best = d.min(-1, keepdims=True)
    # of the nearest (one, or two at a border) the even code
    tie = d == best
    code = np.where(tie.sum(-1) == 1, tie.argmax(-1), (tie * (np.arange(8) % 2 == 0)).argmax(-1)).astype(np.uint8)
    code |= np.signbit(a).astype(np.uint8) << 3
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    code = code.reshape(x.shape)
    return torch.from_numpy(code[:, 0::2] | code[:, 1::2] << 4), torch.from_numpy(s.reshape(x.shape[0], -1))


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values [rows, cols]."""
    c, s = codes.cpu().numpy(), scales.cpu().numpy().astype(np.int64)
    nib = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    v = VALUES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return torch.from_numpy(v * np.repeat(f, 32, 1))


def rounded(v: torch.Tensor, dtype) -> torch.Tensor:
    """The values as the products read them: rounded to the 16-bit type (exact in fp32 before that)."""
    return v.float().to(dtype).double()


def random_matrix(rows: int, cols: int, g: torch.Generator, lo: int = 118, hi: int = 124):
    """Codes and scales of a weight, every code, scales from a range."""
    return (torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8),
            torch.randint(lo, hi, (rows, cols // 32), generator=g, dtype=torch.uint8))


def layer_norm(h, weight, bias, eps):
    h = h.double()
    mean = h.mean(1, keepdim=True)
    var = (h - mean).square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    return (h - mean) * rstd * weight.double() + bias.double(), mean, var, rstd


def layer_norm_grad(dy, x, weight, mean, rstd):
    dy, c = dy.double(), (x.double() - mean) * rstd
    g = dy * weight.double()
    dx = rstd * (g - g.mean(1, keepdim=True) - c * (g * c).mean(1, keepdim=True))
    return dx, (dy * c).sum(0), dy.sum(0)

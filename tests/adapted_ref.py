"""Plain 64-bit forms of the adapted layer's operators, for the tests: the
dropout mask from numpy's unsigned words, products and activations in fp64."""
from __future__ import annotations

import math

import numpy as np
import torch

U16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}       # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}    # at least half a subnormal step
U32 = 2.0 ** -24


def philox4x32_7(counter, key):
    """One call: four 32-bit words of counter and two of key, python integers."""
    c, k = list(counter), list(key)
    for _ in range(7):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p: float) -> int:
    return int(np.floor(np.float32(p) * np.float32(65536) + np.float32(0.5)))


def keep(elements, p: float, seed: int, offset: int) -> np.ndarray:
    """Truth values of the given flat element indices (numpy int64)."""
    u = np.uint64
    e = np.asarray(elements).astype(np.uint64)
    g = e >> u(3)
    lo = u(0xFFFFFFFF)
    c = [g & lo, g >> u(32), np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(7):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> u(32)) ^ c[1] ^ u(k[0]), p1 & lo, (p0 >> u(32)) ^ c[3] ^ u(k[1]), p0 & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.stack(c, -1)
    lane = (e & u(7)).astype(np.int64)
    word = np.take_along_axis(words, (lane >> 1)[..., None], -1)[..., 0]
    half = np.where(lane & 1, word >> u(16), word & u(0xFFFF))
    return half >= threshold(p)


def factor(p: float) -> float:
    return 65536.0 / (65536 - threshold(p))


def mask(shape, p, seed, offset, first=0) -> torch.Tensor:
    """keep / (1 - p) of a tensor of this shape whose first element has flat index `first`, in fp64."""
    n = int(np.prod(shape))
    if threshold(p) == 0:
        return torch.ones(shape, dtype=torch.float64)
    k = keep(np.arange(first, first + n, dtype=np.int64), p, seed, offset)
    return torch.from_numpy(k.reshape(shape)).double() * factor(p)


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.special.expit(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.special.expit(z)
        return s + z * s * torch.special.expit(-z)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


# Largest |act'| and |act''| over the reals, rounded up.
LIPSCHITZ = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}
CURVE = {"none": 0.0, "silu": 0.5, "gelu": 0.8, "gelu_tanh": 0.81}


def act_err(z):
    """Rounding of an fp32 activation at z: the logistic's exp (argument error carried, 2 steps), sum and
    reciprocal (1 step each), the cubic's three steps scaled by the argument's slope (|2 t'| z <= 8 where the
    logistic has not reached its limit), the product; 64 half steps cover them all."""
    return 64 * U32 * z.abs()

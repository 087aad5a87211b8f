"""The activations of nf4_linear and their slopes in nf4_act_grad at every value of a 16-bit type."""
import math

import numpy as np
import pytest
import torch

import quantized_lora_fine_nf4_amd as q
from adapted_ref import TINY, U16, U32
from conftest import print_case

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float16]
IDS = ["bf16", "fp16"]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
N = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()


def every_value(dtype):
    """All 65,536 bit patterns of the type."""
    return torch.from_numpy(np.arange(N, dtype=np.uint16).view(np.int16).copy()).view(dtype)


def act_id(name):
    return getattr(q, "NF4_ACT_" + name.upper())


def forward(bias, act, m, out_dtype, x=None):
    """(out, preact) of nf4_linear over a weight of zeros, so that z is the bias (plus 0 x)."""
    rows, cols, dt = bias.numel(), 128, bias.dtype
    codes = torch.full((rows * cols // 2,), 0x77, dtype=torch.uint8, device="cuda")   # level 7 is 0
    absmax = torch.ones(rows * cols // 64, device="cuda")
    layer = q.nf4_layer(rows * cols, None, codes.data_ptr(), absmax.data_ptr(), None, None, None)
    f = q.fmt(q.NF4_BF16 if dt == torch.bfloat16 else q.NF4_FP16, dq=False)
    x = torch.zeros(m, cols, dtype=dt, device="cuda") if x is None else x.cuda()
    out = torch.empty(m, rows, dtype=out_dtype, device="cuda")
    pre = torch.empty(m, rows, dtype=dt, device="cuda")
    ws = torch.empty(max(q.nf4_matmul_workspace_bytes(rows, cols, False, m), 256), dtype=torch.uint8, device="cuda")
    q.nf4_linear(layer, rows, cols, f, x, out, ws, bias=bias.cuda(), act=act_id(act), preact=pre)
    torch.cuda.synchronize()
    return out.cpu(), pre.cpu()


def gradient(z, act, dy=None):
    """(dz, dbias) of nf4_act_grad at z [m, n], dy ones unless given."""
    m, n = z.shape
    dy = torch.ones_like(z) if dy is None else dy
    dz = torch.empty(m, n, dtype=z.dtype, device="cuda")
    db = torch.empty(n, device="cuda")
    ws = torch.empty(max(q.nf4_act_grad_workspace_bytes(m, n), 256), dtype=torch.uint8, device="cuda")
    q.nf4_act_grad(dy.cuda(), z.cuda(), act_id(act), dz, dbias=db, ws=ws)
    torch.cuda.synchronize()
    return dz.cpu(), db.cpu()


# ---- NaN -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("act", ACTS)
def test_nan_preactivation_stays_nan(dtype, act):
    """Every NaN pattern, and no finite value, gives NaN: out and preact forward, dz and dbias of the gradient (none:
    the gradient does not read the preactivation)."""
    print_case("NaN preactivations", dtype, act)
    z = every_value(dtype)
    z[torch.isinf(z)] = 0
    nan = torch.isnan(z)
    for m in (1, 40, 150):
        for out_dtype in (dtype, torch.float32):
            out, pre = forward(z, act, m, out_dtype)
            assert torch.equal(torch.isnan(out), nan.expand(m, N)), (m, out_dtype)
            assert torch.equal(torch.isnan(pre), nan.expand(m, N)), (m, out_dtype)
    dz, db = gradient(z[None], act)
    want = nan if act != "none" else torch.zeros_like(nan)
    assert torch.equal(torch.isnan(dz[0]), want) and torch.equal(torch.isnan(db), want)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("m", [1, 3, 20, 100, 300])
def test_nan_token_reaches_its_outputs_and_gradients(act, m):
    """One token's input NaN (inf - inf in the layer before): that row of out, preact and dz is NaN and so is all of
    dbias; the other rows are finite."""
    print_case("NaN token", act, m)
    g = torch.Generator().manual_seed(m)
    x = torch.randn(m, 128, generator=g).to(torch.float16)
    bad = m // 2
    x[bad, 5] = float("nan")
    out, pre = forward(torch.randn(2048, generator=g).to(torch.float16), act, m, torch.float16, x=x)
    dz, db = gradient(pre, act)
    rows = torch.zeros(m, dtype=torch.bool)
    rows[bad] = True
    for t in (out, pre, dz):
        assert torch.isnan(t[rows]).all() and torch.isfinite(t[~rows]).all()
    assert torch.isnan(db).all()


# ---- infinities ------------------------------------------------------------

@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("m", [1, 40, 300])
def test_infinite_preactivation_gives_the_limit(dtype, act, m):
    """out is infinite at +infinity and 0 at -infinity and at the type's lowest value, as the slopes there are 1 and 0
    for the gradient."""
    print_case("infinite preactivations", dtype, act, m)
    inf, big = float("inf"), torch.finfo(dtype).max
    bias = torch.tensor([inf, -inf, big, -big] * 64, dtype=dtype)
    for out_dtype in (dtype, torch.float32):
        out, pre = forward(bias, act, m, out_dtype)
        want = torch.tensor([inf, 0.0, big, 0.0] * 64, dtype=out_dtype).expand(m, 256)
        assert torch.equal(pre, bias.expand(m, 256))
        assert torch.equal(out, want), out[0, :4]
    dz, db = gradient(bias[None], act)
    want = torch.tensor([[1.0, 0.0, 1.0, 0.0] * 64])
    assert torch.equal(dz.float(), want) and torch.equal(db[None], want)


# ---- accuracy, tails included ----------------------------------------------
#
# Bounds in half steps u = 2^-24 of fp32, to first order (the factor 1.01 covers the second).  Of its own result the
# hardware's 2^t and reciprocal are within a step (2 u).
#   e^x: log2(e) and its product with x are rounded, so t is within 2 u |t| and e^x within (2 |x| + 2) u of itself.
#   S(x) = 1 / (1 + e^-x): e^-x acts with the weight 1 - S; the sum is rounded (1 u), the reciprocal (2 u).
#   P(z): z^2 / 2 is rounded once more, so e = e^(-z^2/2) is within (1.5 z^2 + 2) u.  For z < 0, P = e q(t) t / 2:
#     t = 1 / (1 + c |z|) with three roundings in c, one of the sum and 2 u of the reciprocal, at most 6 u; q(t) t is
#     erfc(x) e^(x^2), whose relative slope in t is at most 3 (x = 0), so 18 u; the polynomial's fit and evaluation 6 u;
#     two products: (1.5 z^2 + 28) u of P.  For z >= 0 the same of 1 - P, and 1 u of P.
#   tanh's argument x = K (z + 0.044715 z^3) has three roundings in the cubic term, and the sum's, K's and the product's:
#     6 u of |x| more in the exponent than S has by itself.
# Where S or e is below the least normal fp32 the kernel has 0.

K_TANH = math.sqrt(8 / math.pi)
LEAST = 2.0 ** -126


def logistic(x, extra):
    """(S, 1 - S, error of S) at x whose own error is `extra` u |x|."""
    s, c = torch.special.expit(x), torch.special.expit(-x)
    return s, c, s * (c * ((2 + extra) * x.abs() + 2) + 3) * U32 + LEAST


def normal(z):
    """(P, error of P) for the normal distribution function."""
    p, other = torch.special.erfc(-z / math.sqrt(2)) / 2, torch.special.erfc(z / math.sqrt(2)) / 2
    return p, torch.minimum(p, other) * (1.5 * z * z + 28) * U32 + (z >= 0) * p * U32 + LEAST


def tanh_argument(z):
    return K_TANH * (z + 0.044715 * z ** 3)


def value(z, act):
    """(act(z), bound); z below -100 counts as -100, where every factor is below 1e-43."""
    if act == "relu":
        return z.clamp(min=0), torch.zeros_like(z)
    lo, c = z.clamp(min=-100), z.clamp(-100, 100)
    if act == "gelu":
        f, err = normal(c)
    else:
        f, _, err = logistic(c, 0) if act == "silu" else logistic(tanh_argument(c), 6)
    return lo * f, lo.abs() * (err + f * U32)


def slope(z, act):
    """(act'(z), bound) with z limited to +-100, beyond which every slope is 0 or 1 within 1e-40."""
    if act == "relu":
        return (z > 0).double(), torch.zeros_like(z)
    z = z.clamp(-100, 100)
    if act == "silu":
        s, c, err = logistic(z, 0)
        inner = 1 + z * c
        d = s * inner
        # S through its derivative; 1 - S, the inner sum and the product rounded
        return d, err * (1 + z * (c - s)).abs() + (s * z.abs() * c + s * inner.abs() + d.abs()) * U32
    if act == "gelu":
        p, err = normal(z)
        density = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        d = p + density
        return d, err + density.abs() * (1.5 * z * z + 4) * U32 + d.abs() * U32 + z.abs() * LEAST
    x = tanh_argument(z)
    w = K_TANH * (1 + 3 * 0.044715 * z * z)   # x', five roundings
    s, c, err = logistic(x, 6)
    term = z * s * c * w
    d = s + term
    return d, err * (1 + z * w * (c - s)).abs() + (8 * term.abs() + d.abs()) * U32


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("act", ACTS[1:])
def test_every_finite_value(dtype, act):
    """act(z) and act'(z) of every finite 16-bit z in fp32 against the bounds above, and rounded once to 16 bits."""
    print_case("every finite value", dtype, act)
    z = every_value(dtype)
    z[~torch.isfinite(z)] = 0
    want, tol = value(z.double(), act)
    out, _ = forward(z, act, 1, torch.float32)
    excess = ((out[0].double() - want).abs() - 1.01 * tol).max().item()
    assert excess <= 0, z[((out[0].double() - want).abs() - 1.01 * tol).argmax()]
    out, _ = forward(z, act, 1, dtype)
    assert ((out[0].double() - want).abs() <= 1.01 * tol + U16[dtype] * want.abs() + TINY[dtype]).all()
    want, tol = slope(z.double(), act)
    dz, db = gradient(z[None], act)
    excess = ((db.double() - want).abs() - 1.01 * tol).max().item()
    assert excess <= 0, z[((db.double() - want).abs() - 1.01 * tol).argmax()]
    assert ((dz[0].double() - want).abs() <= 1.01 * tol + U16[dtype] * want.abs() + TINY[dtype]).all()


def test_the_bounds_see_a_lost_tail():
    """The bounds against forms that lose the tail: 0 below -5, and the logistic's argument cut at -20."""
    z = every_value(torch.bfloat16)
    z = z[torch.isfinite(z)].double()
    for act in ACTS[2:]:
        want, tol = value(z, act)
        assert (want.abs() > 1.01 * tol)[(z < -5) & (z > -9)].all(), act
    want, tol = value(z, "silu")
    cut = z * torch.special.expit(z.clamp(min=-20))
    assert ((cut - want).abs() > 1.01 * tol)[(z < -21) & (z > -80)].all()

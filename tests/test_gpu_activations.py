"""The activations of nf4_linear and their slopes in nf4_act_grad at every value of a 16-bit type."""
import numpy as np
import pytest
import torch

import quantized_lora_fine_nf4_amd as q
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

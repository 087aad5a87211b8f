"""The adapted layer's operators (nf4_dropout, nf4_act_grad, nf4_lora_project,
nf4_lora_grad, nf4_linear) against their 64-bit forms (adapted_ref.py).

Tolerances, elementwise.  Products of two 16-bit values are exact in fp32; a
sum of K of them in any order and rounding is within 2 K 2^-24 of the sum of
their magnitudes (the matrix core may round each addition toward zero: one step
instead of half of one).  A 16-bit result adds half a step of it; fp32 factors
and sums add a few 2^-24 of what they act on, counted at each test.
"""
import numpy as np
import pytest
import torch

import adapted_ref as ref
import quantized_lora_fine_nf4_amd as q
from adapted_ref import TINY, U16, U32
from conftest import print_case

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float16]
IDS = ["bf16", "fp16"]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
SEED, OFFSET = 0x1234_5678_9ABC_DEF0, 0x0FED_CBA9_8765_4321


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()


def rng(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def act_id(name):
    return getattr(q, "NF4_ACT_" + name.upper())


def draw(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def guarded(shape, dtype, pad=64):
    """A poisoned tensor of this shape with poisoned elements before and after it."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape)


def untouched(buf, shape, pad=64):
    n = int(np.prod(shape))
    return bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[pad + n:]).all())


def workspace(nbytes):
    """Filled with NaN bits: partials of nobody must not be read."""
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None


def check(got, want, tol, what=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    excess = ((got - want).abs() / tol).max().item()
    assert excess <= 1.0, (what, excess)
    return excess


# ---- dropout ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 8192, 100_003])
@pytest.mark.parametrize("p", [2.0 ** -16, 0.1, 0.5, 65535 / 65536])
def test_dropout_is_the_defined_mask(dtype, n, p):
    """Bit for bit: the kept elements are x times the fp32 factor, rounded once."""
    print_case("nf4_dropout", dtype, n, p)
    x = draw((n,), dtype, n)
    buf, out = guarded((n,), dtype)
    q.nf4_dropout(x.cuda(), out, p, rng())
    k = torch.from_numpy(ref.keep(np.arange(n), p, SEED, OFFSET))
    want = torch.where(k, (x.float() * torch.tensor(ref.factor(p), dtype=torch.float32)).to(dtype), torch.zeros((), dtype=dtype))
    assert torch.equal(out.cpu(), want)
    assert untouched(buf, (n,))


def test_dropout_keeps_the_stated_share():
    """Kept shares of 2^20 elements under five seeds and three offsets each: within 5 standard deviations
    (sqrt(p (1 - p) / n) = 2.9e-4 at p = 0.1) of 1 - p, and no two masks equal."""
    n, p = 1 << 20, 0.1
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    seen = set()
    for seed in range(5):
        for off in (0, 1, 1 << 40):
            q.nf4_dropout(x, out, p, rng(seed, off))
            kept = (out != 0).float().mean().item()
            t = ref.threshold(p) / 65536
            assert abs(kept - (1 - t)) < 5 * (t * (1 - t) / n) ** 0.5
            seen.add(out.cpu().view(torch.int16).numpy().tobytes())
    assert len(seen) == 15


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_dropout_zero_probability_in_place_and_dropped_infinities(dtype):
    x = draw((1000,), dtype, 3).cuda()
    out = torch.empty_like(x)
    q.nf4_dropout(x, out, 0.0, None)
    assert torch.equal(out, x)
    q.nf4_dropout(x, out, 0.3, rng())
    y = x.clone()
    q.nf4_dropout(y, y, 0.3, rng())
    assert torch.equal(y, out)
    k = torch.from_numpy(ref.keep(np.arange(1000), 0.3, SEED, OFFSET)).cuda()
    bad = x.clone()
    bad[~k] = float("nan")
    bad[(~k).nonzero()[::2, 0]] = float("inf")
    q.nf4_dropout(bad, bad, 0.3, rng())
    assert torch.equal(bad, out)


def test_dropout_past_32_bit_offsets():
    """2^32 + 1003 elements: the mask past element 2^32 (group index past 2^29, byte offset past 2^33)."""
    n = (1 << 32) + 1003
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    q.nf4_dropout(x, x, 0.5, rng())
    for first in (0, (1 << 31) - 500, (1 << 32) - 500, n - 999):
        count = min(1000, n - first)
        want = ref.keep(first + np.arange(count, dtype=np.int64), 0.5, SEED, OFFSET)
        assert np.array_equal((x[first:first + count] != 0).cpu().numpy(), want), first


# ---- the epilogue's gradient -----------------------------------------------

@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n", [(1, 8), (3, 40), (33, 512), (257, 1000), (64, 4096), (2500, 24)])
def test_act_grad(dtype, act, m, n):
    """dz: half a step, and in fp32 the slope's error: the logistic within 8 half steps, times up to 1 + |z| where
    it is multiplied by z (limited to where it differs from its limit, |z| < 20 in fp32); 64 (1 + |z|) half steps
    of dy cover it.  dbias: the sum of those errors and m half steps (doubled) of the sum of magnitudes."""
    print_case("nf4_act_grad", dtype, act, m, n)
    dy, z = draw((m, n), dtype, m + n, 0.3), draw((m, n), dtype, 2 * m + n, 2.0)
    z[0, 0], z[0, 1], z[0, 2] = 0.0, 30.0, -30.0
    buf, dz = guarded((m, n), dtype)
    bbuf, db = guarded((n,), torch.float32)
    ws = workspace(q.nf4_act_grad_workspace_bytes(m, n))
    dyd, zd = dy.cuda(), z.cuda()
    q.nf4_act_grad(dyd, None if act == "none" else zd, act_id(act), dz, dbias=db, ws=ws)
    want = dy.double() * ref.slope(z.double(), act)
    err = dy.double().abs() * 64 * U32 * (1 + z.double().abs().clamp(max=20))
    check(dz, want, U16[dtype] * want.abs() + 1.01 * err + TINY[dtype], "dz")
    check(db, want.sum(0), err.sum(0) + 2 * (m + 8) * U32 * want.abs().sum(0) + 1e-30, "dbias")
    assert untouched(buf, (m, n)) and untouched(bbuf, (n,))
    # without the bias gradient, and in place
    again = dyd.clone()
    q.nf4_act_grad(again, None if act == "none" else zd, act_id(act), again)
    assert torch.equal(again, dz)
    # the bias gradient alone, and again: the same bits
    db2 = torch.full_like(db, float("nan"))
    q.nf4_act_grad(dyd, zd, act_id(act), None if act == "none" else torch.empty_like(dz), dbias=db2, ws=ws)
    assert torch.equal(db, db2)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("act", ACTS[1:])
def test_act_grad_of_infinite_preactivations(dtype, act):
    """A 16-bit preactivation that overflowed: the slope's limits 1 and 0."""
    z = torch.tensor([[float("inf"), float("-inf")] * 4], dtype=dtype, device="cuda")
    dy = torch.full((1, 8), 3.0, dtype=dtype, device="cuda")
    dz = torch.empty_like(dy)
    q.nf4_act_grad(dy, z, act_id(act), dz)
    assert torch.equal(dz.cpu().float(), torch.tensor([[3.0, 0.0] * 4]))


def test_act_grad_past_32_bit_offsets():
    """2^32 + 2^16 elements: the last rows against the same rows alone."""
    n, m = 1 << 16, (1 << 16) + 1
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    dy[-3:] = draw((3, n), torch.bfloat16, 1).cuda()
    z[-3:] = draw((3, n), torch.bfloat16, 2).cuda()
    ws = workspace(q.nf4_act_grad_workspace_bytes(m, n))
    db = torch.empty(n, device="cuda")
    tail, tail_dy, tail_z = torch.empty_like(dy[-3:]), dy[-3:].clone(), z[-3:].clone()
    q.nf4_act_grad(dy, z, q.NF4_ACT_SILU, dy, dbias=db, ws=ws)
    q.nf4_act_grad(tail_dy, tail_z, q.NF4_ACT_SILU, tail)
    assert torch.equal(dy[-3:], tail)
    assert not dy[:-3].any()
    want = (tail_dy.double() * ref.slope(tail_z.double(), "silu")).sum(0).cpu()
    mag = (tail_dy.double() * ref.slope(tail_z.double(), "silu")).abs().sum(0).cpu() + 3.0
    check(db, want, 64 * 21 * U32 * mag)


# ---- the adapter's products ------------------------------------------------

@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("back,p", [(False, 0.0), (False, 0.2), (True, 0.0)], ids=["fwd", "drop", "bwd"])
@pytest.mark.parametrize("m,k,r", [(1, 8, 1), (1, 5120, 16), (5, 136, 4), (16, 128, 16), (17, 1000, 24), (33, 2048, 64),
                                   (1030, 264, 20), (1100, 520, 64), (1025, 128, 128), (40, 4104, 100),
                                   # 16 ranks a workgroup and 32 rows; 32 ranks; 64 ranks and 32 rows; any-rank gathers
                                   (4100, 72, 7), (2100, 200, 30), (2200, 136, 61), (4200, 80, 127), (4112, 64, 16)])
def test_project(dtype, back, p, m, k, r):
    """Half a step, and in fp32: k products summed (k / 32 matrix steps per wave, up to 16 waves), scale times
    factor and the product with it (3 half steps)."""
    print_case("nf4_lora_project", dtype, "bwd" if back else "fwd", p, m, k, r)
    x, w = draw((m, k), dtype, m + k + r), draw((k, r) if back else (r, k), dtype, k + r, k ** -0.5)
    buf, h = guarded((m, r), dtype)
    q.nf4_lora_project(x.cuda(), w.cuda(), h, scale=1.7, backward=back, p=p, rng=rng() if p else None)
    wd = w.double() if back else w.double().t()
    xd = x.double() * ref.mask((m, k), p, SEED, OFFSET)
    want, mag = 1.7 * xd @ wd, 1.7 * xd.abs() @ wd.abs()
    check(h, want, U16[dtype] * want.abs() + 1.01 * (2 * k + 8) * U32 * mag + TINY[dtype])
    assert untouched(buf, (m, r))
    h2 = torch.empty_like(h)
    q.nf4_lora_project(x.cuda(), w.cuda(), h2, scale=1.7, backward=back, p=p, rng=rng() if p else None)
    assert torch.equal(h, h2)


def test_project_masks_as_dropout_does():
    """Dropped infinities and NaN add nothing, and the mask is nf4_dropout's."""
    m, k, r, p = 50, 256, 16, 0.25
    x, w = draw((m, k), torch.bfloat16, 1).cuda(), draw((r, k), torch.bfloat16, 2).cuda()
    h, h2 = (torch.empty(m, r, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q.nf4_lora_project(x, w, h, p=p, rng=rng())
    ones = torch.ones_like(x)
    q.nf4_dropout(ones, ones, p, rng())
    x[ones == 0] = float("nan")
    x[(ones == 0) & (torch.rand(m, k, device="cuda") < 0.5)] = float("inf")
    q.nf4_lora_project(x, w, h2, p=p, rng=rng())
    assert torch.equal(h, h2)


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("k,r", [(8, 16), (136, 16), (136, 4), (136, 5), (1000, 40), (552, 64)])
def test_project_infinite_last_weight(back, k, r):
    """Lengths that end inside a step: an infinite weight in the last place stays an infinity."""
    x = draw((37, k), torch.bfloat16, 1).abs().cuda() + 0.5
    w = draw((k, r) if back else (r, k), torch.bfloat16, 2).cuda()
    (w if back else w.t())[k - 1, r - 1] = float("-inf")
    h = torch.empty(37, r, dtype=torch.bfloat16, device="cuda")
    q.nf4_lora_project(x, w, h, backward=back)
    assert (h[:, r - 1] == float("-inf")).all() and h[:, :r - 1].isfinite().all()


def test_project_past_32_bit_offsets():
    """(2^19 + 5) x 8192: the last rows' mask and product, against the 64-bit form."""
    m, k, r, p = (1 << 19) + 5, 8192, 8, 0.5
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    t = draw((20, k), torch.bfloat16, 5)
    x[-20:] = t.cuda()
    w = draw((r, k), torch.bfloat16, 6, 0.01)
    h = torch.empty(m, r, dtype=torch.bfloat16, device="cuda")
    q.nf4_lora_project(x, w.cuda(), h, p=p, rng=rng())
    assert not h[:-20].any()
    xd = t.double() * ref.mask((20, k), p, SEED, OFFSET, first=(m - 20) * k)
    want, mag = xd @ w.double().t(), xd.abs() @ w.double().abs().t()
    check(h[-20:], want, U16[torch.bfloat16] * want.abs() + 1.01 * (2 * k + 8) * U32 * mag)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("side,p", [("A", 0.0), ("A", 0.2), ("B", 0.0)], ids=["A", "A-drop", "B"])
@pytest.mark.parametrize("m,n,r", [(1, 8, 1), (1, 128, 16), (31, 136, 5), (33, 1000, 16), (300, 264, 24),
                                   (777, 2048, 64), (2500, 64, 128), (1300, 136, 100), (4096, 256, 16), (500, 264, 30),
                                   (600, 136, 61), (900, 72, 127)])
def test_lora_grad(dtype, side, p, m, n, r):
    """fp32: m products summed (in 32-row matrix steps, waves and splits) and the factor (2 half steps)."""
    print_case("nf4_lora_grad", dtype, side, p, m, n, r)
    u, x = draw((m, r), dtype, m + r, 0.5), draw((m, n), dtype, m + n)
    shape = (r, n) if side == "A" else (n, r)
    buf, grad = guarded(shape, torch.float32)
    need = q.nf4_lora_grad_workspace_bytes(m, n, r)
    q.nf4_lora_grad(u.cuda(), x.cuda(), grad, workspace(need), side=side, p=p, rng=rng() if p else None)
    xd, ud = x.double() * ref.mask((m, n), p, SEED, OFFSET), u.double()
    want, mag = ud.t() @ xd, ud.abs().t() @ xd.abs()
    if side == "B":
        want, mag = want.t(), mag.t()
    check(grad, want, (2 * m + 8) * U32 * mag + 1e-30)
    assert untouched(buf, shape)
    g2 = torch.empty_like(grad)
    q.nf4_lora_grad(u.cuda(), x.cuda(), g2, workspace(need), side=side, p=p, rng=rng() if p else None)
    assert torch.equal(grad, g2)


@pytest.mark.parametrize("side", ["A", "B"])
@pytest.mark.parametrize("m,n,r", [(1, 8, 16), (33, 136, 16), (47, 128, 4), (1999, 64, 64), (550, 264, 5)])
def test_lora_grad_infinite_last_token(side, m, n, r):
    """Token counts that end inside a step: an infinity in the last token stays one, in u or in x."""
    for of_u in (True, False):
        u = draw((m, r), torch.float16, 1).abs().cuda() + 0.5
        x = draw((m, n), torch.float16, 2).abs().cuda() + 0.5
        (u if of_u else x)[m - 1, 0] = float("inf")
        grad = torch.empty((r, n) if side == "A" else (n, r), device="cuda")
        q.nf4_lora_grad(u, x, grad, workspace(q.nf4_lora_grad_workspace_bytes(m, n, r)), side=side)
        rows = grad if (side == "A") == of_u else grad.t()
        assert (rows[0] == float("inf")).all() and rows[1:].isfinite().all()


def test_lora_grad_past_32_bit_offsets():
    m, n, r, p = (1 << 18) + 7, 1 << 14, 16, 0.5
    x = torch.ones(m, n, dtype=torch.bfloat16, device="cuda")
    u = torch.zeros(m, r, dtype=torch.bfloat16, device="cuda")
    t = draw((9, r), torch.bfloat16, 5)
    u[-9:] = t.cuda()
    grad = torch.empty(r, n, device="cuda")
    q.nf4_lora_grad(u, x, grad, workspace(q.nf4_lora_grad_workspace_bytes(m, n, r)), p=p, rng=rng())
    k = ref.mask((9, n), p, SEED, OFFSET, first=(m - 9) * n)
    want, mag = t.double().t() @ k, t.double().abs().t() @ k
    check(grad, want, 64 * U32 * mag + 1e-30)


# ---- the linear layer ------------------------------------------------------

class Weight:
    """A matrix in NF4 form on the GPU: any codes, constants near those of N(0, 0.02) blocks."""

    def __init__(self, rows, cols, dtype, dq, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        nb = rows * cols // 64
        self.rows, self.cols, self.dtype = rows, cols, dtype
        self.codes = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
        self.f = q.fmt(q.NF4_BF16 if dtype == torch.bfloat16 else q.NF4_FP16, dq)
        ptr = lambda t: int(t.data_ptr())
        if dq:
            self.qa = torch.randint(40, 128, (nb,), generator=g, device="cuda", dtype=torch.int8)
            self.s2 = torch.rand(-(-nb // 256), generator=g, device="cuda") * 2e-4 + 4e-4
            self.const = self.qa.float() * self.s2.repeat_interleave(256)[:nb]
            self.layer = q.nf4_layer(rows * cols, None, ptr(self.codes), None, ptr(self.qa), ptr(self.s2), None)
        else:
            self.const = torch.rand(nb, generator=g, device="cuda") * 0.05 + 0.02
            self.layer = q.nf4_layer(rows * cols, None, ptr(self.codes), ptr(self.const), None, None, None)

    def dense(self):
        lv = torch.from_numpy(q.nf4_levels()).cuda()
        w = torch.stack([lv[(self.codes & 15).int()], lv[(self.codes >> 4).int()]], 1).view(-1, 64)
        return (w * self.const[:, None]).to(self.dtype).double().view(self.rows, self.cols)


class Case:
    """Operands of one nf4_linear call on the GPU and its 64-bit result with its error bound."""

    def __init__(self, W, m, r, back, p=0.0, act="none", bias=False, residual=False, out_f32=False, seed=0):
        dt = W.dtype
        kred, ncol = (W.rows, W.cols) if back else (W.cols, W.rows)
        self.W, self.m, self.back, self.p, self.act, self.out_f32, self.ncol = W, m, back, p, act, out_f32, ncol
        d = lambda shape, s, std=1.0, t=dt: draw(shape, t, seed + s, std).cuda()
        self.x = d((m, kred), 1)
        self.lora = (d((m, r), 2, 0.5), d((r, ncol) if back else (ncol, r), 3, 0.2)) if r else None
        self.bias = d((ncol,), 4) if bias else None
        self.res = d((m, ncol), 5, 1.0, torch.float32 if out_f32 else dt) if residual else None

    def run(self, preact=False, ws="own", inplace=False):
        need = q.nf4_matmul_workspace_bytes(self.W.rows, self.W.cols, self.back, self.m)
        ws = workspace(need) if isinstance(ws, str) else ws
        buf, out = guarded((self.m, self.ncol), torch.float32 if self.out_f32 else self.W.dtype)
        res = self.res
        if inplace:
            out.copy_(res)
            res = out
        pbuf, pre = guarded((self.m, self.ncol), self.W.dtype) if preact else (None, None)
        q.nf4_linear(self.W.layer, self.W.rows, self.W.cols, self.W.f, self.x, out, ws, backward=self.back,
                     lora=self.lora, bias=self.bias, act=act_id(self.act), preact=pre, residual=res, p=self.p,
                     rng=rng() if self.p else None)
        assert untouched(buf, out.shape) and (pbuf is None or untouched(pbuf, out.shape))
        return (out, pre) if preact else out

    def expect(self, rows=None):
        """(z, its error, out, its error) for the given rows, on the CPU."""
        idx = slice(None) if rows is None else rows
        x, W = self.x[idx].double(), self.W.dense()
        Wt = W if self.back else W.t().contiguous()
        z, mag = x @ Wt, x.abs() @ Wt.abs()
        terms = x.shape[1]
        if self.lora:
            u, v = self.lora[0][idx].double(), self.lora[1].double()
            v = v if self.back else v.t().contiguous()
            lr, lm = u @ v, u.abs() @ v.abs()
            if self.p:
                every = range(self.m) if rows is None else rows
                k = torch.cat([ref.mask((1, self.ncol), self.p, SEED, OFFSET, first=int(i) * self.ncol) for i in every])
                lr, lm = lr * k.cuda(), lm * k.cuda()
            z, mag, terms = z + lr, mag + lm, terms + u.shape[1]
        if self.bias is not None:
            z, mag = z + self.bias.double(), mag + self.bias.double().abs()
        # the sums, the factor, its product, the bias and the splits' sums
        ez = 2 * (terms + 24) * U32 * mag + 1e-30
        out = ref.act(z, self.act)
        eo = ref.LIPSCHITZ[self.act] * ez + (ref.act_err(z) if self.act != "none" else 0)
        if self.res is not None:
            r = self.res[idx].double()
            eo = eo + U32 * (out.abs() + r.abs())
            out = out + r
        if not self.out_f32:
            eo = 1.01 * eo + U16[self.W.dtype] * out.abs() + TINY[self.W.dtype]
        return z.cpu(), ez.cpu(), out.cpu(), eo.cpu()

    def check(self, out, pre=None, rows=None):
        z, ez, o, eo = self.expect(rows)
        idx = slice(None) if rows is None else torch.as_tensor(rows, device="cuda")
        check(out[idx], o, eo, "out")
        if pre is not None:
            dt = self.W.dtype
            check(pre[idx], z, U16[dt] * z.abs() + 1.01 * ez + TINY[dt], "preact")


# m: the few-token kernel (1, 5, 16, 17, 32), 128 x 128 tiles split (33, 128) and whole (200 without room to
# split), 256 x 256 tiles split (300 with a long reduction)
@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,cols,m", [(256, 384, 1), (128, 128, 5), (512, 256, 16), (256, 384, 17), (128, 1024, 32),
                                         (256, 384, 33), (384, 128, 128), (256, 128, 200), (128, 2048, 300)])
@pytest.mark.parametrize("r,act,bias,residual,f32", [(16, "none", False, False, False), (0, "gelu", True, False, False),
                                                     (8, "silu", True, True, True), (5, "gelu_tanh", False, True, False),
                                                     (67, "none", True, True, True),
                                                     (100, "relu", True, False, True), (128, "silu", False, False, False)])
def test_linear_forward(dtype, rows, cols, m, r, act, bias, residual, f32):
    print_case("nf4_linear", dtype, rows, cols, m, r, act, bias, residual, f32)
    W = Weight(rows, cols, dtype, dq=(r % 8 == 0), seed=rows + cols)
    c = Case(W, m, r, False, act=act, bias=bias, residual=residual, out_f32=f32, seed=m + r)
    out, pre = c.run(preact=True)
    c.check(out, pre)
    assert torch.equal(c.run(), out)             # again, without the preactivation: the same bits
    if residual:
        assert torch.equal(c.run(inplace=True), out)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,cols,m", [(256, 384, 1), (128, 128, 33), (384, 256, 77), (256, 128, 200), (2048, 128, 300),
                                         (256, 5120, 200)])
@pytest.mark.parametrize("r,p,residual,f32", [(16, 0.0, False, False), (0, 0.0, True, False), (8, 0.1, True, True),
                                              (5, 0.5, False, False), (100, 0.1, True, False), (128, 0.0, False, True),
                                              (67, 0.1, False, False), (127, 0.0, True, True),
                                              (128, 0.3, False, True)])
def test_linear_backward(dtype, rows, cols, m, r, p, residual, f32):
    print_case("nf4_linear backward", dtype, rows, cols, m, r, p, residual, f32)
    W = Weight(rows, cols, dtype, dq=(r % 8 == 0), seed=rows + cols)
    c = Case(W, m, r, True, p=p, residual=residual, out_f32=f32, seed=m + r)
    out = c.run()
    c.check(out)
    assert torch.equal(c.run(), out)
    if residual:
        assert torch.equal(c.run(inplace=True), out)


# whole 256 x 256 tiles: one round short of full, whole rounds with leftover tiles split (with a workspace that the
# shape asks for) and row pieces of leftover tiles (a reduction too short to split)
BIG = [(False, 13824, 256, 700), (False, 4992, 4096, 3900), (False, 5120, 256, 3300), (True, 256, 9216, 1000),
       (True, 4096, 4992, 3900), (True, 256, 5120, 3300), (True, 256, 5120, 3100)]


@pytest.mark.parametrize("back,rows,cols,m", BIG, ids=[f"{'bwd' if b else 'fwd'}-{r}x{c}-{m}" for b, r, c, m in BIG])
@pytest.mark.parametrize("dtype,r,f32", [(torch.bfloat16, 16, False), (torch.float16, 72, True), (torch.bfloat16, 93, True)],
                         ids=["bf16-r16", "fp16-r72-f32", "bf16-r93-f32"])
def test_linear_large_tiles(back, rows, cols, m, dtype, r, f32):
    """Sampled rows of every tile row's first and last, and every row of the last 300."""
    print_case("nf4_linear large tiles", dtype, "bwd" if back else "fwd", rows, cols, m, r)
    W = Weight(rows, cols, dtype, dq=not f32, seed=rows + cols)
    kw = dict(p=0.1) if back else dict(act="silu", bias=True)
    c = Case(W, m, r, back, residual=True, out_f32=f32, seed=m + r, **kw)
    out, pre = (c.run(), None) if back else c.run(preact=True)
    idx = sorted({i for t in range(0, m, 256) for i in (t, min(t + 255, m - 1))} | set(range(max(0, m - 300), m)))
    c.check(out, pre, rows=idx)
    assert torch.equal(c.run(), out)
    if back:   # without dropout too: the accumulators' own path
        c.p = 0.0
        c.check(c.run(), None, rows=idx)


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
def test_linear_past_32_bit_offsets(back):
    """160,000 x 13,824 outputs (2.2e9): the last rows, with preactivation and residual forward (in place) and the
    mask of the low-rank term backward."""
    rows, cols, m, r = (128, 13824, 160_000, 8) if back else (13824, 128, 160_000, 8)
    print_case("nf4_linear past 32 bits", "bwd" if back else "fwd")
    W = Weight(rows, cols, torch.bfloat16, True, seed=3)
    kw = dict(p=0.2) if back else dict(act="silu", bias=True)
    c = Case(W, m, r, back, seed=9, **kw)
    idx = [0, 77_000, 155_343, 155_344] + list(range(m - 40, m))
    if back:
        c.check(c.run(), None, rows=idx)
        return
    c.res = torch.ones(m, c.ncol, dtype=torch.bfloat16, device="cuda")
    out, pre = torch.empty_like(c.res), torch.empty_like(c.res)
    need = q.nf4_matmul_workspace_bytes(rows, cols, back, m)
    out.fill_(1.0)
    q.nf4_linear(W.layer, rows, cols, W.f, c.x, out, workspace(need), lora=c.lora, bias=c.bias, act=q.NF4_ACT_SILU,
                 preact=pre, residual=out)
    c.check(out, pre, rows=idx)


def test_linear_empty_epilogue_is_the_matmul():
    for back, m in ((False, 1), (False, 100), (False, 600), (True, 20), (True, 600)):
        W = Weight(2048, 1024, torch.bfloat16, True, 5)
        c = Case(W, m, 0, back, out_f32=True)
        out = c.run()
        want = torch.empty_like(out)
        ws = workspace(q.nf4_matmul_workspace_bytes(W.rows, W.cols, back, m))
        q.nf4_matmul_ws(W.layer, W.rows, W.cols, W.f, c.x, want, ws, backward=back)
        assert torch.equal(out, want), (back, m)


# parts of the reduction (its super-chunks of 128): one (1), two (8 + 1), three (8 + 8 + 1), five (2 x 4 + 1), nine, nine
# (4 x 8 + 1), sixteen, and one of more workgroups than the chip holds at once
@pytest.mark.parametrize("rows,cols", [(128, 128), (16384, 1152), (16384, 2176), (8192, 1152), (1024, 1152), (4096, 4224),
                                       (2048, 8192), (32768, 384)])
@pytest.mark.parametrize("dtype,dq,f32", [(torch.bfloat16, True, False), (torch.float16, False, True)], ids=["dq", "plain"])
def test_linear_single_token(rows, cols, dtype, dq, f32):
    print_case("nf4_linear single token", dtype, rows, cols)
    W = Weight(rows, cols, dtype, dq, seed=rows + cols)
    c = Case(W, 1, 40, False, act="silu", bias=True, residual=True, out_f32=f32, seed=3)
    out, pre = c.run(preact=True)
    c.check(out, pre)
    assert torch.equal(c.run(inplace=True), out)
    # as the first of two tokens, the other one not finite: the same bits
    two = Case(W, 2, 40, False, act="silu", bias=True, residual=True, out_f32=f32, seed=4)
    two.x[0], two.lora[0][0], two.res[0] = c.x[0], c.lora[0][0], c.res[0]
    two.x[1] = float("nan")
    two.lora = (two.lora[0], c.lora[1])
    two.bias = c.bias
    both, pre2 = two.run(preact=True)
    assert torch.equal(both[0], out[0]) and torch.equal(pre2[0], pre[0]) and torch.isnan(both[1]).all()
    # and without an epilogue, as the matmul
    bare = Case(W, 1, 0, False, out_f32=f32, seed=3)
    want = torch.empty(1, rows, dtype=out.dtype, device="cuda")
    q.nf4_matmul_ws(W.layer, rows, cols, W.f, bare.x, want, workspace(q.nf4_matmul_workspace_bytes(rows, cols, False, 1)))
    assert torch.equal(bare.run(), want)


def test_linear_one_dimensional_token():
    W = Weight(256, 128, torch.bfloat16, True, 5)
    c = Case(W, 1, 8, False, act="silu", residual=True)
    want = c.run()
    out = torch.empty(256, dtype=torch.bfloat16, device="cuda")
    ws = workspace(q.nf4_matmul_workspace_bytes(256, 128, False, 1))
    q.nf4_linear(W.layer, 256, 128, W.f, c.x[0], out, ws, lora=c.lora, act=q.NF4_ACT_SILU, residual=c.res[0])
    assert torch.equal(out, want[0])


def test_linear_dropped_low_rank_values_add_nothing():
    """An infinite adapter column: kept elements are infinite, dropped ones are the product alone."""
    W = Weight(256, 384, torch.bfloat16, True, 5)
    for m in (20, 600):
        c = Case(W, m, 8, True, p=0.5, out_f32=True)
        c.lora[0][:] = 1.0
        c.lora[1][:, 7] = 1e38
        out = c.run()
        plain = Case(W, m, 0, True, out_f32=True)
        plain.x = c.x
        base = plain.run()
        k = ref.mask((m, 384), 0.5, SEED, OFFSET)[:, 7].bool().cuda()
        assert torch.isinf(out[k, 7]).all() and torch.equal(out[~k, 7], base[~k, 7])


# rows, cols, m and the workspace in bytes that shows the plan: 256 x 256 tiles split in two (16 k-steps each; 128 x 128
# tiles would be split in sixteen), whole (more than 256 tiles of 128 x 128, a reduction too short to split), and whole
# with the leftover tiles split (320 tiles, 64 of them in four splits of 256 x 256 partials)
@pytest.mark.parametrize("rows,cols,m,need", [(2048, 128, 300, 2 * 300 * 128 * 4), (256, 9216, 1000, 0),
                                              (4096, 4992, 3900, 4 * 64 * 256 * 256 * 4)], ids=["split", "whole", "tail"])
@pytest.mark.parametrize("r", [8, 72])
def test_large_tiles_dropped_low_rank_values_add_nothing(rows, cols, m, need, r):
    """Infinite adapter columns in the 256 x 256 kernels' own store: kept elements are infinite, dropped ones the
    product alone."""
    print_case("dropped infinities, large tiles", rows, cols, m, r)
    assert q.nf4_matmul_workspace_bytes(rows, cols, True, m) == need
    W = Weight(rows, cols, torch.bfloat16, True, 5)
    c = Case(W, m, r, True, p=0.5, out_f32=True)
    at = [7, 64, cols - 1]
    c.lora[0][:] = 1.0
    c.lora[1][:, at] = 1e38
    out = c.run()
    plain = Case(W, m, 0, True, out_f32=True)
    plain.x = c.x
    base = plain.run()
    k = ref.mask((m, cols), 0.5, SEED, OFFSET)[:, at].bool().cuda()
    assert torch.isinf(out[:, at][k]).all() and torch.equal(out[:, at][~k], base[:, at][~k])


# ---- together --------------------------------------------------------------

class Layer:
    """One adapted layer's buffers and its forward and backward run, as a training program makes them."""

    def __init__(self, rows, cols, m, r, dtype, act, p, scale, seed=0):
        self.W = Weight(rows, cols, dtype, True, seed)
        self.m, self.r, self.act, self.p, self.s, self.dt = m, r, act, p, scale, dtype
        d = lambda shape, s, std=1.0: draw(shape, dtype, seed + s, std).cuda()
        e = lambda shape, t=dtype: torch.empty(shape, dtype=t, device="cuda")
        self.x, self.A, self.B = d((m, cols), 1), d((r, cols), 2, cols ** -0.5), d((rows, r), 3, 0.1)
        self.bias, self.res, self.dy = d((rows,), 4, 0.1), d((m, rows), 5), d((m, rows), 6, 0.3)
        self.dxin = d((m, cols), 7)
        self.rng = rng()
        self.h, self.z, self.out = e((m, r)), e((m, rows)), e((m, rows))
        self.dz, self.db, self.dh = e((m, rows)), e((rows,), torch.float32), e((m, r))
        self.dA, self.dB, self.dx = e((r, cols), torch.float32), e((rows, r), torch.float32), e((m, cols))
        f = max(q.nf4_matmul_workspace_bytes(rows, cols, b, m) for b in (False, True))
        g = max(q.nf4_act_grad_workspace_bytes(m, rows), q.nf4_lora_grad_workspace_bytes(m, rows, r),
                q.nf4_lora_grad_workspace_bytes(m, cols, r))
        self.ws = workspace(max(f, g, 256))

    def step(self):
        W, a = self.W, act_id(self.act)
        q.nf4_lora_project(self.x, self.A, self.h, scale=self.s, p=self.p, rng=self.rng)
        q.nf4_linear(W.layer, W.rows, W.cols, W.f, self.x, self.out, self.ws, lora=(self.h, self.B), bias=self.bias,
                     act=a, preact=self.z, residual=self.res)
        q.nf4_act_grad(self.dy, self.z, a, self.dz, dbias=self.db, ws=self.ws)
        q.nf4_lora_project(self.dz, self.B, self.dh, scale=self.s, backward=True)
        q.nf4_lora_grad(self.h, self.dz, self.dB, self.ws, side="B")
        q.nf4_lora_grad(self.dh, self.x, self.dA, self.ws, side="A", p=self.p, rng=self.rng)
        q.nf4_linear(W.layer, W.rows, W.cols, W.f, self.dz, self.dx, self.ws, backward=True, lora=(self.dh, self.A),
                     p=self.p, rng=self.rng, residual=self.dxin)

    def outputs(self):
        return [t.clone() for t in (self.h, self.out, self.z, self.dz, self.db, self.dh, self.dA, self.dB, self.dx)]


def formula(W, x, A, B, bias, res, dy, mask, s, act):
    """The layer's loss sum(dy out) and its gradients in 64 bits."""
    h = s * (x * mask) @ A.t()
    z = x @ W.t() + h @ B.t() + bias
    out = ref.act(z, act) + res
    dz = dy * ref.slope(z, act)
    dh = s * dz @ B
    return dict(out=out, loss=(dy * out).sum(), bias=dz.sum(0), B=dz.t() @ h, A=dh.t() @ (x * mask),
                x=dz @ W + (dh @ A) * mask, h=h, z=z, dz=dz, dh=dh)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_formula_gradients_are_the_differences(act):
    """The 64-bit gradients against central differences of the 64-bit loss (step 1e-4 along random directions:
    third-order remainder about 1e-8 of the gradient's scale, cancellation 1e-16 loss / 1e-4)."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    m, rows, cols, r, s, p = 7, 12, 16, 3, 1.5, 0.3
    a = dict(x=n(m, cols), A=n(r, cols), B=n(rows, r), bias=n(rows))
    rest = dict(W=n(rows, cols) * 0.3, res=n(m, rows), dy=n(m, rows), mask=ref.mask((m, cols), p, 1, 2), s=s, act=act)
    grads = formula(**a, **rest)
    for k, v in a.items():
        d = n(*v.shape)
        up, dn = (formula(**dict(a, **{k: v + e * d}), **rest)["loss"] for e in (1e-4, -1e-4))
        got, want = (grads[k] * d).sum().item(), ((up - dn) / 2e-4).item()
        scale = (grads[k].abs() * d.abs()).sum().item()
        assert abs(got - want) <= 1e-6 * scale, (k, got, want)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,cols,m,r,act,p", [(256, 384, 50, 16, "silu", 0.1), (384, 256, 300, 8, "gelu", 0.0),
                                                 (1280, 640, 700, 64, "gelu_tanh", 0.2)])
def test_layer_forward_and_backward(dtype, rows, cols, m, r, act, p):
    """The whole run against the 64-bit formulas; the bounds follow each 16-bit intermediate (half a step) and each
    fp32 sum (2 K half steps of the magnitudes, K the terms) through what is computed from it."""
    print_case("adapted layer", dtype, rows, cols, m, r, act, p)
    L = Layer(rows, cols, m, r, dtype, act, p, 2.0, seed=rows + m)
    L.step()
    u = U16[dtype] * 1.02
    d = lambda t: t.double()
    W, x, A, B = L.W.dense(), d(L.x), d(L.A), d(L.B)
    k = ref.mask((m, cols), p, SEED, OFFSET).cuda()
    f = formula(W, x, A, B, d(L.bias), d(L.res), d(L.dy), k, 2.0, act)
    acc = lambda a, b, terms: 2 * (terms + 24) * U32 * (a.abs() @ b.abs())
    tiny = TINY[dtype]
    eh = u * f["h"].abs() + 2 * acc(x * k, A.t(), cols) + tiny
    ez = acc(x, W.t(), cols) + acc(f["h"], B.t(), r) + eh @ B.abs().t() + 4 * U32 * f["z"].abs()
    ezp = ez + u * f["z"].abs() + tiny
    eo = ref.LIPSCHITZ[act] * ez + ref.act_err(f["z"]) + u * f["out"].abs() + tiny
    edz32 = d(L.dy).abs() * (ref.CURVE[act] * ezp + 64 * U32 * (1 + f["z"].abs().clamp(max=20)))
    edz = edz32 + u * f["dz"].abs() + tiny
    edh = 2 * (edz @ B.abs() + acc(f["dz"], B, rows)) + u * f["dh"].abs() + tiny
    edB = edz.t() @ (f["h"].abs() + eh) + f["dz"].abs().t() @ eh + acc(f["dz"].t(), f["h"], m)
    edA = edh.t() @ (x * k).abs() + acc(f["dh"].t(), x * k, m)
    dx = f["x"] + d(L.dxin)
    edx = edz @ W.abs() + acc(f["dz"], W, rows) + k * (edh @ A.abs() + acc(f["dh"], A, r)) + u * dx.abs() \
        + 4 * U32 * d(L.dxin).abs() + tiny
    for name, got, want, tol in (("h", L.h, f["h"], eh), ("preact", L.z, f["z"], ezp), ("out", L.out, f["out"], eo),
                                 ("dz", L.dz, f["dz"], edz), ("dh", L.dh, f["dh"], edh), ("dA", L.dA, f["A"], edA),
                                 ("dB", L.dB, f["B"], edB), ("dx", L.dx, dx, edx),
                                 ("dbias", L.db, f["bias"], edz32.sum(0) + 2 * (m + 8) * U32 * f["dz"].abs().sum(0))):
        check(got, want.cpu(), tol.cpu(), name)


@pytest.mark.parametrize("m", [20, 700])
def test_layer_captured_into_a_graph(m):
    """The run captured once and replayed with new inputs and new seeds, eager runs of another layer between the
    replays: every replay has the eager run's bits."""
    mk = lambda seed: Layer(1280, 640, m, 16, torch.bfloat16, "silu", 0.1, 2.0, seed=seed)
    cap, eager, other = mk(1), mk(1), mk(2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        cap.step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap.step()
    for i in range(3):
        new = draw((m, 640), torch.bfloat16, 50 + i).cuda()
        state = rng(77 + i, i)
        for L in (cap, eager):
            L.x.copy_(new)
            L.rng.copy_(state)
        g.replay()
        other.step()
        eager.step()
        torch.cuda.synchronize()
        for a, b in zip(cap.outputs(), eager.outputs()):
            assert torch.equal(a, b), i


def test_layers_on_two_streams_at_once():
    """Two layers with their own workspaces, on two streams at once, twenty times: each has its own bits."""
    Ls = [Layer(1280, 640, 300, 16, torch.bfloat16, "silu", 0.1, 2.0, seed=s) for s in (1, 2)]
    want = []
    for L in Ls:
        L.step()
        want.append(L.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ls]
    for _ in range(20):
        for L, s in zip(Ls, streams):
            with torch.cuda.stream(s):
                L.step()
    torch.cuda.synchronize()
    for L, w in zip(Ls, want):
        for a, b in zip(L.outputs(), w):
            assert torch.equal(a, b)


def test_stream_argument_orders_the_work():
    """A call on an explicit stream sees what that stream wrote before it."""
    s = torch.cuda.Stream()
    x = torch.zeros(1 << 22, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            x += 1
    q.nf4_dropout(x, out, 0.5, rng(), stream=s)
    torch.cuda.synchronize()
    k = torch.from_numpy(ref.keep(np.arange(1000), 0.5, SEED, OFFSET))
    assert torch.equal(out[:1000].cpu().float(), k.float() * 40)

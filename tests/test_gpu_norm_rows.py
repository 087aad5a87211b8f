"""The layer norm and its gradient where a workgroup takes several rows one after
another, and the column sums of rows past the registers, against the 64-bit forms
(mx4_ref.py) on the device.

Tolerances as in test_gpu_norm.py.
"""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import quantized_lora_fine_nf4_amd as q
from conftest import print_case
from mx4_ref import TINY, U16, U32

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16

# Forward up to 2,048 workgroups of four rows (n <= 2048) or one: more rows than that in one round, a ragged last
# round, and five rounds; 64, 256 and 1,024 threads a row, one piece a thread and as many as it may have.
FORWARD = [(8197, 520), (8193, 2048), (34000, 72), (4099, 2056), (2049, 8192), (9000, 2312), (4100, 5120),
           (2053, 8200), (2051, 24576), (4500, 16392)]
# The gradient: more rows than one round of its workgroups, at 64, 256 and 512 threads a row.
GRADIENT = [(150, 8200), (131, 16384), (1100, 10248), (4500, 1536), (3000, 264), (1300, 4104), (1031, 8192)]
# Rows past the registers: the column sums in few blocks of rows, in a ragged last one and in all 64 of them.
LONG = [(17, 16392), (40, 16392), (1100, 16392), (1025, 24584), (333, 40000)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def draw(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def guarded(shape, dtype, pad=64):
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape)


def untouched(buf, pad=64):
    return bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[-pad:]).all())


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None


def within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    excess = ((got - want).abs() / tol).max().item()
    assert excess <= 1.0, (what, excess)


def check_norm(x, w, b, eps, residual, out, stats, total):
    """Every row of a call's results; row blocks, so that the 64-bit forms stay small."""
    for i in range(0, x.shape[0], 4096):
        s = slice(i, i + 4096)
        h = x[s]
        if residual is not None:
            h = (x[s].float() + residual[s].float()).to(x.dtype)
            assert torch.equal(total[s], h)
        y, mean, var, rstd = ref.layer_norm(h, w, b, eps)
        d = (h.double() - mean).abs()
        em = 40 * U32 * h.double().abs().mean(1, keepdim=True)
        rel = 25 * U32 + em * em / (2 * (var + eps))
        within(stats[s, :1], mean, em + U32 * mean.abs() + 1e-45, ("mean", i))
        within(stats[s, 1:], rstd, rstd * rel, ("rstd", i))
        ww = w.double().abs()
        tol = ww * rstd * (em + 3 * U32 * d) + ww * rstd * d * rel + 4 * U32 * (ww * rstd * d + b.double().abs())
        within(out[s], y, tol * (1 + U16[x.dtype]) + U16[x.dtype] * y.abs() + TINY[x.dtype], ("out", i))


@pytest.mark.parametrize("m,n", FORWARD)
def test_layer_norm_of_several_rounds(m, n):
    """Into buffers of their own and in place: the rows that are fetched ahead are other ones than those written."""
    for dtype in (BF16, FP16):
        # another mean and deviation in each row: one that takes a neighbour's shows
        x = draw((m, n), torch.float32, m + n)
        x = (x * torch.linspace(0.5, 4.0, m, device="cuda")[:, None] + torch.linspace(-3, 3, m, device="cuda")[:, None]).to(dtype)
        w, b = draw((n,), dtype, 1, 0.5, 1.0), draw((n,), dtype, 2, 0.3)
        for residual in (None, draw((m, n), dtype, 3, 1.5)):
            print_case("nf4_layer_norm rounds", dtype, m, n, residual is not None)
            ob, out = guarded((m, n), dtype)
            sb, stats = guarded((m, 2), torch.float32)
            tb, total = guarded((m, n), dtype) if residual is not None else (None, None)
            q.nf4_layer_norm(x, w, b, out, stats, 1e-5, residual=residual, total=total)
            check_norm(x, w, b, 1e-5, residual, out, stats, total)
            assert untouched(ob) and untouched(sb) and (tb is None or untouched(tb))
            if residual is None:
                y, st = x.clone(), torch.empty_like(stats)
                q.nf4_layer_norm(y, w, b, y, st, 1e-5)
                assert torch.equal(y, out) and torch.equal(st, stats)
                continue
            for swap in (False, True):
                a, r, st = x.clone(), residual.clone(), torch.empty_like(stats)
                o, t = (r, a) if swap else (a, r)
                q.nf4_layer_norm(a, w, b, o, st, 1e-5, residual=r, total=t)
                assert torch.equal(o, out) and torch.equal(t, total) and torch.equal(st, stats), swap


def check_grad(dy, x, w, stats, residual, dx, dw, db, dtype):
    m = x.shape[0]
    sums = torch.zeros(4, x.shape[1], dtype=torch.float64, device="cuda")   # dweight, dbias and their magnitudes
    for i in range(0, m, 4096):
        s = slice(i, i + 4096)
        mean, rstd = stats[s, :1].double(), stats[s, 1:].double()
        wdx, wdw, wdb = ref.layer_norm_grad(dy[s], x[s], w, mean, rstd)
        c = ((x[s].double() - mean) * rstd).abs()
        sums += torch.stack([wdw, wdb, (dy[s].double().abs() * c).sum(0), dy[s].double().abs().sum(0)])
        t = (dy[s].double() * w.double()).abs()
        tol = rstd * 48 * U32 * (t + t.mean(1, keepdim=True) + c * (t * c).mean(1, keepdim=True))
        if residual is not None:
            wdx = wdx + residual[s].double()
            tol = tol + 2 * U32 * (wdx.abs() + residual[s].double().abs())
        within(dx[s], wdx, tol * (1 + U16[dtype]) + U16[dtype] * wdx.abs() + TINY[dtype], ("dx", i))
    within(dw, sums[0], (m + 8) * U32 * sums[2] + 1e-45, "dweight")
    within(db, sums[1], (m + 8) * U32 * sums[3] + 1e-45, "dbias")


def stats_of(x, eps=1e-5):
    out = torch.empty(x.shape[0], 2, device="cuda")
    for i in range(0, x.shape[0], 4096):
        _, mean, _, rstd = ref.layer_norm(x[i:i + 4096], torch.ones(1, device="cuda"), torch.zeros(1, device="cuda"), eps)
        out[i:i + 4096] = torch.cat([mean, rstd], 1).float()
    return out


@pytest.mark.parametrize("m,n", GRADIENT + LONG)
def test_layer_norm_grad_of_several_rounds(m, n):
    space = lambda: workspace(q.nf4_layer_norm_grad_workspace_bytes(m, n))
    for dtype in (BF16, FP16):
        x = draw((m, n), torch.float32, m + n)
        x = (x * torch.linspace(0.5, 4.0, m, device="cuda")[:, None] + torch.linspace(-3, 3, m, device="cuda")[:, None]).to(dtype)
        w, dy = draw((n,), dtype, 1, 0.5, 1.0), draw((m, n), dtype, 7, 0.3, 0.1)
        stats = stats_of(x)
        for residual in (None, draw((m, n), dtype, 3, 0.5)):
            print_case("nf4_layer_norm_grad rounds", dtype, m, n, residual is not None)
            xb, dx = guarded((m, n), dtype)
            wb, dw = guarded((n,), torch.float32)
            bb, db = guarded((n,), torch.float32)
            q.nf4_layer_norm_grad(dy, x, w, stats, dx, dw, db, space(), residual=residual)
            check_grad(dy, x, w, stats, residual, dx, dw, db, dtype)
            assert untouched(xb) and untouched(wb) and untouched(bb)
        # dx in the place of each input in turn
        for alias in range(3):
            a = [dy.clone(), x.clone(), residual.clone()]
            dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
            q.nf4_layer_norm_grad(a[0], a[1], w, stats, a[alias], dw2, db2, space(), residual=a[2])
            assert torch.equal(a[alias], dx) and torch.equal(dw2, dw) and torch.equal(db2, db), alias


def test_column_sums_of_more_long_rows_than_a_grid():
    """Both column sums where the rows past the registers are more than a grid has workgroups."""
    m, n = 65536 + 5, 16392
    print_case("nf4_layer_norm_grad", m, n)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(m, n, dtype=BF16, device="cuda").normal_(generator=g)
    dy = torch.empty_like(x).normal_(generator=g)
    weight = torch.randn(n, generator=g, device="cuda").to(x.dtype)
    stats = torch.empty(m, 2, device="cuda")
    stats[:, 0] = torch.randn(m, generator=g, device="cuda")
    stats[:, 1] = torch.rand(m, generator=g, device="cuda") + 0.5
    dw, db, dx = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x)
    q.nf4_layer_norm_grad(dy, x, weight, stats, dx, dw, db, workspace(q.nf4_layer_norm_grad_workspace_bytes(m, n)))
    check_grad(dy, x, weight, stats, None, dx, dw, db, BF16)


@pytest.mark.parametrize("n", [64, 520, 5120, 8200, 24584])
def test_a_variance_past_fp32(n):
    """Differences of 2^70, whose squares fp32 does not hold: rstd is 0, out the bias, and the gradient what comes past
    the norm; the tokens beside it are as without it."""
    print_case("nf4_layer_norm, variance past fp32", n)
    m = 5
    x, w, b = draw((m, n), BF16, n), draw((n,), BF16, 1), draw((n,), BF16, 2)
    out, stats = torch.empty_like(x), torch.empty(m, 2, device="cuda")
    q.nf4_layer_norm(x, w, b, out, stats)
    big = x.clone()
    big[2] = 2.0 ** 70 * (1 - 2 * (torch.arange(n, device="cuda") % 2))   # mean 0
    got, st = torch.empty_like(x), torch.empty(m, 2, device="cuda")
    q.nf4_layer_norm(big, w, b, got, st)
    assert st[2].tolist() == [0, 0] and torch.equal(got[2], b)
    keep = torch.arange(m, device="cuda") != 2
    assert torch.equal(got[keep], out[keep]) and torch.equal(st[keep], stats[keep])
    dy, r = draw((m, n), BF16, 3), draw((m, n), BF16, 4)
    dx, dw, db = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    q.nf4_layer_norm_grad(dy, big, w, st, dx, dw, db, workspace(q.nf4_layer_norm_grad_workspace_bytes(m, n)), residual=r)
    assert torch.equal(dx[2], r[2]) and torch.isfinite(dw).all()

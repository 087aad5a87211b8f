"""The layer norm and its gradient against their 64-bit forms (mx4_ref.py), and
one training step of a norm, a product in four bits and their gradients.

Tolerances, elementwise, u = 2^-24.  A row's sum passes at most 40 fp32 additions
(pieces of a lane, lanes, waves): 40 u of the magnitudes' sum.  So the mean is off
by em = 40 u mean|h|; the sum of (h - mean)^2 by em^2 (the differences' own sum is
0) and 44 u of itself; rstd by half of that relative, and 3 u; the factors and the
sum of out add 4 u of their magnitudes, its rounding half a step.
"""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import quantized_lora_fine_nf4_amd as q
from conftest import print_case
from mx4_ref import TINY, U16, U32

pytestmark = pytest.mark.gpu
DT = [torch.bfloat16, torch.float16]
IDS = ["bf16", "fp16"]
SHAPES = [(1, 8), (1, 5120), (2, 16), (3, 504), (4, 512), (5, 520), (17, 1024), (7, 1544), (33, 2048), (9, 2056),
          (300, 64), (17, 5120), (5, 4096), (6, 6152), (3, 8192), (4, 8200), (3, 16384), (2, 16392), (3, 24576),
          (2, 24584), (3, 40000), (1027, 2048), (777, 5120), (2100, 264)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()


def draw(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def guarded(shape, dtype, pad=64):
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape)


def untouched(buf, shape, pad=64):
    n = int(np.prod(shape))
    return bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[pad + n:]).all())


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None


def within(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    excess = ((got - want).abs() / tol).max().item()
    assert excess <= 1.0, (what, excess)


def run_norm(x, w, b, eps, residual=None):
    m, n = x.shape
    ob, out = guarded((m, n), x.dtype)
    sb, stats = guarded((m, 2), torch.float32)
    tb, total = guarded((m, n), x.dtype) if residual is not None else (None, None)
    q.nf4_layer_norm(x.cuda(), w.cuda(), b.cuda(), out, stats, eps,
                     residual=None if residual is None else residual.cuda(), total=total)
    torch.cuda.synchronize()
    assert untouched(ob, out.shape) and untouched(sb, stats.shape)
    assert total is None or untouched(tb, total.shape)
    return out, stats, total


def check_norm(x, w, b, eps, residual=None):
    out, stats, total = run_norm(x, w, b, eps, residual)
    h = x
    if residual is not None:
        h = (x.float() + residual.float()).to(x.dtype)
        assert torch.equal(total.cpu(), h)
    y, mean, var, rstd = ref.layer_norm(h, w, b, eps)
    d = (h.double() - mean).abs()
    em = 40 * U32 * h.double().abs().mean(1, keepdim=True)
    rel = 25 * U32 + em * em / (2 * (var + eps))
    within(stats[:, :1], mean, em + U32 * mean.abs() + 1e-45, "mean")
    within(stats[:, 1:], rstd, rstd * rel, "rstd")
    ww = w.double().abs()
    tol = ww * rstd * (em + 3 * U32 * d) + ww * rstd * d * rel + 4 * U32 * (ww * rstd * d + b.double().abs())
    within(out, y, tol * (1 + U16[x.dtype]) + U16[x.dtype] * y.abs() + TINY[x.dtype], "out")
    return out, stats, total


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("m,n", SHAPES)
def test_layer_norm(dtype, m, n):
    x, w, b = draw((m, n), dtype, m + n, 2.0, 0.7), draw((n,), dtype, 1, 0.5, 1.0), draw((n,), dtype, 2, 0.3)
    for residual in (None, draw((m, n), dtype, 3, 1.5)):
        print_case("nf4_layer_norm", dtype, m, n, residual is not None)
        check_norm(x, w, b, 1e-5, residual)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_layer_norm_hard_rows(dtype):
    """A mean far above the deviation, equal values, one large value, zeros."""
    print_case("nf4_layer_norm hard rows", dtype)
    n = 2056
    x = draw((6, n), dtype, 4)
    x[0] = (x[0].float() * 0.5 + 64.0).to(dtype)
    x[1] = 3.0
    x[2] = 0.0
    x[3, 17] = 3000.0
    x[4] = x[4] * 2 ** -10
    w, b = draw((n,), dtype, 5), draw((n,), dtype, 6)
    for eps in (1e-5, 1e-3):
        check_norm(x, w, b, eps)


def test_layer_norm_keeps_what_is_not_finite_in_its_row():
    print_case("nf4_layer_norm not finite")
    for n in (72, 520, 2056, 8200, 24584):
        x, w, b = draw((5, n), torch.bfloat16, n), draw((n,), torch.bfloat16, 1), draw((n,), torch.bfloat16, 2)
        good = run_norm(x, w, b, 1e-5)[0].cpu()
        x[1, n - 1], x[3, 0] = float("nan"), float("inf")
        out = run_norm(x, w, b, 1e-5)[0].cpu()
        assert torch.isnan(out[[1, 3]]).all()
        assert torch.equal(out[[0, 2, 4]], good[[0, 2, 4]])


def test_layer_norm_in_place():
    print_case("nf4_layer_norm in place")
    for n in (136, 5120, 24584):
        x, r, w, b = (draw(s, torch.bfloat16, i) for i, s in enumerate([(37, n), (37, n), (n,), (n,)]))
        want, wstats, wtotal = run_norm(x, w, b, 1e-5, r)
        xd, rd, stats = x.cuda(), r.cuda(), torch.empty(37, 2, device="cuda")
        q.nf4_layer_norm(xd, w.cuda(), b.cuda(), xd, stats, 1e-5, residual=rd, total=rd)
        assert torch.equal(xd, want) and torch.equal(rd, wtotal) and torch.equal(stats, wstats)
        xd = x.cuda()
        q.nf4_layer_norm(xd, w.cuda(), b.cuda(), xd, stats, 1e-5)
        assert torch.equal(xd, run_norm(x, w, b, 1e-5)[0])


# ---- gradient --------------------------------------------------------------

def run_grad(dy, x, w, stats, residual=None):
    m, n = x.shape
    xb, dx = guarded((m, n), x.dtype)
    wb, dw = guarded((n,), torch.float32)
    bb, db = guarded((n,), torch.float32)
    q.nf4_layer_norm_grad(dy.cuda(), x.cuda(), w.cuda(), stats.cuda(), dx, dw, db,
                          workspace(q.nf4_layer_norm_grad_workspace_bytes(m, n)),
                          residual=None if residual is None else residual.cuda())
    torch.cuda.synchronize()
    assert untouched(xb, dx.shape) and untouched(wb, dw.shape) and untouched(bb, db.shape)
    return dx, dw, db


def check_grad(dy, x, w, stats, residual=None):
    """Given stats, c is off by 2 u of itself, dy weight by u; the two row sums by 48 u of their magnitudes; the
    last sum and product by 4 u.  A column's sum over m tokens: m + 8 additions and factors."""
    dx, dw, db = run_grad(dy, x, w, stats, residual)
    mean, rstd = stats[:, :1].double(), stats[:, 1:].double()
    wdx, wdw, wdb = ref.layer_norm_grad(dy, x, w, mean, rstd)
    c = ((x.double() - mean) * rstd).abs()
    t = (dy.double() * w.double()).abs()
    mt, mtc = t.mean(1, keepdim=True), (t * c).mean(1, keepdim=True)
    tol = rstd * 48 * U32 * (t + mt + c * mtc)
    if residual is not None:
        wdx = wdx + residual.double()
        tol = tol + 2 * U32 * (wdx.abs() + residual.double().abs())
    within(dx, wdx, tol * (1 + U16[x.dtype]) + U16[x.dtype] * wdx.abs() + TINY[x.dtype], "dx")
    m = x.shape[0]
    within(dw, wdw, (m + 8) * U32 * (dy.double().abs() * c).sum(0) + 1e-45, "dweight")
    within(db, wdb, (m + 8) * U32 * dy.double().abs().sum(0) + 1e-45, "dbias")
    return dx, dw, db


def stats_of(x, eps=1e-5):
    _, mean, _, rstd = ref.layer_norm(x, torch.ones(1), torch.zeros(1), eps)
    return torch.cat([mean, rstd], 1).float()


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("m,n", SHAPES)
def test_layer_norm_grad(dtype, m, n):
    x, w = draw((m, n), dtype, m + n, 2.0, 0.7), draw((n,), dtype, 1, 0.5, 1.0)
    dy = draw((m, n), dtype, 7, 0.3, 0.1)
    for residual in (None, draw((m, n), dtype, 3, 0.5)):
        print_case("nf4_layer_norm_grad", dtype, m, n, residual is not None)
        check_grad(dy, x, w, stats_of(x), residual)


def test_layer_norm_grad_against_differences():
    """The kernel's dx, dweight and dbias of L = sum(dy out) against central differences of the 64-bit forward form.
    Their own error is h^2 / 6 of the third derivative (below 1e-6 here, h = 1e-3); the kernel's as above, under
    2^-11 of the largest gradient per element in fp16."""
    print_case("nf4_layer_norm_grad differences")
    m, n, h = 3, 24, 1e-3
    x, w, b = draw((m, n), torch.float16, 1, 1.5, 0.3), draw((n,), torch.float16, 2, 0.5, 1.0), draw((n,), torch.float16, 3)
    dy = draw((m, n), torch.float16, 4, 0.5)
    dx, dw, db = (t.double().cpu() for t in run_grad(dy, x, w, stats_of(x)))

    def loss(x, w, b):
        return (dy.double() * ref.layer_norm(x, w, b, 1e-5)[0]).sum().item()

    args = [x.double(), w.double(), b.double()]
    for i, got in enumerate((dx, dw, db)):
        for k in range(got.numel()):
            side = []
            for sign in (1, -1):
                moved = [a.clone() for a in args]
                moved[i].view(-1)[k] += sign * h
                side.append(loss(*moved))
            want = (side[0] - side[1]) / (2 * h)
            assert abs(got.view(-1)[k].item() - want) <= 2.0 ** -11 * got.abs().max().item() + 2e-6, (i, k)


def test_layer_norm_grad_not_finite():
    """A NaN of dy reaches dx of its token and the sums of its column; dx may be dy, x or residual."""
    print_case("nf4_layer_norm_grad not finite, in place")
    for n in (72, 2056, 5120, 16392):
        m = 19
        x, dy, r, w = (draw(s, torch.bfloat16, i) for i, s in enumerate([(m, n), (m, n), (m, n), (n,)]))
        st = stats_of(x)
        good = run_grad(dy, x, w, st, r)
        bad = dy.clone()
        bad[4, 8] = float("nan")
        dx, dw, db = run_grad(bad, x, w, st, r)
        keep = torch.arange(m) != 4
        cols = torch.arange(n) != 8
        assert torch.isnan(dx[4]).all() and torch.equal(dx[keep.cuda()], good[0][keep.cuda()])
        assert torch.isnan(dw[8]) and torch.isnan(db[8])
        assert torch.equal(dw[cols.cuda()], good[1][cols.cuda()]) and torch.equal(db[cols.cuda()], good[2][cols.cuda()])
        for alias in range(3):
            a = [dy.cuda(), x.cuda(), r.cuda()]
            dw2, db2 = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
            q.nf4_layer_norm_grad(a[0], a[1], w.cuda(), st.cuda(), a[alias], dw2, db2,
                                  workspace(q.nf4_layer_norm_grad_workspace_bytes(m, n)), residual=a[2])
            assert torch.equal(a[alias], good[0]) and torch.equal(dw2, good[1]) and torch.equal(db2, good[2])


# ---- together --------------------------------------------------------------

def step_buffers(m, n, rows):
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")
    f32, u8 = torch.float32, torch.uint8
    return {"y": e(m, n), "total": e(m, n), "stats": e(m, 2, dtype=f32), "xc": e(m, n // 2, dtype=u8),
            "xs": e(m, n // 32, dtype=u8), "out": e(m, rows), "dh": e(m, n), "dx": e(m, n), "dw": e(n, dtype=f32),
            "db": e(n, dtype=f32), "ws4": workspace(q.mx4_matmul4_workspace_bytes(rows, n, m)),
            "wsb": workspace(q.mx4_matmul_workspace_bytes(rows, n, True, m)),
            "wsn": workspace(q.nf4_layer_norm_grad_workspace_bytes(m, n))}


def step(s, x, r, w, b, codes, scales, dout):
    """One block's front: norm, activations to four bits, product; then the gradients back to the residual
    sum (any [m, n] tensor stands for the gradient past the norm)."""
    q.nf4_layer_norm(x, w, b, s["y"], s["stats"], 1e-5, residual=r, total=s["total"])
    q.mx4_quantize(s["y"], s["xc"], s["xs"])
    q.mx4_matmul4(codes, scales, s["xc"], s["xs"], s["out"], s["ws4"])
    q.mx4_matmul(codes, scales, dout, s["dh"], s["wsb"], backward=True)
    q.nf4_layer_norm_grad(s["dh"], s["total"], w, s["stats"], s["dx"], s["dw"], s["db"], s["wsn"], residual=s["total"])



@pytest.mark.parametrize("m,n,rows", [(5, 256, 512), (77, 2080, 1032), (300, 512, 768)])
def test_a_step_of_all_of_them(m, n, rows):
    """Each stage against the 64-bit form of its own inputs; the weight quantised here and scored by its error."""
    print_case("step", m, n, rows)
    wm = draw((rows, n), torch.bfloat16, 1, 0.02)
    codes, scales = torch.empty(rows, n // 2, dtype=torch.uint8, device="cuda"), torch.empty(rows, n // 32, dtype=torch.uint8, device="cuda")
    err = torch.empty(1, dtype=torch.float64, device="cuda")
    q.mx4_quantize(wm.cuda(), codes, scales, err, workspace(q.mx4_quantize_workspace_bytes(rows, n)))
    wc, wsc = ref.quantize(wm)
    assert torch.equal(codes.cpu(), wc) and torch.equal(scales.cpu(), wsc)
    x, r, w, b = (draw(sh, torch.bfloat16, i) for i, sh in enumerate([(m, n), (m, n), (n,), (n,)]))
    dout = draw((m, rows), torch.bfloat16, 9, 0.1)
    s = step_buffers(m, n, rows)
    step(s, x.cuda(), r.cuda(), w.cuda(), b.cuda(), codes, scales, dout.cuda())
    torch.cuda.synchronize()
    out, stats, total = check_norm(x, w, b, 1e-5, r)
    assert torch.equal(s["y"], out) and torch.equal(s["total"], total)
    c, sc = ref.quantize(s["y"].cpu())
    assert torch.equal(s["xc"].cpu(), c) and torch.equal(s["xs"].cpu(), sc)
    wv, xv = ref.values(wc, wsc), ref.values(c, sc)
    want = xv @ wv.t().contiguous()
    within(s["out"], want, 2 * n * U32 * (xv.abs() @ wv.abs().t().contiguous()) + U16[torch.bfloat16] * want.abs(), "out")
    want = dout.double() @ wv
    within(s["dh"], want, 2 * rows * U32 * (dout.double().abs() @ wv.abs()) + U16[torch.bfloat16] * want.abs() + 1e-30, "dh")
    dx, dw, db = check_grad(s["dh"].cpu(), total.cpu(), w, stats.cpu(), total.cpu())
    assert torch.equal(s["dx"], dx) and torch.equal(s["dw"], dw) and torch.equal(s["db"], db)


def test_the_error_ranks_layers():
    """mx4_quantize's errors go into the selection as they are: the worst matrices stay in 16 bits."""
    print_case("mx4 errors into aqlora_select_topk")
    mats = [draw((64, 256), torch.bfloat16, i, 0.01 * (1 + (5 * i) % 7)) for i in range(6)]
    err = torch.empty(6, dtype=torch.float64, device="cuda")
    codes, scales = torch.empty(64, 128, dtype=torch.uint8, device="cuda"), torch.empty(64, 8, dtype=torch.uint8, device="cuda")
    for i, wm in enumerate(mats):
        q.mx4_quantize(wm.cuda(), codes, scales, err[i:i + 1], workspace(q.mx4_quantize_workspace_bytes(64, 256)))
    cost = torch.full((6,), 2 * 64 * 256 - q.mx4_storage_bytes(64, 256), dtype=torch.int64, device="cuda")
    sel, k = torch.empty(6, dtype=torch.uint8, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    q.aqlora_select_topk(err, cost, int(cost[0]) * 2, -1, sel, k, workspace(q.aqlora_workspace_bytes(6)))
    want = [(m.double() - ref.values(*ref.quantize(m))).square().sum().item() for m in mats]
    top = sorted(range(6), key=lambda i: -want[i])[:2]
    assert k.item() == 2 and sorted(torch.nonzero(sel).flatten().tolist()) == sorted(top)


def test_captured_and_on_another_stream():
    """The whole step in a graph, replayed with new inputs and eager work in between, and on a side stream: the same
    bits as eager calls."""
    print_case("graph and stream")
    m, n, rows = 70, 512, 1024
    wm = draw((rows, n), torch.bfloat16, 1, 0.02).cuda()
    codes, scales = torch.empty(rows, n // 2, dtype=torch.uint8, device="cuda"), torch.empty(rows, n // 32, dtype=torch.uint8, device="cuda")
    q.mx4_quantize(wm, codes, scales)
    ins = [[draw(sh, torch.bfloat16, 10 * k + i).cuda() for i, sh in enumerate([(m, n), (m, n), (n,), (n,)])] +
           [draw((m, rows), torch.bfloat16, 10 * k + 9, 0.1).cuda()] for k in range(4)]
    names = ("y", "total", "stats", "out", "dh", "dx", "dw", "db")
    want = []
    for v in ins:
        s = step_buffers(m, n, rows)
        step(s, *v[:4], codes, scales, v[4])
        want.append([s[k].clone() for k in names])
    hold = [t.clone() for t in ins[0]]
    s = step_buffers(m, n, rows)
    step(s, *hold[:4], codes, scales, hold[4])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, *hold[:4], codes, scales, hold[4])
    for k in (1, 2, 3, 0, 2):
        for t, v in zip(hold, ins[k]):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s[name], w) for name, w in zip(names, want[k])), k
        step(step_buffers(m, n, rows), *ins[0][:4], codes, scales, ins[0][4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = step_buffers(m, n, rows)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(s, *ins[3][:4], codes, scales, ins[3][4])
    side.synchronize()
    assert all(torch.equal(s[name], w) for name, w in zip(names, want[3]))


def test_long_rows_more_than_a_grid():
    """More rows past the registers than workgroups: the same bits as those rows alone."""
    m, n = 65536 + 5, 24584
    print_case("nf4_layer_norm, nf4_layer_norm_grad", m, n)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(m, n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy = torch.empty_like(x).normal_(generator=g)
    weight, bias = (torch.randn(n, generator=g, device="cuda").to(x.dtype) for _ in range(2))
    out, stats = torch.empty_like(x), torch.empty(m, 2, device="cuda")
    q.nf4_layer_norm(x, weight, bias, out, stats)
    dw, db = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dx = torch.empty_like(x)
    space = torch.empty(q.nf4_layer_norm_grad_workspace_bytes(m, n), dtype=torch.uint8, device="cuda")
    q.nf4_layer_norm_grad(dy, x, weight, stats, dx, dw, db, space)
    k = 7
    out2, stats2, dx2 = torch.empty(k, n, dtype=x.dtype, device="cuda"), torch.empty(k, 2, device="cuda"), torch.empty(k, n, dtype=x.dtype, device="cuda")
    q.nf4_layer_norm(x[-k:].contiguous(), weight, bias, out2, stats2)
    space = torch.empty(q.nf4_layer_norm_grad_workspace_bytes(k, n), dtype=torch.uint8, device="cuda")
    q.nf4_layer_norm_grad(dy[-k:].contiguous(), x[-k:].contiguous(), weight, stats2, dx2, torch.empty_like(dw), torch.empty_like(db),
                          space if space.numel() else None)
    assert torch.equal(out[-k:], out2) and torch.equal(stats[-k:], stats2) and torch.equal(dx[-k:], dx2)
    # a sum of m terms in any order: within m u of the magnitudes' sum
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for i in range(0, m, 8192):
        want += dy[i:i + 8192].double().sum(0)
        size += dy[i:i + 8192].double().abs().sum(0)
    assert ((db.double() - want).abs() <= m * U32 * size).all()


# ---- plain calls, and those that are not ------------------------------------

def all_calls(dtype, m=5, n=256, rows=64, seed=0):
    """Each call with good arguments, by name: (function, arguments by name, what it writes)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    def e(*shape, t=dtype):
        return torch.zeros(*shape, dtype=t, device="cuda")

    def u8(nbytes):
        return e(nbytes, t=torch.uint8) if nbytes else None
    w = r(rows, n)
    c, s = e(rows, n // 2, t=torch.uint8), e(rows, n // 32, t=torch.uint8)
    q.mx4_quantize(w, c, s)
    x, dy = r(m, n), r(m, rows)
    xc, xs = e(m, n // 2, t=torch.uint8), e(m, n // 32, t=torch.uint8)
    q.mx4_quantize(x, xc, xs)
    stats = e(m, 2, t=torch.float32)
    q.nf4_layer_norm(x, r(n), r(n), e(m, n), stats)
    f32 = torch.float32
    return {
        "norm": (q.nf4_layer_norm, dict(x=x, weight=r(n), bias=r(n), out=e(m, n), stats=e(m, 2, t=f32), residual=r(m, n),
                                        total=e(m, n)), ("out", "stats", "total")),
        "norm grad": (q.nf4_layer_norm_grad, dict(dy=r(m, n), x=x, weight=r(n), stats=stats, dx=e(m, n), dweight=e(n, t=f32),
                                                  dbias=e(n, t=f32), residual=r(m, n),
                                                  ws=u8(q.nf4_layer_norm_grad_workspace_bytes(m, n))), ("dx", "dweight", "dbias")),
        "quantize": (q.mx4_quantize, dict(x=w, codes=e(*c.shape, t=torch.uint8), scales=e(*s.shape, t=torch.uint8),
                                          err=e(1, t=torch.float64), ws=u8(q.mx4_quantize_workspace_bytes(rows, n))),
                     ("codes", "scales", "err")),
        "dequantize": (q.mx4_dequantize, dict(codes=c, scales=s, out=e(rows, n)), ("out",)),
        "matmul": (q.mx4_matmul, dict(codes=c, scales=s, x=x, out=e(m, rows), ws=u8(q.mx4_matmul_workspace_bytes(rows, n, False, m))),
                   ("out",)),
        "matmul back": (q.mx4_matmul, dict(codes=c, scales=s, x=dy, out=e(m, n, t=f32), backward=True,
                                           ws=u8(q.mx4_matmul_workspace_bytes(rows, n, True, m))), ("out",)),
        "matmul4": (q.mx4_matmul4, dict(codes=c, scales=s, xcodes=xc, xscales=xs, out=e(m, rows),
                                        ws=u8(q.mx4_matmul4_workspace_bytes(rows, n, m))), ("out",)),
    }


CALLS = ("norm", "norm grad", "quantize", "dequantize", "matmul", "matmul back", "matmul4")


def test_plain_calls_are_made_by_the_compiled_module(monkeypatch):
    """With it and with Python's own checks the same bits, on the current stream and on a given one."""
    native = q._load_calls()
    assert native is not q._NoCalls, "the compiled module is missing"
    for dtype in DT:
        for name in CALLS:
            print_case("plain call", name, dtype)
            got = []
            for plain, stream in ((native, None), (q._NoCalls, None), (native, torch.cuda.Stream())):
                monkeypatch.setattr(q, "_plain", plain)
                fn, kw, outs = all_calls(dtype)[name]
                torch.cuda.synchronize()
                fn(**kw, stream=stream)
                torch.cuda.synchronize()
                got.append([kw[k].clone() for k in outs])
            for other in got[1:]:
                assert all(torch.equal(a, b) for a, b in zip(got[0], other)), name
            # what it takes as plain it makes: a status and not None
            monkeypatch.setattr(q, "_plain", native)
            if name == "dequantize":
                fn, kw, _ = all_calls(dtype)[name]
                assert native.dequantize(kw["codes"], kw["scales"], kw["out"], None) == q.NF4_OK


@pytest.mark.parametrize("name", CALLS)
def test_what_does_not_fit_is_refused(name):
    """Each tensor in turn: another shape, another type, on the CPU, every other element, an address off by one element.
    Nothing is written."""
    for key in all_calls(torch.bfloat16)[name][1]:
        for what in ("shape", "type", "cpu", "strides", "address"):
            fn, kw, outs = all_calls(torch.bfloat16)[name]
            t = kw[key]
            if not isinstance(t, torch.Tensor):
                continue
            if key == "ws" and what in ("shape", "type") or t.numel() < 2 and what == "strides":
                continue
            print_case("refused", name, key, what)
            if what == "shape":
                kw[key] = torch.cat([t, t])
            elif what == "type":
                kw[key] = t.to(torch.float64 if t.dtype != torch.float64 else torch.float32)
            elif what == "cpu":
                kw[key] = t.cpu()
            elif what == "strides":
                kw[key] = torch.cat([t.reshape(-1), t.reshape(-1)])[::2].view(t.shape) if t.dim() == 1 else t.t().contiguous().t()
            else:
                if key in ("scales", "xscales", "err", "stats"):
                    continue   # one element on is aligned as it has to be
                kw[key] = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
            if what == "strides" and kw[key].is_contiguous():
                continue
            for k in outs:
                kw[k].fill_(7)
            before = [kw[k].clone() for k in outs]
            with pytest.raises(q.NF4Error):
                fn(**kw)
            torch.cuda.synchronize()
            assert all(torch.equal(a, kw[k]) for a, k in zip(before, outs))

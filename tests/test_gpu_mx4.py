"""The microscaled 4-bit codec and its products against their 64-bit forms
(mx4_ref.py).

Codes, scales and values are compared bit for bit.  Products, elementwise: the
operands' products are exact in fp32 (a 4-bit value has 2 significant bits, a
16-bit one at most 11), a sum of K of them in any order and rounding is within
2 K 2^-24 of the sum of their magnitudes (the matrix core may round each addition
toward zero: one step instead of half of one), and a 16-bit result adds half a
step of it.
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


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def guarded(shape, dtype, pad=256, fill=None):
    n = int(np.prod(shape))
    fill = (0x5A if dtype == torch.uint8 else float("nan")) if fill is None else fill
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return buf, buf[pad:pad + n].view(shape)


def untouched(buf, shape, pad=256):
    n = int(np.prod(shape))
    edge = torch.cat([buf[:pad], buf[pad + n:]])
    return bool((edge == 0x5A).all()) if buf.dtype == torch.uint8 else bool(torch.isnan(edge).all())


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None


# ---- codec -----------------------------------------------------------------

def quantize(x, with_err=True):
    rows, cols = x.shape
    cb, codes = guarded((rows, cols // 2), torch.uint8)
    sb, scales = guarded((rows, cols // 32), torch.uint8)
    err = torch.full((1,), float("nan"), dtype=torch.float64, device="cuda") if with_err else None
    q.mx4_quantize(x.cuda(), codes, scales, err, workspace(q.mx4_quantize_workspace_bytes(rows, cols)) if with_err else None)
    torch.cuda.synchronize()
    assert untouched(cb, codes.shape) and untouched(sb, scales.shape)
    return codes.cpu(), scales.cpu(), None if err is None else err.item()


def check_codec(x):
    want_c, want_s = ref.quantize(x)
    for with_err in (False, True):
        c, s, err = quantize(x, with_err)
        assert torch.equal(s, want_s), "scales"
        known = (want_s != 255).repeat_interleave(16, 1)
        assert torch.equal(c[known], want_c[known]), "codes"
    if (want_s != 255).all():
        e = (x.double() - ref.values(want_c, want_s)).square().sum().item()
        assert abs(err - e) <= x.numel() * 2.0 ** -52 * e, (err, e)
    else:
        assert np.isnan(err)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (7, 1056), (17, 5120), (333, 2048), (2049, 4096)])
def test_quantize_is_the_definition(dtype, rows, cols):
    print_case("mx4_quantize", dtype, rows, cols)
    x = torch.randn(rows, cols, generator=gen(rows + cols)) * torch.exp2(torch.randn(rows, 1, generator=gen(1)) * 3)
    check_codec(x.to(dtype))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_quantize_every_value(dtype):
    """All finite 16-bit patterns, next to a largest one that gives them each of several scales."""
    print_case("mx4_quantize every value", dtype)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(dtype)
    bits = bits[torch.isfinite(bits)]
    order = bits[torch.randperm(bits.numel(), generator=gen(5))]
    check_codec(order[:order.numel() // 64 * 64].view(-1, 64))
    # sorted by magnitude: groups of nearly equal values, the largest one decides; subnormals and zeros among them
    by = bits[bits.double().abs().argsort(stable=True)]
    check_codec(by[:by.numel() // 32 * 32].view(-1, 32))
    # one fixed largest value per row
    top = torch.tensor([1.0, 1.9375, 4.0, 5.0, 0.0078125, 480.0], dtype=dtype)
    for t in top:
        small = bits[bits.double().abs() <= t.double()]
        small = torch.cat([small, small.new_zeros(-small.numel() % 31)]).view(-1, 31)
        check_codec(torch.cat([small, t.expand(small.shape[0], 1)], 1))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_quantize_zeros_and_values_that_are_not_finite(dtype):
    print_case("mx4_quantize edge values", dtype)
    x = torch.randn(8, 128, generator=gen(3)).to(dtype)
    x[1] = 0
    x[2, :32] = -0.0
    x[3, 33] = float("nan")
    x[4, 64] = float("inf")
    x[5, 127] = -float("inf")
    x[6, :64] = torch.finfo(dtype).max
    x[7, :32] = torch.finfo(dtype).smallest_normal / 4
    check_codec(x)
    c, s, _ = quantize(x)
    v = ref.values(c, s)
    for row, blk in ((3, 1), (4, 2), (5, 3)):
        assert torch.isnan(v[row, 32 * blk:32 * blk + 32]).all() and int(torch.isnan(v[row]).sum()) == 32


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_dequantize_every_code_and_scale(dtype):
    print_case("mx4_dequantize", dtype)
    codes = torch.arange(256, dtype=torch.uint8).view(1, 16, 16).expand(256, 16, 16).reshape(256, 256)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).expand(256, 16).contiguous()
    buf, out = guarded((256, 512), dtype)
    q.mx4_dequantize(codes.contiguous().cuda(), scales.cuda(), out)
    want = ref.values(codes, scales).float().to(dtype)
    got = out.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and int(nan.sum()) == 512
    assert torch.equal(got[~nan].view(torch.int16), want[~nan].view(torch.int16))
    assert untouched(buf, out.shape)


@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (129, 2080)])
def test_dequantize_shapes(rows, cols):
    print_case("mx4_dequantize", rows, cols)
    c, s = ref.random_matrix(rows, cols, gen(2), 0, 255)
    buf, out = guarded((rows, cols), torch.bfloat16)
    q.mx4_dequantize(c.cuda(), s.cuda(), out)
    assert torch.equal(out.cpu().view(torch.int16), ref.values(c, s).float().bfloat16().view(torch.int16))
    assert untouched(buf, out.shape)


# ---- products --------------------------------------------------------------

def product(a, b):
    return a @ b.t().contiguous()


def check_product(got, a, b, what):
    """got = a b^T, a and b fp64 operands as the kernel reads them."""
    want, scale, k = product(a, b), product(a.abs(), b.abs()), a.shape[1]
    tol = 2 * k * U32 * scale + U16[got.dtype] * want.abs() + TINY[got.dtype]
    excess = ((got.double().cpu() - want).abs() / tol).max().item()
    assert excess <= 1.0, (what, excess)


# Few and many tokens, rows and columns of whole tiles and not, reductions of one block up to split ones.
SHAPES = [(1, 8, 32), (1, 64, 64), (1, 4096, 2048), (2, 40, 96), (5, 136, 160), (16, 128, 128), (17, 264, 1056),
          (31, 1000, 512), (33, 512, 2080), (64, 256, 4096), (65, 328, 544), (127, 1024, 256), (128, 128, 8192),
          (129, 248, 288), (255, 2048, 320), (256, 256, 256), (257, 264, 2048), (333, 1160, 1120), (512, 512, 1024),
          (1000, 776, 96), (2048, 520, 160)]


def make_product(m, rows, cols, dtype, back, seed):
    g = gen(seed)
    codes, scales = ref.random_matrix(rows, cols, g)
    x = torch.randn(m, rows if back else cols, generator=g).to(dtype)
    return codes, scales, x


def run_matmul(codes, scales, x, out_dtype, back):
    rows, cols = codes.shape[0], codes.shape[1] * 2
    m, n = x.shape[0], cols if back else rows
    buf, out = guarded((m, n), out_dtype)
    ws = workspace(q.mx4_matmul_workspace_bytes(rows, cols, back, m))
    q.mx4_matmul(codes.cuda(), scales.cuda(), x.cuda(), out, ws, backward=back)
    torch.cuda.synchronize()
    assert untouched(buf, out.shape)
    return out


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "back"])
@pytest.mark.parametrize("m,rows,cols", SHAPES)
def test_matmul(m, rows, cols, back):
    for dtype, out_dtype in ((torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                             (torch.bfloat16, torch.float32)):
        print_case("mx4_matmul", m, rows, cols, back, dtype, out_dtype)
        codes, scales, x = make_product(m, rows, cols, dtype, back, m + rows + cols)
        out = run_matmul(codes, scales, x, out_dtype, back)
        w = ref.rounded(ref.values(codes, scales), dtype)
        check_product(out, x.double(), w.t().contiguous() if back else w, (dtype, out_dtype))


@pytest.mark.parametrize("m,rows,cols", SHAPES)
def test_matmul4(m, rows, cols):
    for out_dtype in (torch.bfloat16, torch.float16, torch.float32):
        print_case("mx4_matmul4", m, rows, cols, out_dtype)
        g = gen(m + rows + cols)
        codes, scales = ref.random_matrix(rows, cols, g)
        xc, xs = ref.random_matrix(m, cols, g, 122, 129)
        buf, out = guarded((m, rows), out_dtype)
        q.mx4_matmul4(codes.cuda(), scales.cuda(), xc.cuda(), xs.cuda(), out,
                      workspace(q.mx4_matmul4_workspace_bytes(rows, cols, m)))
        torch.cuda.synchronize()
        assert untouched(buf, out.shape)
        check_product(out, ref.values(xc, xs), ref.values(codes, scales), out_dtype)


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "back"])
def test_matmul_reads_scales_over_the_whole_range(back):
    """Weights from subnormal to the largest scales, in fp16 and bf16 (both round the value that the format gives)."""
    for dtype, lo, hi in ((torch.bfloat16, 1, 40), (torch.float16, 100, 120), (torch.bfloat16, 180, 200)):
        print_case("mx4_matmul scales", dtype, lo, hi, back)
        codes, scales = ref.random_matrix(256, 512, gen(lo), lo, hi)
        x = torch.randn(48, 256 if back else 512, generator=gen(hi)).to(dtype)
        out = run_matmul(codes, scales, x, torch.float32, back)
        w = ref.rounded(ref.values(codes, scales), dtype)
        check_product(out, x.double(), w.t().contiguous() if back else w, (dtype, lo))


@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("cols", [160, 512])
def test_products_keep_what_is_not_finite_in_its_row_and_column(m, cols):
    """A NaN or infinity of x reaches its token only, a weight's NaN scale its output column (backward: its group of
    32 columns) only; padding of the last step and tokens past the end never count."""
    rows = 200
    g = gen(cols)
    codes, scales = ref.random_matrix(rows, cols, g)
    print_case("products, not finite", m, cols)
    x = torch.randn(m, cols, generator=g).bfloat16()
    x[m - 1, cols - 1] = float("inf")
    x[0, 0] = float("nan")
    out = run_matmul(codes, scales, x, torch.float32, False).cpu()
    bad = ~torch.isfinite(out)
    assert bad[0].all() and bad[m - 1].all() and not bad[1:m - 1].any()
    if m > 1 and cols % 64:
        zero = (codes[:, -1] >> 4) & 7 == 0   # infinity times a zero weight
        assert torch.equal(torch.isnan(out[m - 1]), zero) or m == 1
    s2 = scales.clone()
    s2[rows - 1, cols // 32 - 1] = 255
    x = torch.randn(m, cols, generator=g).bfloat16()
    out = run_matmul(codes, s2, x, torch.float32, False).cpu()
    assert torch.isnan(out[:, rows - 1]).all() and torch.isfinite(out[:, :rows - 1]).all()
    dy = torch.randn(m, rows, generator=g).bfloat16()
    out = run_matmul(codes, s2, dy, torch.float32, True).cpu()
    assert torch.isnan(out[:, cols - 32:]).all() and torch.isfinite(out[:, :cols - 32]).all()
    dy[0, rows - 1] = float("-inf")
    out = run_matmul(codes, scales, dy, torch.float32, True).cpu()
    assert not torch.isfinite(out[0]).any() and torch.isfinite(out[1:]).all()
    xc, xs = ref.random_matrix(m, cols, g, 120, 128)
    xs[m - 1, cols // 32 - 1] = 255
    out = torch.empty(m, rows, device="cuda")
    q.mx4_matmul4(codes.cuda(), scales.cuda(), xc.cuda(), xs.cuda(), out, workspace(q.mx4_matmul4_workspace_bytes(rows, cols, m)))
    out = out.cpu()
    assert torch.isnan(out[m - 1]).all() and torch.isfinite(out[:m - 1]).all()


def test_products_repeat_bit_for_bit():
    for m, rows, cols, back in ((7, 512, 4096, False), (100, 4096, 512, True), (300, 520, 4128, False)):
        print_case("repeat", m, rows, cols, back)
        codes, scales, x = make_product(m, rows, cols, torch.bfloat16, back, 1)
        a = run_matmul(codes, scales, x, torch.float32, back)
        b = run_matmul(codes, scales, x, torch.float32, back)
        assert torch.equal(a, b)


def test_odd_scale_addresses():
    """Scales are bytes: a view that starts at any address is read right."""
    print_case("odd scale addresses")
    m, rows, cols = 70, 264, 288
    codes, scales, x = make_product(m, rows, cols, torch.bfloat16, False, 9)
    w = ref.rounded(ref.values(codes, scales), torch.bfloat16)
    for off in (1, 2, 3, 5):
        buf = torch.empty(scales.numel() + off, dtype=torch.uint8, device="cuda")
        sv = buf[off:].view(scales.shape)
        sv.copy_(scales)
        for mm in (1, 70):
            out = torch.empty(mm, rows, dtype=torch.float32, device="cuda")
            q.mx4_matmul(codes.cuda(), sv, x[:mm].contiguous().cuda(), out, workspace(q.mx4_matmul_workspace_bytes(rows, cols, False, mm)))
            check_product(out, x[:mm].double(), w, off)
            xc, xs, _ = quantize(x[:mm].contiguous(), False)
            q.mx4_matmul4(codes.cuda(), sv, xc.cuda(), xs.cuda(), out, workspace(q.mx4_matmul4_workspace_bytes(rows, cols, mm)))
            check_product(out, ref.values(xc, xs), ref.values(codes, scales), off)
        dy = torch.randn(mm, rows, generator=gen(off)).bfloat16()
        dx = torch.empty(mm, cols, dtype=torch.float32, device="cuda")
        q.mx4_matmul(codes.cuda(), sv, dy.cuda(), dx, workspace(q.mx4_matmul_workspace_bytes(rows, cols, True, mm)), backward=True)
        check_product(dx, dy.double(), w.t().contiguous(), off)

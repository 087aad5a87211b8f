"""The microscaled products over the whole range of scales, each output at its own
magnitude, at the ends of fp32's range, and with scales at any byte address, in
the few-token kernels and in the tiled ones.

Tolerances as in test_gpu_mx4.py.  The 64-bit product is taken on the device.

A weight's scale is s[row, group] = base + a[row] + b[group], with a and b from 0 to
63.  Forward the values of x in a group are multiplied by 2^-b, backward those of a
row by 2^-a: what an output adds up is all of one magnitude, and a value that is
flushed, or read under a neighbour's scale, stands out in it.
"""
import pytest
import torch

import mx4_ref as ref
import quantized_lora_fine_nf4_amd as q
from conftest import print_case
from mx4_ref import TINY, U16, U32

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# tokens, weight rows, columns: one, two and four weight rows by four tokens, 16 x 16 tiles, workgroups that share a
# compute unit backward, small tiles that have one alone and that share one, large tiles with small ones beside them
SIZES = [(1, 1032, 2080), (3, 4232, 2080), (7, 1032, 2080), (7, 4232, 2080), (8, 4232, 2048), (12, 4232, 2080),
         (16, 264, 2080), (16, 4104, 8224), (30, 8200, 2080), (48, 264, 2080), (48, 4104, 8224), (333, 1032, 2080),
         (1500, 4232, 2080), (4200, 4232, 2080)]


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def values(codes, scales):
    return ref.values(codes, scales).cuda()


def workspace(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda") if nbytes else None


def guarded(m, n, dtype, pad=256):
    buf = torch.full((m * n + 2 * pad,), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[pad:pad + m * n].view(m, n)


def untouched(buf, pad=256):
    return bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[-pad:]).all())


def check(got, a, b, what):
    """got = a b, in 64 bits on the device."""
    want, scale = a @ b, a.abs() @ b.abs()
    assert scale.max().item() < 2.0 ** 127 and scale.min().item() > 2.0 ** -110, "outputs within fp32's normal range"
    tol = 2 * a.shape[1] * U32 * scale + U16[got.dtype] * want.abs() + TINY[got.dtype]
    excess = ((got.double() - want).abs() / tol).max().item()
    assert excess <= 1.0, (what, excess)


def matmul(codes, scales, x, out_dtype, back):
    rows, cols, m = codes.shape[0], 2 * codes.shape[1], x.shape[0]
    buf, out = guarded(m, cols if back else rows, out_dtype)
    q.mx4_matmul(codes, scales, x, out, workspace(q.mx4_matmul_workspace_bytes(rows, cols, back, m)), backward=back)
    assert untouched(buf)
    return out


def matmul4(codes, scales, xc, xs, out_dtype):
    rows, cols, m = codes.shape[0], 2 * codes.shape[1], xc.shape[0]
    buf, out = guarded(m, rows, out_dtype)
    q.mx4_matmul4(codes, scales, xc, xs, out, workspace(q.mx4_matmul4_workspace_bytes(rows, cols, m)))
    assert untouched(buf)
    return out


def steps(n, top):
    """n whole numbers from 0 to top, both of them among the first ones, in no order."""
    v = torch.arange(n, device="cuda") * 37 % (top + 1)
    v[1 if n > 1 else 0] = top
    return v


def weight(rows, cols, base, top, seed):
    """codes, scales over base .. base + 2 top, and the two parts a and b of the scales."""
    g = gen(seed)
    a, b = steps(rows, top), steps(cols // 32, top)
    s = base + a[:, None] + b[None, :]
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    # under scales of 2^126 and 2^127 the magnitudes 0, 0.5, 1 and 1.5, which bfloat16 holds there
    codes[(s > 252).repeat_interleave(16, 1)] &= 0xBB
    assert s.min().item() == base and s.max().item() == base + 2 * top < 255
    return codes, s.to(torch.uint8), a, b


def draw16(m, shift, dtype, e, seed):
    """[m, len(shift)] normal values times 2^(e - shift)."""
    return (torch.randn(m, shift.numel(), generator=gen(seed), device="cuda", dtype=torch.float64) *
            torch.exp2((e - shift).double())).to(dtype)


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "back"])
@pytest.mark.parametrize("m,rows,cols", SIZES)
def test_matmul_under_every_scale(m, rows, cols, back):
    """All 255 scales in bfloat16 (subnormal weights against large tokens, the largest against small ones), and in
    float16 those around its range, whose weights it rounds to subnormals and to zero."""
    for dtype, base, top, e in ((BF16, 0, 63, 50), (BF16, 64, 63, 0), (BF16, 128, 63, -45), (FP16, 100, 20, 8)):
        print_case("mx4_matmul scales", m, rows, cols, back, dtype, base)
        codes, scales, a, b = weight(rows, cols, base, top, m + rows + base)
        x = draw16(m, a if back else b.repeat_interleave(32), dtype, e, m)
        w = values(codes, scales).to(FP32).to(dtype).double()
        assert torch.isfinite(w).all()
        if dtype is FP16 and not back:
            live = (w != 0).any(1)   # rows of weights under half its smallest number
            w, out = w[live], matmul(codes, scales, x, FP32, back)
            assert (out[:, ~live] == 0).all()
            check(out[:, live], x.double(), w.t().contiguous(), (dtype, base))
            continue
        out = matmul(codes, scales, x, FP32, back)
        check(out, x.double(), w if back else w.t().contiguous(), (dtype, base))


@pytest.mark.parametrize("m,rows,cols", SIZES)
def test_matmul4_under_every_scale(m, rows, cols):
    """Small scales of one operand against large ones of the other, both ways round."""
    for base, xbase in ((0, 190), (64, 127), (128, 63)):
        print_case("mx4_matmul4 scales", m, rows, cols, base)
        codes, scales, _, b = weight(rows, cols, base, 63, m + rows + base)
        xc = torch.randint(0, 256, (m, cols // 2), generator=gen(m), dtype=torch.uint8, device="cuda")
        xs = xbase + steps(m, 63 if m > 1 else 0)[:, None] - b[None, :]
        assert xs.min().item() >= 0 and xs.max().item() < 255
        xs = xs.to(torch.uint8)
        out = matmul4(codes, scales, xc, xs, FP32)
        check(out, values(xc, xs), values(codes, scales).t().contiguous(), base)


@pytest.mark.parametrize("m,rows", [s[:2] for s in SIZES])
def test_products_at_the_ends_of_fp32(m, rows):
    """What is far below fp32's smallest number is 0, what is past its largest an infinity of its sign.  One group of 32 is
    not 0 in each row, so that an infinity meets no other."""
    cols = 544
    print_case("ends of fp32", m, rows)
    g = gen(m + rows)
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 0, dtype=torch.uint8, device="cuda")
    xc = torch.randint(0, 256, (m, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    xs = torch.full((m, cols // 32), 10, dtype=torch.uint8, device="cuda")   # 544 * 36 * 2^-244 in all
    out = matmul4(codes, scales, xc, xs, FP32)
    assert (out == 0).all()
    # all weights 6 and -6 in turn of the rows, all tokens 6: 32 * 36 * 2^(s + t - 254)
    codes.zero_()
    xc.fill_(0x77)
    xs.fill_(254)
    at = torch.arange(rows, device="cuda") % (cols // 32)
    odd = torch.arange(rows, device="cuda") % 2
    for i in range(16):
        codes[torch.arange(rows, device="cuda"), 16 * at + i] = (0x77 + 0x88 * odd).to(torch.uint8)
    sign = (1 - 2 * odd).double()
    for s, big in ((200, True), (110, False)):
        scales.fill_(s)
        out = matmul4(codes, scales, xc, xs, FP32)
        want = sign * (float("inf") if big else 32 * 36 * 2.0 ** (s + 254 - 254))
        assert torch.equal(out.double(), want.expand(m, rows)), s
    # and of a 16-bit operand
    scales.fill_(250)
    x = torch.full((m, cols), 2.0 ** 100, dtype=BF16, device="cuda")
    assert torch.equal(matmul(codes, scales, x, FP32, False).double(), (sign * float("inf")).expand(m, rows))


@pytest.mark.parametrize("m,rows", [s[:2] for s in SIZES])
def test_sums_below_the_normal_range_of_fp32(m, rows):
    """Subnormal sums keep fp32's step there: each addition of K is within one such step, toward zero or nearest."""
    cols = 544
    for s, t in ((1, 110), (60, 50), (120, 3)):   # units of 0.25 * 2^(s + t - 254): 2^-145, -146 and -133
        print_case("subnormal sums", m, rows, s, t)
        g = gen(m + s)
        codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
        xc = torch.randint(0, 256, (m, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows, cols // 32), s, dtype=torch.uint8, device="cuda")
        xs = torch.full((m, cols // 32), t, dtype=torch.uint8, device="cuda")
        want = values(xc, xs) @ values(codes, scales).t().contiguous()
        out = matmul4(codes, scales, xc, xs, FP32)
        # sums of multiples of 2^-146 or more, below 2^-119: fp32 holds all of them up to 2^24 units
        tol = cols * 2.0 ** -149 + 2 * cols * U32 * (values(xc, xs).abs() @ values(codes, scales).abs().t().contiguous())
        assert ((out.double() - want).abs() <= tol).all(), (s, t)


# tokens, rows, cols: few tokens (four columns' rows at a time, and tiles), small tiles alone and in pairs, large tiles;
# rows of scales of odd lengths (17) and of even ones
ODD = [(1, 264, 288), (5, 4232, 544), (70, 264, 288), (333, 1032, 544), (600, 4232, 544), (1500, 4232, 800),
       (4200, 4232, 544)]


@pytest.mark.parametrize("m,rows,cols", ODD)
def test_scales_at_any_address(m, rows, cols):
    """Scales are bytes: views that start at odd addresses are read right by every kernel, and nothing beside them."""
    g = gen(m + cols)
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(118, 124, (rows, cols // 32), generator=g, dtype=torch.uint8, device="cuda")
    xc = torch.randint(0, 256, (m, cols // 2), generator=g, dtype=torch.uint8, device="cuda")
    xs = torch.randint(122, 129, (m, cols // 32), generator=g, dtype=torch.uint8, device="cuda")
    x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
    dy = torch.randn(m, rows, generator=g, device="cuda").to(BF16)
    v = values(codes, scales)
    want = [matmul(codes, scales, x, FP32, False), matmul(codes, scales, dy, FP32, True), matmul4(codes, scales, xc, xs, FP32)]
    check(want[0], x.double(), v.t().contiguous(), "forward")
    check(want[1], dy.double(), v, "backward")
    check(want[2], values(xc, xs), v.t().contiguous(), "codes")

    def moved(s, off):
        buf = torch.full((s.numel() + off + 16,), 255, dtype=torch.uint8, device="cuda")   # NaN around it
        buf[off:off + s.numel()] = s.reshape(-1)
        return buf[off:off + s.numel()].view(s.shape)

    for off in (1, 2, 3, 5):
        print_case("scales at", off, m, rows, cols)
        sv, xv = moved(scales, off), moved(xs, 8 - off)
        got = [matmul(codes, sv, x, FP32, False), matmul(codes, sv, dy, FP32, True), matmul4(codes, sv, xc, xv, FP32)]
        for a, b in zip(got, want):
            assert torch.equal(a, b), off

"""The microscaled products where they run on whole tiles, on whole rounds of
large tiles with smaller ones beside them, at every number of few tokens, on
matrices past 32-bit offsets, in graphs and on several streams.

Tolerances as in test_gpu_mx4.py.  The 64-bit product is taken on the device.
"""
import pytest
import torch

import mx4_ref as ref
import quantized_lora_fine_nf4_amd as q
from conftest import print_case
from mx4_ref import TINY, U16, U32

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    q.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(rows, cols, g, lo=118, hi=124):
    return (torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device="cuda"),
            torch.randint(lo, hi, (rows, cols // 32), generator=g, dtype=torch.uint8, device="cuda"))


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
    tol = 2 * a.shape[1] * U32 * scale + U16[got.dtype] * want.abs() + TINY[got.dtype]
    excess = ((got.double() - want).abs() / tol).max().item()
    assert excess <= 1.0, (what, excess)


def matmul(codes, scales, x, out, back=False, stream=None, ws=None):
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    if ws is None:
        ws = workspace(q.mx4_matmul_workspace_bytes(rows, cols, back, x.shape[0]))
    q.mx4_matmul(codes, scales, x, out, ws, backward=back, stream=stream)
    return ws


def matmul4(codes, scales, xc, xs, out, stream=None, ws=None):
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    if ws is None:
        ws = workspace(q.mx4_matmul4_workspace_bytes(rows, cols, xc.shape[0]))
    q.mx4_matmul4(codes, scales, xc, xs, out, ws, stream=stream)
    return ws


# tokens, output columns, reduction: one round of large tiles, whole and ragged; large ones with small ones beside
# them, the small ones' reduction whole and split; short and odd reductions
TILED = [(4096, 4096, 512), (3900, 4000, 544), (3900, 4064, 96), (4097, 4128, 288), (4000, 4608, 512), (4000, 4256, 2080),
         (2100, 8448, 1056), (520, 32768, 160), (1111, 4384, 2080), (300, 2080, 8224)]


@pytest.mark.parametrize("back", [False, True], ids=["fwd", "back"])
@pytest.mark.parametrize("m,ncol,kred", TILED)
def test_matmul_on_whole_tiles(m, ncol, kred, back):
    rows, cols = (kred - 24, ncol) if back else (ncol - 8, kred)   # rows of eights, columns of 32s
    g = gen(m + ncol + kred)
    codes, scales = matrix(rows, cols, g)
    v = values(codes, scales)
    for dtype, out_dtype in ((BF16, BF16), (FP16, FP16), (FP16, FP32)):
        print_case("mx4_matmul tiles", m, rows, cols, back, dtype, out_dtype)
        x = torch.randn(m, rows if back else cols, generator=g, device="cuda").to(dtype)
        buf, out = guarded(m, cols if back else rows, out_dtype)
        matmul(codes, scales, x, out, back)
        w = v.float().to(dtype).double()
        check(out, x.double(), w if back else w.t().contiguous(), (dtype, out_dtype))
        assert untouched(buf)


@pytest.mark.parametrize("m,ncol,kred", TILED)
def test_matmul4_on_whole_tiles(m, ncol, kred):
    g = gen(m + ncol + kred)
    codes, scales = matrix(ncol - 8, kred, g)
    xc, xs = matrix(m, kred, g, 122, 129)
    a, b = values(xc, xs), values(codes, scales).t().contiguous()
    for out_dtype in (BF16, FP16, FP32):
        print_case("mx4_matmul4 tiles", m, ncol - 8, kred, out_dtype)
        buf, out = guarded(m, ncol - 8, out_dtype)
        matmul4(codes, scales, xc, xs, out)
        check(out, a, b, out_dtype)
        assert untouched(buf)


@pytest.mark.parametrize("rows", [136, 1032, 4104])
@pytest.mark.parametrize("cols", [32, 64, 96, 160, 224, 256, 288, 704, 768, 800, 960, 1024, 1056, 1504, 1568, 2080])
def test_matmul_around_rounds_of_scales(rows, cols):
    """Tiles that have a compute unit alone, that share it, and large ones, with reductions that end before, at and after
    a round of scales and with rows shorter than what is loaded of them at once; one row of NaN scales, and nothing of a
    neighbour's in another one."""
    m = 4200
    g = gen(rows + cols)
    codes, scales = matrix(rows, cols, g)
    bad = rows // 2 + 1
    scales[bad] = 255
    w = values(codes, scales).float().to(BF16).double()
    ok = torch.arange(rows, device="cuda") != bad
    print_case("rounds of scales", m, rows, cols)
    x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
    buf, out = guarded(m, rows, BF16)
    matmul(codes, scales, x, out)
    check(out[:, ok], x.double(), w[ok].t().contiguous(), "forward")
    assert torch.isnan(out[:, bad]).all() and untouched(buf)


@pytest.mark.parametrize("m", [600, 1500, 4200])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 9, 11, 13])
def test_every_end_of_the_buffers_turns(steps, m):
    """Reductions of so many steps, and of so many whole ones and a part of one: forward and backward (steps of 64) and
    of both operands in codes (256), with a NaN in every matrix's neighbourhood and not in it."""
    g = gen(31 * steps + m)
    for short in (0, 32):
        k64, k256, n = 64 * steps - short, 256 * steps - 3 * short, 4232
        print_case("ends", m, steps, short)
        codes, scales = matrix(n, k64, g)
        x = torch.full((m + 1, k64), float("nan"), dtype=BF16, device="cuda")[:m]
        x.copy_(torch.randn(m, k64, generator=g, device="cuda"))
        buf, out = guarded(m, n, BF16)
        matmul(codes, scales, x, out)
        check(out, x.double(), values(codes, scales).double().t().contiguous(), "forward")
        assert untouched(buf)
        # backward the reduction is the weight's rows, eights of them
        n = 4224
        codes, scales = matrix(k64, n, g)
        buf, out = guarded(m, n, BF16)
        matmul(codes, scales, x, out, back=True)
        check(out, x.double(), values(codes, scales).double(), "backward")
        assert untouched(buf)
        n = 4232
        codes, scales = matrix(n, k256, g)
        xc, xs = matrix(m, k256, g)
        buf, out = guarded(m, n, BF16)
        matmul4(codes, scales, xc, xs, out)
        check(out, values(xc, xs).double(), values(codes, scales).double().t().contiguous(), "codes")
        assert untouched(buf)


@pytest.mark.parametrize("rows,cols", [(1032, 544), (4096, 4096), (520, 6176), (2048, 224)])
def test_every_number_of_few_tokens(rows, cols):
    """All the token counts at which another kernel, tile or split may begin."""
    g = gen(rows + cols)
    codes, scales = matrix(rows, cols, g)
    v = values(codes, scales)
    w, vt = v.float().to(BF16).double(), v.t().contiguous()
    wt = w.t().contiguous()
    for m in (*range(1, 19), 24, 31, 32, 33, 47, 48, 49, 63, 64, 65, 96, 129):
        print_case("few tokens", m, rows, cols)
        x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
        buf, out = guarded(m, rows, BF16)
        matmul(codes, scales, x, out)
        check(out, x.double(), wt, ("forward", m))
        assert untouched(buf)
        y = torch.randn(m, rows, generator=g, device="cuda").to(BF16)
        buf, out = guarded(m, cols, FP32)
        matmul(codes, scales, y, out, True)
        check(out, y.double(), w, ("backward", m))
        assert untouched(buf)
        xc, xs = matrix(m, cols, g, 122, 129)
        buf, out = guarded(m, rows, FP16)
        matmul4(codes, scales, xc, xs, out)
        check(out, values(xc, xs), vt, ("codes", m))
        assert untouched(buf)


@pytest.mark.parametrize("m,rows,cols", [(700, 1000, 1504), (1500, 520, 480), (4096, 72, 512), (4097, 72, 512), (300, 3000, 96),
                                         (333, 88, 2528), (1001, 2000, 64), (200, 1000, 2016), (130, 8, 32)])
def test_many_tokens_through_small_weights(m, rows, cols):
    """Where the few-token kernels take many tokens too: waves that share the columns, and one wave for all of them."""
    g = gen(m + cols)
    codes, scales = matrix(rows, cols, g)
    scales[rows // 2, 0] = 255
    v = values(codes, scales)
    w = v.float().to(FP16).double()
    ok = torch.arange(rows, device="cuda") != rows // 2
    print_case("many tokens, small weight", m, rows, cols)
    for out_dtype in (FP16, FP32):
        x = torch.randn(m, cols, generator=g, device="cuda").to(FP16)
        buf, out = guarded(m, rows, out_dtype)
        matmul(codes, scales, x, out)
        check(out[:, ok], x.double(), w[ok].t().contiguous(), ("forward", out_dtype))
        assert torch.isnan(out[:, rows // 2]).all() and untouched(buf)
        xc, xs = matrix(m, cols, g, 122, 129)
        buf, out = guarded(m, rows, out_dtype)
        matmul4(codes, scales, xc, xs, out)
        check(out[:, ok], values(xc, xs), v[ok].t().contiguous(), ("codes", out_dtype))
        assert torch.isnan(out[:, rows // 2]).all() and untouched(buf)
        y = torch.randn(m, rows, generator=g, device="cuda").to(FP16)
        buf, out = guarded(m, cols, out_dtype)
        matmul(codes, scales, y, out, True)
        check(out[:, 32:], y.double(), w[:, 32:].nan_to_num(), ("backward", out_dtype)) if cols > 32 else None
        assert torch.isnan(out[:, :32]).all() and untouched(buf)


@pytest.mark.parametrize("m", [600, 4000])
def test_large_tiles_keep_what_is_not_finite(m):
    """The first piece of the last, ragged step holds what a piece past the row's end reads in its place; a neighbour
    row, the next token's first value and tokens past the last one are not finite either."""
    rows, cols = 4232, 544
    g = gen(m)
    codes, scales = matrix(rows, cols, g)
    x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
    x[5, 512] = float("inf")
    x[7, 0] = float("nan")
    print_case("large tiles, not finite", m)
    out = torch.empty(m, rows, device="cuda")
    matmul(codes, scales, x, out)
    bad = (~torch.isfinite(out)).any(1).nonzero().flatten().tolist()
    assert bad == [5, 7] and torch.isnan(out[7]).all()
    x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
    s2 = scales.clone()
    s2[9, 16] = 255
    s2[rows - 1, 0] = 255
    matmul(codes, s2, x, out)
    bad = (~torch.isfinite(out)).any(0).nonzero().flatten().tolist()
    assert bad == [9, rows - 1]
    xc, xs = matrix(m, cols, g, 122, 129)
    matmul4(codes, s2, xc, xs, out)
    assert (~torch.isfinite(out)).any(0).nonzero().flatten().tolist() == [9, rows - 1]
    xs[3, 16] = 255
    xs[m - 1, 0] = 255
    matmul4(codes, scales, xc, xs, out)
    assert (~torch.isfinite(out)).any(1).nonzero().flatten().tolist() == [3, m - 1]
    dy = torch.randn(m, rows, generator=g, device="cuda").to(BF16)
    dx = torch.empty(m, cols, device="cuda")
    s2 = scales.clone()
    s2[rows - 1, 1] = 255   # the row that rows past the last one read in their place
    matmul(codes, s2, dy, dx, True)
    assert (~torch.isfinite(dx)).any(0).nonzero().flatten().tolist() == list(range(32, 64))
    dy[11, rows - 1] = float("inf")
    matmul(codes, scales, dy, dx, True)
    assert (~torch.isfinite(dx)).any(1).nonzero().flatten().tolist() == [11]


# ---- past 32 bits ----------------------------------------------------------

def test_outputs_and_tokens_past_32_bits():
    m, rows, cols = (1 << 19) + 77, 8200, 256
    print_case("past 32 bits: outputs", m, rows, cols)
    g = gen(1)
    codes, scales = matrix(rows, cols, g)
    v = values(codes, scales).float().to(BF16).double()
    x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
    at = torch.tensor([0, 1, 255, 256, (1 << 18) + 3, (1 << 19) - 1, 1 << 19, m - 2, m - 1], device="cuda")
    out = torch.empty(m, rows, dtype=BF16, device="cuda")
    matmul(codes, scales, x, out)
    check(out[at], x[at].double(), v.t().contiguous(), "forward")
    dx = torch.empty(m, cols, dtype=FP32, device="cuda")
    matmul(codes, scales, out, dx, True)
    check(dx[at], out[at].double(), v, "backward")


def test_token_codes_past_32_bits():
    m, rows, cols = (1 << 20) + 300, 136, 8224
    print_case("past 32 bits: token codes", m, rows, cols)
    g = gen(2)
    codes, scales = matrix(rows, cols, g)
    xc, xs = matrix(m, cols, g, 122, 129)
    at = torch.tensor([0, 255, 256, (1 << 19) + 3, 1 << 20, m - 2, m - 1], device="cuda")
    out = torch.empty(m, rows, dtype=FP32, device="cuda")
    matmul4(codes, scales, xc, xs, out)
    check(out[at], values(xc[at], xs[at]), values(codes, scales).t().contiguous(), "codes")


def test_weights_past_32_bits():
    rows, cols = (1 << 17) + 40, (1 << 16) + 32
    g = gen(3)
    codes, scales = matrix(rows, cols, g)
    last = values(codes[-64:], scales[-64:]).float().to(BF16).double()
    for m in (1, 7, 30, 300):
        print_case("past 32 bits: weight", m, rows, cols)
        x = torch.randn(m, cols, generator=g, device="cuda").to(BF16)
        out = torch.empty(m, rows, dtype=FP32, device="cuda")
        matmul(codes, scales, x, out)
        check(out[:, -64:], x.double(), last.t().contiguous(), ("forward", m))
        xc, xs = matrix(m, cols, g, 122, 129)
        matmul4(codes, scales, xc, xs, out)
        check(out[:, -64:], values(xc, xs), values(codes[-64:], scales[-64:]).t().contiguous(), ("codes", m))
        dy = torch.zeros(m, rows, dtype=BF16, device="cuda")
        dy[:, -64:] = torch.randn(m, 64, generator=g, device="cuda").to(BF16)
        dx = torch.empty(m, cols, dtype=FP32, device="cuda")
        matmul(codes, scales, dy, dx, True)
        check(dx, dy[:, -64:].double(), last, ("backward", m))


def test_narrow_weights_with_more_tokens_than_a_launch_takes():
    m, rows, cols = 1 << 20, 16456, 64
    print_case("narrow weight, many tokens", m, rows, cols)
    g = gen(4)
    codes, scales = matrix(rows, cols, g)
    xc, xs = matrix(m, cols, g, 122, 129)
    out = torch.empty(m, rows, dtype=BF16, device="cuda")
    matmul4(codes, scales, xc, xs, out)
    cut = (1 << 34) // rows
    at = torch.cat([torch.arange(0, 40), torch.arange(cut - 40, cut + 40), torch.arange(m - 40, m)]).cuda()
    check(out[at], values(xc[at], xs[at]), values(codes, scales).t().contiguous(), "codes")


def test_codec_past_32_bits():
    rows, cols = (1 << 16) + 3, 1 << 16
    print_case("past 32 bits: codec", rows, cols)
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-2:] = torch.randn(2, cols, generator=gen(5), device="cuda").to(BF16)
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    err = torch.empty(1, dtype=torch.float64, device="cuda")
    q.mx4_quantize(x, codes, scales, err, workspace(q.mx4_quantize_workspace_bytes(rows, cols)))
    c, s = ref.quantize(x[-2:].cpu())
    assert torch.equal(codes[-2:].cpu(), c) and torch.equal(scales[-2:].cpu(), s)
    assert not codes[:-2].any() and not scales[:-2].any()
    e = (x[-2:].cpu().double() - ref.values(c, s)).square().sum().item()
    assert abs(err.item() - e) <= 2 * cols * 2.0 ** -52 * e
    q.mx4_dequantize(codes, scales, x)
    assert torch.equal(x[-2:].cpu(), ref.values(c, s).to(BF16)) and not x[:-2].any()


# ---- graphs and streams ----------------------------------------------------

# few tokens, split small tiles, large tiles with small ones beside them
MIX = [(3, 1032, 2080, True), (40, 2048, 4128, False), (300, 2080, 4128, False), (300, 4128, 2080, True),
       (4000, 4256, 2080, False)]


def test_captured_and_replayed():
    jobs = []
    for m, rows, cols, back in MIX:
        g = gen(m)
        codes, scales = matrix(rows, cols, g)
        x = torch.randn(m, rows if back else cols, generator=g, device="cuda").to(BF16)
        jobs.append([codes, scales, x, torch.empty(m, cols if back else rows, dtype=BF16, device="cuda"), back])
        matmul(*jobs[-1])   # loads the kernels
    g4 = gen(9)
    c4, s4 = matrix(2080, 4128, g4)
    xc, xs = matrix(300, 4128, g4, 122, 129)
    out4 = torch.empty(300, 2080, dtype=FP32, device="cuda")
    matmul4(c4, s4, xc, xs, out4)
    torch.cuda.synchronize()
    spaces = [workspace(q.mx4_matmul_workspace_bytes(j[0].shape[0], 2 * j[0].shape[1], j[4], j[2].shape[0])) for j in jobs]
    ws4 = workspace(q.mx4_matmul4_workspace_bytes(2080, 4128, 300))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for j, ws in zip(jobs, spaces):
            matmul(*j, ws=ws)
        matmul4(c4, s4, xc, xs, out4, ws=ws4)
    for k in range(4):
        print_case("captured products, replay", k)
        for j in jobs:
            j[2].copy_(torch.randn(j[2].shape, generator=gen(100 + k), device="cuda"))
            j[3].fill_(float("nan"))
        xc.random_(0, 256, generator=gen(k))
        out4.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for j in jobs:
            eager = torch.empty_like(j[3])
            matmul(j[0], j[1], j[2], eager, j[4])
            assert torch.equal(eager, j[3]), tuple(j[2].shape)
        eager = torch.empty_like(out4)
        matmul4(c4, s4, xc, xs, eager)
        assert torch.equal(eager, out4)
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls that share operands, each with an output and a workspace of its own, on two streams at the same time."""
    for m, rows, cols, back in MIX:
        print_case("two streams", m, rows, cols, back)
        g = gen(m)
        codes, scales = matrix(rows, cols, g)
        x = torch.randn(m, rows if back else cols, generator=g, device="cuda").to(BF16)
        want = torch.empty(m, cols if back else rows, dtype=FP32, device="cuda")
        matmul(codes, scales, x, want, back)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        nbytes = q.mx4_matmul_workspace_bytes(rows, cols, back, m)
        runs = [(s, torch.full_like(want, float("nan")), workspace(nbytes)) for s in streams for _ in range(3)]
        torch.cuda.synchronize()
        for s, out, ws in runs:
            q.mx4_matmul(codes, scales, x, out, ws, backward=back, stream=s)
        torch.cuda.synchronize()
        for _, out, _ in runs:
            assert torch.equal(out, want)

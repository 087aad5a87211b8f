"""The adapted linear layer's operators as they are measured: cases, inputs, plain forms.

A QLoRA layer keeps its weight W in NF4 and learns a low-rank adapter:

    h   = s drop(x) A^T                       lora_project, forward
    z   = x W^T + h B^T + bias                linear, forward
    out = act(z) + residual
    dz  = dout act'(z), dbias = sum dz        act_grad
    dh  = s dz B                              lora_project, backward
    dB  = dz^T h, dA = dh^T drop(x)           lora_grad
    dx  = dz W + drop(dh A) + residual        linear, backward

The dropout mask is a function of (seed, offset, element): Philox4x32 with 7
rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1,
2, 3", 2011), counter (group of eight elements, offset), key seed, one 16-bit
lane per element, low half of each word first.
"""
import math

import numpy as np
import torch

own = False

BF16, FP16 = "bf16", "fp16"
TORCH = {BF16: torch.bfloat16, FP16: torch.float16}
DEV = "cuda"

# The 16 NF4 levels (fp32).
LEVELS = np.array([0xbf800000, 0xbf3239b1, 0xbf066b2e, 0xbeca329e, 0xbe91a24b, 0xbe3d353d, 0xbdba7869, 0x00000000,
                   0x3da2fb01, 0x3e24cadf, 0x3e7c04da, 0x3ead0336, 0x3ee1a4b5, 0x3f1007a9, 0x3f3913b0, 0x3f800000],
                  np.uint32).view(np.float32)

# (rows, cols) of the matrices of the 1.4B-, 7B- and 14B-shaped stacks.
SHAPES = [(6144, 2048), (2048, 2048), (8192, 2048), (2048, 8192), (4096, 4096), (11008, 4096), (4096, 11008),
          (5120, 5120), (13824, 5120), (5120, 13824)]
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def case_dropout(name, m, n, dtype, p):
    return {"name": name, "op": "dropout", "m": m, "n": n, "dtype": dtype, "p": p}


def case_linear(name, m, rows, cols, dtype, dq, rank, act="none", bias=False, preact=False, residual=False):
    return {"name": name, "op": "linear", "m": m, "rows": rows, "cols": cols, "dtype": dtype, "dq": dq, "rank": rank,
            "act": act, "bias": bias, "preact": preact, "residual": residual}


def case_linear_back(name, m, rows, cols, dtype, dq, rank, p, residual):
    return {"name": name, "op": "linear_back", "m": m, "rows": rows, "cols": cols, "dtype": dtype, "dq": dq,
            "rank": rank, "p": p, "residual": residual}


def case_act_grad(name, m, n, dtype, act, bias):
    return {"name": name, "op": "act_grad", "m": m, "n": n, "dtype": dtype, "act": act, "bias": bias}


def case_project(name, m, k, rank, dtype, back, p):
    return {"name": name, "op": "project", "m": m, "k": k, "rank": rank, "dtype": dtype, "back": back, "p": p}


def case_lora_grad(name, m, n, rank, dtype, side, p):
    return {"name": name, "op": "lora_grad", "m": m, "n": n, "rank": rank, "dtype": dtype, "side": side, "p": p}


def listed():
    return [
        # dropout of one short sequence's hidden state (latency) and of a training batch's FFN activation
        case_dropout("dropout 17x5120 bf16", 17, 5120, BF16, 0.05),
        case_dropout("dropout 8192x13824 fp16", 8192, 13824, FP16, 0.1),
        # one decoded token through the gate matrix of the 14B shape, adapter unmerged
        case_linear("linear 1 token 13824x5120", 1, 13824, 5120, BF16, True, 16, act="silu"),
        # a training batch through the same matrix, the preactivation kept for the backward pass
        case_linear("linear 4096 tokens 13824x5120", 4096, 13824, 5120, BF16, True, 16, act="silu", bias=True,
                    preact=True),
        # input gradient of a short odd batch through the 1.4B shape's up matrix, fp16 without double quantisation
        case_linear_back("linear back 333 tokens 8192x2048", 333, 8192, 2048, FP16, False, 64, 0.1, False),
        # input gradient of a training batch, added to the gradient of the layers that share the input
        case_linear_back("linear back 4096 tokens 13824x5120", 4096, 13824, 5120, BF16, True, 16, 0.05, True),
        # gradient through the activation of a training batch, with the bias gradient
        case_act_grad("act grad 4096x13824", 4096, 13824, BF16, "silu", True),
        # down projection of one decoded token (latency), and of a training batch with dropout
        case_project("project 1 token 5120 r16", 1, 5120, 16, BF16, False, 0.0),
        case_project("project 8192 tokens 5120 r64", 8192, 5120, 64, BF16, False, 0.05),
        # its gradient: the batch's output gradient through B
        case_project("project back 4096 tokens 13824 r16", 4096, 13824, 16, BF16, True, 0.0),
        # adapter gradients of a training batch, and of a ragged one at a high rank
        case_lora_grad("grad A 4096 tokens 5120 r16", 4096, 5120, 16, BF16, "A", 0.05),
        case_lora_grad("grad B 1999 tokens 8192 r64", 1999, 8192, 64, FP16, "B", 0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice([BF16, FP16])
    p = rng.choice([0.0, 0.05, 0.1, 0.5])
    rank = rng.choice([4, 8, 16, 24, 32, 64, 100, 128])
    op = rng.choice(["dropout", "linear", "linear", "linear_back", "linear_back", "act_grad", "project", "project",
                     "lora_grad", "lora_grad"])
    if op == "dropout":
        c = case_dropout("", _log_int(rng, 1, 8192), _log_int(rng, 1, 13824), dtype, rng.choice([0.05, 0.1, 0.5]))
    elif op in ("linear", "linear_back"):
        if rng.random() < 0.5:
            rows, cols = rng.choice(SHAPES)
        else:
            rows, cols = 128 * _log_int(rng, 1, 100), 128 * _log_int(rng, 1, 50)
        m = _log_int(rng, 1, 4096)
        dq = rng.random() < 0.6
        if op == "linear":
            c = case_linear("", m, rows, cols, dtype, dq, rng.choice([0, rank]), rng.choice(ACTS), rng.random() < 0.5,
                            rng.random() < 0.5, rng.random() < 0.4)
            if c["rank"] == 0 and c["act"] == "none":
                c["bias"] = True
        else:
            c = case_linear_back("", m, rows, cols, dtype, dq, rank, p, rng.random() < 0.5)
    elif op == "act_grad":
        c = case_act_grad("", _log_int(rng, 1, 4096), 8 * _log_int(rng, 1, 1728), dtype, rng.choice(ACTS[1:]),
                          rng.random() < 0.7)
    elif op == "project":
        back = rng.random() < 0.5
        c = case_project("", _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1728), rank, dtype, back, 0.0 if back else p)
    else:
        side = rng.choice("AB")
        c = case_lora_grad("", _log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1728), rank, dtype, side,
                           p if side == "A" else 0.0)
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(TORCH[dtype])


def _quantised(g, rows, cols, dq):
    """A weight matrix in its NF4 form: codes two to a byte, low nibble first; fp32 absmax per 64 weights, or
    int8 with an fp32 scale per 256 of them."""
    w = (torch.randn(rows * cols // 64, 64, generator=g, device=DEV) * 0.02).to(torch.bfloat16).float()
    absmax = w.abs().amax(1)
    lv = torch.from_numpy(LEVELS).to(DEV)
    code = torch.bucketize((w / absmax[:, None]).reshape(-1), (lv[1:] + lv[:-1]) / 2, out_int32=True).to(torch.uint8)
    out = {"codes": code[0::2] | (code[1::2] << 4)}
    if dq:
        grp = absmax.view(-1, 256) if absmax.numel() % 256 == 0 else absmax.view(1, -1)
        s2 = grp.amax(1) / 127
        out["qabsmax"] = torch.round(grp / s2[:, None]).to(torch.int8).reshape(-1)
        out["scale2"] = s2
    else:
        out["absmax"] = absmax
    return out


def _rng_state(g):
    return torch.randint(0, 1 << 62, (2,), generator=g, device=DEV, dtype=torch.int64)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], case["dtype"]
    s = {"case": dict(case), "rng": _rng_state(g)}
    if op == "dropout":
        s["x"] = _normal(g, (case["m"], case["n"]), 1.0, dt)
    elif op in ("linear", "linear_back"):
        m, rows, cols, r = case["m"], case["rows"], case["cols"], case["rank"]
        back = op == "linear_back"
        nout = cols if back else rows
        s.update(_quantised(g, rows, cols, case["dq"]))
        s["x"] = _normal(g, (m, rows if back else cols), 0.1 if back else 1.0, dt)
        if r:
            s["u"] = _normal(g, (m, r), 0.1 if back else 0.5, dt)
            s["v"] = _normal(g, (r, cols) if back else (rows, r), 0.05, dt)
        if case.get("bias"):
            s["bias"] = _normal(g, (rows,), 0.1, dt)
        if case["residual"]:
            s["residual"] = _normal(g, (m, nout), 1.0, dt)
    elif op == "act_grad":
        s["dy"] = _normal(g, (case["m"], case["n"]), 0.1, dt)
        s["z"] = _normal(g, (case["m"], case["n"]), 1.5, dt)
    elif op == "project":
        k, r = case["k"], case["rank"]
        s["x"] = _normal(g, (case["m"], k), 0.1 if case["back"] else 1.0, dt)
        s["w"] = _normal(g, (k, r) if case["back"] else (r, k), 1.0 / math.sqrt(k), dt)
    else:
        s["u"] = _normal(g, (case["m"], case["rank"]), 0.5 if case["side"] == "B" else 0.1, dt)
        s["x"] = _normal(g, (case["m"], case["n"]), 1.0 if case["side"] == "A" else 0.1, dt)
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program that calls the framework keeps: the matrix's handle, workspaces and output buffers."""
    import quantized_lora_fine_nf4_amd as q
    c = s["case"]
    op, t16 = c["op"], TORCH[c["dtype"]]
    need = 0
    if op == "dropout":
        s["out"] = torch.empty_like(s["x"])
    elif op in ("linear", "linear_back"):
        back = op == "linear_back"
        ptr = lambda k: int(s[k].data_ptr()) if k in s else None
        s["layer"] = q.nf4_layer(c["rows"] * c["cols"], None, ptr("codes"), ptr("absmax"), ptr("qabsmax"),
                                 ptr("scale2"), None)
        s["fmt"] = q.fmt(q.NF4_BF16 if c["dtype"] == BF16 else q.NF4_FP16, c["dq"])
        s["out"] = _empty((c["m"], c["cols"] if back else c["rows"]), t16)
        if c.get("preact"):
            s["preact"] = _empty((c["m"], c["rows"]), t16)
        need = q.nf4_matmul_workspace_bytes(c["rows"], c["cols"], back, c["m"])
    elif op == "act_grad":
        s["dz"] = torch.empty_like(s["dy"])
        if c["bias"]:
            s["dbias"] = _empty((c["n"],), torch.float32)
            need = q.nf4_act_grad_workspace_bytes(c["m"], c["n"])
    elif op == "project":
        s["h"] = _empty((c["m"], c["rank"]), t16)
    else:
        s["grad"] = _empty((c["rank"], c["n"]) if c["side"] == "A" else (c["n"], c["rank"]), torch.float32)
        need = q.nf4_lora_grad_workspace_bytes(c["m"], c["n"], c["rank"])
    s["ws"] = _empty((need,), torch.uint8) if need else None


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import quantized_lora_fine_nf4_amd as q
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        q.nf4_dropout(s["x"], s["out"], c["p"], s["rng"])
        return s["out"]
    if op == "linear":
        q.nf4_linear(s["layer"], c["rows"], c["cols"], s["fmt"], s["x"], s["out"], s["ws"],
                     lora=(s["u"], s["v"]) if c["rank"] else None, bias=s.get("bias"),
                     act=getattr(q, "NF4_ACT_" + c["act"].upper()), preact=s.get("preact"),
                     residual=s.get("residual"))
        return (s["out"], s["preact"]) if c["preact"] else s["out"]
    if op == "linear_back":
        q.nf4_linear(s["layer"], c["rows"], c["cols"], s["fmt"], s["x"], s["out"], s["ws"], backward=True,
                     lora=(s["u"], s["v"]), p=c["p"], rng=s["rng"] if c["p"] else None, residual=s.get("residual"))
        return s["out"]
    if op == "act_grad":
        q.nf4_act_grad(s["dy"], s["z"], getattr(q, "NF4_ACT_" + c["act"].upper()), s["dz"], dbias=s.get("dbias"),
                       ws=s["ws"])
        return (s["dz"], s["dbias"]) if c["bias"] else s["dz"]
    if op == "project":
        q.nf4_lora_project(s["x"], s["w"], s["h"], scale=2.0, backward=c["back"], p=c["p"],
                           rng=s["rng"] if c["p"] else None)
        return s["h"]
    q.nf4_lora_grad(s["u"], s["x"], s["grad"], s["ws"], side=c["side"], p=c["p"], rng=s["rng"] if c["p"] else None)
    return s["grad"]


# ---- plain forms ----------------------------------------------------------


def _threshold(p):
    return int(round(p * 65536))


def _keep(n, thr, rng):
    """Truth values of n elements in flat order. 32-bit words held in int64: the low and the (masked) high half of
    a wrapped 64-bit product are the unsigned product's."""
    mask = 0xffffffff
    g = torch.arange((n + 7) // 8, dtype=torch.int64, device=rng.device)
    seed, off = rng[0], rng[1]
    c0, c1 = g & mask, g >> 32
    c2, c3 = (off & mask).expand_as(g), ((off >> 32) & mask).expand_as(g)
    k0, k1 = seed & mask, (seed >> 32) & mask
    for _ in range(7):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & mask) ^ c1 ^ k0, p1 & mask, ((p0 >> 32) & mask) ^ c3 ^ k1, p0 & mask
        k0, k1 = (k0 + 0x9E3779B9) & mask, (k1 + 0xBB67AE85) & mask
    lanes = torch.stack([h for c in (c0, c1, c2, c3) for h in (c & 0xffff, c >> 16)], 1)
    return (lanes >= thr).reshape(-1)[:n]


def _dropped(x32, p, rng):
    thr = _threshold(p)
    if thr == 0:
        return x32
    keep = _keep(x32.numel(), thr, rng).view(x32.shape)
    return torch.where(keep, x32 * (65536.0 / (65536 - thr)), torch.zeros((), device=x32.device))


def _dense(s):
    """The weight as the format defines it: level times constant in fp32, rounded to the 16-bit type."""
    c = s["case"]
    lv = torch.from_numpy(LEVELS).to(s["codes"].device)
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], 1).reshape(-1, 64)
    if c["dq"]:
        q = s["qabsmax"].float()
        a = (q.view(s["scale2"].numel(), -1) * s["scale2"][:, None]).reshape(-1)
    else:
        a = s["absmax"]
    return (lv[codes.int()] * a[:, None]).to(TORCH[c["dtype"]]).float().view(c["rows"], c["cols"])


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros((), device=z.device))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    sg = 1 / (1 + torch.exp(-k * (z + 0.044715 * z * z * z)))
    return sg + z * sg * (1 - sg) * k * (1 + 3 * 0.044715 * z * z)


def _run_plain(s):
    c = s["case"]
    op, t16 = c["op"], TORCH[c["dtype"]]
    if op == "dropout":
        return _dropped(s["x"].float(), c["p"], s["rng"]).to(t16)
    if op == "linear":
        z = s["x"].float() @ _dense(s).t()
        if c["rank"]:
            z = z + s["u"].float() @ s["v"].float().t()
        if c["bias"]:
            z = z + s["bias"].float()
        out = _act(z, c["act"])
        if c["residual"]:
            out = out + s["residual"].float()
        return (out.to(t16), z.to(t16)) if c["preact"] else out.to(t16)
    if op == "linear_back":
        out = s["x"].float() @ _dense(s) + _dropped(s["u"].float() @ s["v"].float(), c["p"], s["rng"])
        if c["residual"]:
            out = out + s["residual"].float()
        return out.to(t16)
    if op == "act_grad":
        dz = s["dy"].float() * _act_slope(s["z"].float(), c["act"])
        return (dz.to(t16), dz.sum(0)) if c["bias"] else dz.to(t16)
    x = s["x"].float()
    if op == "project":
        w = s["w"].float() if c["back"] else s["w"].float().t()
        return (2.0 * (_dropped(x, c["p"], s["rng"]) @ w)).to(t16)
    if c["side"] == "A":
        return s["u"].float().t() @ _dropped(x, c["p"], s["rng"])
    return x.t() @ s["u"].float()


# ---- work and 64-bit values -----------------------------------------------


def work(case):
    op = case["op"]
    if op == "dropout":
        n = case["m"] * case["n"]
        return {"bytes": 4 * n + 16, "flops": n}
    if op in ("linear", "linear_back"):
        m, rows, cols, r = case["m"], case["rows"], case["cols"], case["rank"]
        nout = cols if op == "linear_back" else rows
        nb = rows * cols // 64
        b = rows * cols // 2 + (nb + 4 * -(-nb // 256) if case["dq"] else 4 * nb) + 2 * m * (rows + cols)
        b += 2 * r * (m + nout) + 2 * m * nout * (int(case["residual"]) + int(case.get("preact", False)))
        b += 2 * rows * int(case.get("bias", False))
        return {"bytes": b, "flops": 2 * m * rows * cols + 2 * m * nout * r}
    if op == "act_grad":
        return {"bytes": 6 * case["m"] * case["n"] + 4 * case["n"] * int(case["bias"]),
                "flops": 8 * case["m"] * case["n"]}
    if op == "project":
        m, k, r = case["m"], case["k"], case["rank"]
        return {"bytes": 2 * (m * k + k * r + m * r), "flops": 2 * m * k * r}
    m, n, r = case["m"], case["n"], case["rank"]
    return {"bytes": 2 * m * (n + r) + 4 * n * r, "flops": 2 * m * n * r}


def _mask64(count, p, state):
    """The kept elements' factor in flat order, 0 where dropped; numpy's unsigned words, by the groups' index."""
    thr = int(round(p * 65536))
    if thr == 0:
        return None
    u = np.uint64
    seed, off = (int(v) for v in state)
    out = np.empty(((count + 7) // 8, 8), bool)
    half, full = u(32), u(0xffffffff)
    for at in range(0, out.shape[0], 1 << 20):
        idx = np.arange(at, min(at + (1 << 20), out.shape[0]), dtype=u)
        a, b = idx & full, idx >> half
        c, d = np.full_like(idx, off & 0xffffffff), np.full_like(idx, off >> 32)
        key = [seed & 0xffffffff, seed >> 32]
        for _ in range(7):
            lo, hi = a * u(0xD2511F53), c * u(0xCD9E8D57)
            a, b, c, d = (hi >> half) ^ b ^ u(key[0]), hi & full, (lo >> half) ^ d ^ u(key[1]), lo & full
            key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
        words = np.stack([a, b, c, d], 1).astype(np.uint32)
        out[at:at + idx.size] = words.view(np.uint16).reshape(-1, 8) >= thr
    return torch.from_numpy(out.reshape(-1)[:count]).to(DEV).double() * (65536 / (65536 - thr))


def _times64(x, state, p):
    f = _mask64(x.numel(), p, state)
    return x if f is None else torch.where(f.view(x.shape) > 0, x * f.view(x.shape), torch.zeros_like(x))


def _product64(a, b):
    """a @ b in 64 bits, by blocks of rows."""
    return torch.cat([a[i:i + 512] @ b for i in range(0, a.shape[0], 512)])


def _weight64(s):
    c = s["case"]
    byte = s["codes"].to(torch.int64)
    table = torch.tensor(LEVELS.tolist(), dtype=torch.float64, device=byte.device)
    w = torch.empty(c["rows"] * c["cols"], dtype=torch.float64, device=byte.device)
    w[0::2], w[1::2] = table[byte % 16], table[byte // 16]
    blocks = w.numel() // 64
    if c["dq"]:
        at = torch.arange(blocks, device=byte.device) // 256
        const = (s["qabsmax"].double() * s["scale2"].double()[at]).float().double()
    else:
        const = s["absmax"].double()
    w.view(blocks, 64).mul_(const[:, None])
    # the format's two roundings: to fp32, then to the 16-bit type
    return w.float().to(TORCH[c["dtype"]]).double().view(c["rows"], c["cols"])


def _sigmoid64(t):
    return torch.special.expit(t)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    state = s["rng"].cpu().tolist()
    if op == "dropout":
        return _times64(s["x"].double(), state, c["p"])
    if op == "linear":
        z = _product64(s["x"].double(), _weight64(s).t().contiguous())
        if c["rank"]:
            z += _product64(s["u"].double(), s["v"].double().t().contiguous())
        if c["bias"]:
            z += s["bias"].double()
        if c["act"] == "relu":
            out = z.clamp(min=0)
        elif c["act"] == "silu":
            out = z * _sigmoid64(z)
        elif c["act"] == "gelu":
            out = z * torch.special.ndtr(z)
        elif c["act"] == "gelu_tanh":
            out = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        else:
            out = z.clone()
        if c["residual"]:
            out += s["residual"].double()
        return (out, z) if c["preact"] else out
    if op == "linear_back":
        out = _times64(_product64(s["u"].double(), s["v"].double()), state, c["p"])
        out += _product64(s["x"].double(), _weight64(s))
        if c["residual"]:
            out += s["residual"].double()
        return out
    if op == "act_grad":
        z = s["z"].double()
        if c["act"] == "relu":
            d = torch.where(z > 0, 1.0, 0.0).double()
        elif c["act"] == "silu":
            d = _sigmoid64(z) + z * _sigmoid64(z) * _sigmoid64(-z)
        elif c["act"] == "gelu":
            d = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        else:
            t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            d = 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
        d *= s["dy"].double()
        return (d, d.sum(0)) if c["bias"] else d
    x = s["x"].double()
    if op == "project":
        w = s["w"].double() if c["back"] else s["w"].double().t().contiguous()
        return 2 * _product64(_times64(x, state, c["p"]), w)
    if c["side"] == "A":
        return s["u"].double().t().contiguous() @ _times64(x, state, c["p"])
    return x.t().contiguous() @ s["u"].double()

"""Measured cases of the block-scaled FP8 operators: the quantizer, the matrix product, the linear layer
(training step and serving forward) and the mixture-of-experts layer for a few tokens.

FP8 here carries one fp32 scale for each block of 128 along the contraction: 1 x 128 for activations and
gradients, 128 x 128 for weights.  A block of x has s = max(max|x| / FP8_MAX, 1e-12) and the bytes
q = rn_fp8(x * (1 / s)); a product sums (sum over 128 of a * b) * sa * sb over the blocks in fp32.

``run`` gives the plain form (elementary torch operations in fp32) or, where ``own`` is true, the
library's entry points.  ``exact`` is the same definition in 64 bits; the quantizer's three fp32 roundings
(the scale, its reciprocal, the product) belong to its definition, so they are made there too.
"""

import math

import torch

own = False

DEV = "cuda"
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8_DTYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}

# What a case costs at most: multiply-adds of a product, elements of a quantize, weight bytes of the
# experts (the largest listed cases).
MOST_MACS = 8192 ** 3
MOST_ELEMENTS = 8192 * 8192
MOST_EXPERT_BYTES = 64 * 3 * 2048 * 1024


# ------------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # a training linear's activations: rows for the forward, columns for the weight gradient, one read
        dict(name="quantize rows and columns", op="quantize", mode="both", rows=2048, cols=4096, fmt="e4m3", dtype="bf16"),
        # a large weight of a checkpoint, 128 x 128 blocks
        dict(name="quantize weight", op="quantize", mode="block", rows=8192, cols=8192, fmt="e4m3", dtype="bf16"),
        # one token through a 1024 -> 4096 projection: latency
        dict(name="product one token", op="product", form="forward", batch=1, m=1, n=4096, k=1024, bias=True),
        # 64 sequences decoding through a wide projection
        dict(name="product 64 rows", op="product", form="forward", batch=1, m=64, n=8192, k=2048, bias=False),
        # many small equal products
        dict(name="product batch", op="product", form="forward", batch=64, m=512, n=512, k=512, bias=False),
        # a weight gradient over an odd number of tokens: scales of both sides run along the tokens
        dict(name="product weight gradient", op="product", form="dw", batch=1, m=1040, n=4112, k=2001, bias=False),
        # the largest square of the benchmark
        dict(name="product 8192", op="product", form="forward", batch=1, m=8192, n=8192, k=8192, bias=False),
        # training step of the 1024 -> 4096 linear at 4 x 512 tokens: forward, grad_x, grad_w, grad_b
        dict(name="linear training", op="linear", train=True, m=2048, k=1024, n=4096, fmt_g="e5m2"),
        # serving forward of the 4096 -> 1024 linear for 8 tokens, weight already FP8
        dict(name="linear 8 tokens", op="linear", train=False, m=8, k=4096, n=1024, fmt_g="e4m3"),
        # one token, two of eight experts of 1024 -> 4096
        dict(name="experts one token", op="experts", tokens=1, topk=2, experts=8, hidden=1024, inter=4096),
        # 16 tokens over many small experts
        dict(name="experts 16 tokens", op="experts", tokens=16, topk=8, experts=64, hidden=2048, inter=1024),
        # 61 tokens, an inner size that is no multiple of 128
        dict(name="experts ragged", op="experts", tokens=61, topk=4, experts=16, hidden=4096, inter=1360),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log16(rng, lo, hi):
    return 16 * max(1, _log(rng, lo / 16.0, hi / 16.0))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "linear", "experts"])
    if op == "quantize":
        mode = rng.choice(["rows", "columns", "both", "block"])
        while True:
            rows, cols = _log(rng, 1, 16384), _log(rng, 16, 16384)
            if rows * cols <= MOST_ELEMENTS:
                break
        if rng.random() < 0.6:
            cols = max(16, cols // 16 * 16)
        return dict(op=op, mode=mode, rows=rows, cols=cols, fmt=rng.choice(["e4m3", "e5m2"]),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "product":
        form = rng.choice(["forward", "forward", "dx", "dw"])
        while True:
            batch = 1 if rng.random() < 0.7 else rng.randint(2, 32)
            m, n, k = _log(rng, 1, 8192), _log16(rng, 64, 8192), _log16(rng, 64, 8192)
            if form == "dw":  # stored with the tokens as rows: any number of tokens, 16-byte rows
                m, k = max(16, m // 16 * 16), max(1, k - rng.randint(0, 15))
            if batch * m * n * k <= MOST_MACS / 4:
                break
        return dict(op=op, form=form, batch=batch, m=m, n=n, k=k, bias=form == "forward" and rng.random() < 0.5)
    if op == "linear":
        train = rng.random() < 0.6
        while True:
            m = _log(rng, 64, 8192) if train else _log(rng, 1, 512)
            k, n = _log16(rng, 256, 8192), _log16(rng, 256, 8192)
            if m * n * k <= MOST_MACS / 4:
                break
        return dict(op=op, train=train, m=m, k=k, n=n, fmt_g=rng.choice(["e4m3", "e5m2"]))
    while True:
        experts = _log(rng, 4, 128)
        hidden, inter = _log16(rng, 256, 4096), _log16(rng, 256, 4096)
        if 3 * experts * hidden * inter <= MOST_EXPERT_BYTES:
            break
    return dict(op=op, tokens=_log(rng, 1, 64), topk=rng.randint(1, min(8, experts)), experts=experts, hidden=hidden,
                inter=inter)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(gen, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _activations(gen, shape, std=1.0, dtype=torch.bfloat16):
    """Rows of different size with a few outlying channels, as activations have."""
    t = torch.randn(shape, generator=gen, device=DEV) * std
    t *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device=DEV))
    t *= torch.where(torch.rand(shape[-1:], generator=gen, device=DEV) < 0.01, 16.0, 1.0)
    return t.to(dtype)


def _blocks(n):
    return (n + 127) // 128


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[case["dtype"]]
        r, c = case["rows"], case["cols"]
        s["x"] = _randn(gen, (r, c), 0.02, dt) if case["mode"] == "block" else _activations(gen, (r, c), 1.0, dt)
        s["q"], s["s"] = [], []
        if case["mode"] in ("rows", "both"):
            s["q"].append(torch.empty(r, c, dtype=torch.uint8, device=DEV))
            s["s"].append(torch.empty(_blocks(c), r, device=DEV))
        if case["mode"] in ("columns", "both"):
            s["q"].append(torch.empty(r, c, dtype=torch.uint8, device=DEV))
            s["s"].append(torch.empty(_blocks(r), c, device=DEV))
        if case["mode"] == "block":
            s["q"].append(torch.empty(r, c, dtype=torch.uint8, device=DEV))
            s["s"].append(torch.empty(_blocks(r), _blocks(c), device=DEV))
    elif op == "product":
        b, m, n, k, form = case["batch"], case["m"], case["n"], case["k"], case["form"]
        if form == "forward":    # x [m][k] . w [n][k]^T
            a, w = _activations(gen, (b, m, k)), _randn(gen, (b, n, k), 0.02)
            s["a"], s["sa"] = _quantize(a, "e4m3", "rows")
            s["b"], s["sb"] = _quantize(w, "e4m3", "block")
        elif form == "dx":       # g [m][k] . w [k][n]
            a, w = _activations(gen, (b, m, k), 1e-3), _randn(gen, (b, k, n), 0.02)
            s["a"], s["sa"] = _quantize(a, "e5m2", "rows")
            s["b"], s["sb"] = _quantize(w, "e4m3", "block")
        else:                    # g [k][m]^T . x [k][n]: k tokens
            a, w = _activations(gen, (b, k, m), 1e-3), _activations(gen, (b, k, n))
            s["a"], s["sa"] = _quantize(a, "e5m2", "columns")
            s["b"], s["sb"] = _quantize(w, "e4m3", "columns")
        s["bias"] = _randn(gen, (n,), 0.1) if case["bias"] else None
        s["out"] = torch.empty(b, m, n, dtype=torch.bfloat16, device=DEV)
    elif op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _activations(gen, (m, k))
        w = _randn(gen, (n, k), 0.02)
        s["bias"] = _randn(gen, (n,), 0.1)
        s["y"] = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
        if case["train"]:
            s["w"] = w
            s["g"] = _activations(gen, (m, n), 1e-3)
            s["w8"] = torch.empty(n, k, dtype=torch.uint8, device=DEV)
            s["sw"] = torch.empty(_blocks(n), _blocks(k), device=DEV)
            s["x8c"] = torch.empty(m, k, dtype=torch.uint8, device=DEV)
            s["sxc"] = torch.empty(_blocks(m), k, device=DEV)
            s["gx"], s["gw"], s["gb"] = torch.empty_like(s["x"]), torch.empty_like(w), torch.empty_like(s["bias"])
        else:
            s["w8"], s["sw"] = _quantize(w, "e4m3", "block")
    else:
        t, kk, e, h, i = (case[x] for x in ("tokens", "topk", "experts", "hidden", "inter"))
        s["x"] = _activations(gen, (t, h))
        scores = torch.randn(t, e, generator=gen, device=DEV)
        top = scores.softmax(-1).topk(kk, -1)
        s["ids"] = top.indices.to(torch.int32)
        s["weights"] = top.values / top.values.sum(-1, keepdim=True)
        parts, scales = [], []
        for _ in range(e):  # gate and up each have their own blocks
            g, sg = _quantize(_randn(gen, (2, i, h), 0.02), "e4m3", "block")
            parts.append(g)
            scales.append(sg)
        s["w13"], s["s13"] = torch.stack(parts), torch.stack(scales)
        parts, scales = [], []
        for _ in range(e):
            g, sg = _quantize(_randn(gen, (h, i), 0.02), "e4m3", "block")
            parts.append(g)
            scales.append(sg)
        s["w2"], s["s2"] = torch.stack(parts), torch.stack(scales)
        s["out"] = torch.empty(t, h, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------
# plain form
# ------------------------------------------------------------------------------------------------
def _pad(x, r, c):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % c, 0, -x.shape[-2] % r))


def _quantize(x, fmt, mode):
    """Codes (uint8) and scales of x [..][rows][cols]; scales in the library's layouts."""
    top = FP8_MAX[fmt]
    br, bc = {"rows": (1, 128), "columns": (128, 1), "block": (128, 128)}[mode]
    rows, cols = x.shape[-2:]
    p = _pad(x.float(), br, bc)
    lead = p.shape[:-2]
    t = p.view(*lead, p.shape[-2] // br, br, p.shape[-1] // bc, bc)
    # in 64 bits and rounded once: the correctly rounded fp32 quotient and reciprocal
    s = (t.abs().amax((-3, -1)).double() / top).float().clamp_min(1e-12)
    inv = (1.0 / s.double()).float()[..., :, None, :, None]
    q = (t * inv).clamp(-top, top).view(p.shape)[..., :rows, :cols].contiguous().to(FP8_DTYPE[fmt])
    if mode == "rows":
        s = s.transpose(-1, -2)  # [blocks of cols][rows]
    return q.view(torch.uint8), s.contiguous()


def _value(q, fmt):
    return q.view(FP8_DTYPE[fmt]).float()


def _decode(q, s, fmt, mode):
    """fp32 values of codes [..][rows][cols] with their scales."""
    rows, cols = q.shape[-2:]
    v = _value(q, fmt)
    if mode == "rows":
        s = s.transpose(-1, -2).repeat_interleave(128, -1)[..., :cols]
    elif mode == "columns":
        s = s.repeat_interleave(128, -2)[..., :rows, :]
    else:
        s = s.repeat_interleave(128, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]
    return v * s


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        out = []
        modes = {"both": ("rows", "columns")}.get(s["mode"], (s["mode"],))
        for mode in modes:
            q, sc = _quantize(s["x"], s["fmt"], mode)
            out += [q.view(FP8_DTYPE[s["fmt"]]), sc]
        return out
    if op == "product":
        if s["form"] == "forward":
            y = _decode(s["a"], s["sa"], "e4m3", "rows") @ _decode(s["b"], s["sb"], "e4m3", "block").transpose(-1, -2)
        elif s["form"] == "dx":
            y = _decode(s["a"], s["sa"], "e5m2", "rows") @ _decode(s["b"], s["sb"], "e4m3", "block")
        else:
            y = _decode(s["a"], s["sa"], "e5m2", "columns").transpose(-1, -2) @ _decode(s["b"], s["sb"], "e4m3", "columns")
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return y.to(torch.bfloat16)
    if op == "linear":
        x = _decode(*_quantize(s["x"], "e4m3", "rows"), "e4m3", "rows")
        w8, sw = _quantize(s["w"], "e4m3", "block") if s["train"] else (s["w8"], s["sw"])
        w = _decode(w8, sw, "e4m3", "block")
        y = (x @ w.t() + s["bias"].float()).to(torch.bfloat16)
        if not s["train"]:
            return y
        g = _decode(*_quantize(s["g"], s["fmt_g"], "rows"), s["fmt_g"], "rows")
        gx = (g @ w).to(torch.bfloat16)
        gc = _decode(*_quantize(s["g"], s["fmt_g"], "columns"), s["fmt_g"], "columns")
        xc = _decode(*_quantize(s["x"], "e4m3", "columns"), "e4m3", "columns")
        gw = (gc.t() @ xc).to(torch.bfloat16)
        gb = s["g"].float().sum(0).to(torch.bfloat16)
        return y, gx, gw, gb
    # experts: the pairs' weights are gathered and every pair's products taken
    t, kk = s["ids"].shape
    x = _decode(*_quantize(s["x"], "e4m3", "rows"), "e4m3", "rows")
    out = torch.zeros(t, s["hidden"], device=DEV)
    for j in range(kk):  # one expert of each token at a time: bounded memory
        for t0 in range(0, t, 8):
            e = s["ids"][t0:t0 + 8, j].long()
            w13 = _decode(s["w13"][e], s["s13"][e], "e4m3", "block")     # [tokens][2][inter][hidden]
            u = torch.einsum("tcih,th->tci", w13, x[t0:t0 + 8])
            h = u[:, 0] / (1.0 + torch.exp(-u[:, 0])) * u[:, 1]
            h = _decode(*_quantize(h, "e4m3", "rows"), "e4m3", "rows")
            w2 = _decode(s["w2"][e], s["s2"][e], "e4m3", "block")
            out[t0:t0 + 8] += s["weights"][t0:t0 + 8, j, None] * torch.einsum("thi,ti->th", w2, h)
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------
# the library
# ------------------------------------------------------------------------------------------------
def _workspace(s, key, nbytes):
    if key not in s:
        s[key] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=DEV)
    return s[key]


def _run_own(s):
    import fp8_delayed_scaling_amax_b200 as F
    fmts = {"e4m3": F.FP8_E4M3, "e5m2": F.FP8_E5M2}
    op = s["op"]
    if op == "quantize":
        it = {torch.bfloat16: F.FP8_IN_BF16, torch.float16: F.FP8_IN_F16, torch.float32: F.FP8_IN_F32}[s["x"].dtype]
        r, c, fmt, q, sc = s["rows"], s["cols"], fmts[s["fmt"]], s["q"], s["s"]
        if s["mode"] == "block":
            F.fp8_quantize_block128(s["x"], it, r, c, fmt, q[0], sc[0])
        elif s["mode"] == "rows":
            F.fp8_quantize_block(s["x"], it, r, c, fmt, q[0], sc[0], None, None)
        elif s["mode"] == "columns":
            F.fp8_quantize_block(s["x"], it, r, c, fmt, None, None, q[0], sc[0])
        else:
            F.fp8_quantize_block(s["x"], it, r, c, fmt, q[0], sc[0], q[1], sc[1])
        out = []
        for a, b in zip(q, sc):
            out += [a.view(FP8_DTYPE[s["fmt"]]), b]
        return out
    if op == "product":
        b, m, n, k, form = s["batch"], s["m"], s["n"], s["k"], s["form"]
        sa, sb = s["sa"], s["sb"]
        if form == "forward":
            F.fp8_gemm_block(s["a"], s["b"], F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, k, k, n, b, m * k, n * k,
                             m * n, F.BlockScale(sa, 1, 1, m, sa[0].numel()),
                             F.BlockScale(sb, 128, _blocks(k), 1, sb[0].numel()), s["bias"], s["out"])
        elif form == "dx":
            F.fp8_gemm_block(s["a"], s["b"], F.FP8_E5M2, F.FP8_E4M3, F.FP8_LAYOUT_NN, m, n, k, k, n, n, b, m * k, n * k,
                             m * n, F.BlockScale(sa, 1, 1, m, sa[0].numel()),
                             F.BlockScale(sb, 128, 1, _blocks(n), sb[0].numel()), s["bias"], s["out"])
        else:
            F.fp8_gemm_block(s["a"], s["b"], F.FP8_E5M2, F.FP8_E4M3, F.FP8_LAYOUT_TN, m, n, k, m, n, n, b, m * k, n * k,
                             m * n, F.BlockScale(sa, 1, 1, m, sa[0].numel()),
                             F.BlockScale(sb, 1, 1, n, sb[0].numel()), s["bias"], s["out"])
        return s["out"]
    if op == "linear":
        m, k, n = s["m"], s["k"], s["n"]
        nf = F.linear_forward_fp8_block_workspace_size(m, k, n)
        wf = _workspace(s, "wf", nf)
        if not s["train"]:
            F.linear_forward_fp8_block(s["x"], s["w8"], 1, s["sw"], s["bias"], m, k, n, F.FP8_E4M3, None, None, None,
                                       None, wf, nf, s["y"])
            return s["y"]
        F.linear_forward_fp8_block(s["x"], s["w"], 0, None, s["bias"], m, k, n, F.FP8_E4M3, s["w8"], s["sw"], s["x8c"],
                                   s["sxc"], wf, nf, s["y"])
        nb = F.linear_backward_fp8_block_workspace_size(m, k, n)
        wb = _workspace(s, "wb", nb)
        F.linear_backward_fp8_block(s["g"], s["x8c"], s["sxc"], s["w8"], s["sw"], m, k, n, fmts[s["fmt_g"]], F.FP8_E4M3,
                                    1, 1, 1, wb, nb, s["gx"], s["gw"], s["gb"])
        return s["y"], s["gx"], s["gw"], s["gb"]
    t, kk, e, h, i = (s[x] for x in ("tokens", "topk", "experts", "hidden", "inter"))
    nm = F.moe_forward_fp8_block_workspace_size(t, kk, e, h, i)
    wm = _workspace(s, "wm", nm)
    F.moe_forward_fp8_block(s["x"], s["ids"], s["weights"], t, kk, e, h, i, F.FP8_E4M3, s["w13"], s["s13"], s["w2"],
                            s["s2"], wm, nm, s["out"])
    return s["out"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        size = 4 if case["dtype"] == "f32" else 2
        nb = r * c * size
        if case["mode"] in ("rows", "both"):
            nb += r * c + 4 * r * _blocks(c)
        if case["mode"] in ("columns", "both"):
            nb += r * c + 4 * c * _blocks(r)
        if case["mode"] == "block":
            nb += r * c + 4 * _blocks(r) * _blocks(c)
        return {"bytes": nb, "flops": 0}
    if op == "product":
        b, m, n, k = case["batch"], case["m"], case["n"], case["k"]
        return {"bytes": b * (m * k + n * k + 2 * m * n), "flops": 2 * b * m * n * k}
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        if not case["train"]:
            return {"bytes": 2 * m * k + n * k + 2 * m * n + 2 * n, "flops": 2 * m * n * k}
        # x, w, bias and g in; y and the gradients out; what the forward leaves for the backward written and read
        return {"bytes": 2 * (m * k + n * k + n + m * n) + 2 * (m * n + m * k + n * k + n) + 2 * (m * k + n * k),
                "flops": 6 * m * n * k}
    t, kk, e, h, i = (case[x] for x in ("tokens", "topk", "experts", "hidden", "inter"))
    active = e * (1.0 - (1.0 - kk / e) ** t)  # experts that are asked for, on average
    return {"bytes": active * 3 * h * i + 4 * t * h, "flops": 6 * t * kk * h * i}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _r32(v):
    return v.float().double()


def _round_fp8(v, fmt):
    """Nearest FP8 value (ties to even) of float64 v, saturating."""
    mant, low, top = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    e = torch.frexp(v)[1].double() - 1.0
    step = torch.exp2(e.clamp_min(low) - mant)
    return (torch.round(v / step) * step).clamp(-top, top)


def _q64(x, fmt, axis):
    """(values of the codes, scales broadcast to x's shape, scales) of blocks of 128 along `axis` of the last
    two dimensions, or of both where axis is None."""
    d = x.double()
    rows, cols = d.shape[-2:]
    br = 128 if axis in (None, -2) else 1
    bc = 128 if axis in (None, -1) else 1
    nr, nc = -(-rows // br), -(-cols // bc)
    big = torch.zeros(*d.shape[:-2], nr * br, nc * bc, dtype=torch.float64, device=d.device)
    big[..., :rows, :cols] = d.abs()
    amax = big.unflatten(-2, (nr, br)).amax(-2).unflatten(-1, (nc, bc)).amax(-1)
    s = torch.maximum(_r32(amax / FP8_MAX[fmt]), _r32(torch.tensor(1e-12, dtype=torch.float64, device=d.device)))
    at_r = torch.arange(rows, device=d.device) // br
    at_c = torch.arange(cols, device=d.device) // bc
    full = s[..., at_r, :][..., at_c]
    return _round_fp8(_r32(d * _r32(1.0 / full)), fmt), full, s


def _v64(q, s, fmt, axis):
    """float64 values of stored codes and scales (in the layouts that prepare keeps)."""
    v = q.view(FP8_DTYPE[fmt]).double()
    rows, cols = v.shape[-2:]
    at_r, at_c = torch.arange(rows, device=v.device), torch.arange(cols, device=v.device)
    s = s.double()
    if axis == -1:
        return v * s[..., at_c // 128, :].transpose(-1, -2)
    if axis == -2:
        return v * s[..., at_r // 128, :]
    return v * s[..., at_r // 128, :][..., at_c // 128]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        out = []
        for mode in {"both": ("rows", "columns")}.get(case["mode"], (case["mode"],)):
            v, _, sc = _q64(s["x"], case["fmt"], {"rows": -1, "columns": -2, "block": None}[mode])
            out += [v, sc.transpose(-1, -2).contiguous() if mode == "rows" else sc]
        return out
    if op == "product":
        if case["form"] == "forward":
            y = _v64(s["a"], s["sa"], "e4m3", -1) @ _v64(s["b"], s["sb"], "e4m3", None).transpose(-1, -2)
        elif case["form"] == "dx":
            y = _v64(s["a"], s["sa"], "e5m2", -1) @ _v64(s["b"], s["sb"], "e4m3", None)
        else:
            y = _v64(s["a"], s["sa"], "e5m2", -2).transpose(-1, -2) @ _v64(s["b"], s["sb"], "e4m3", -2)
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "linear":
        q, f, _ = _q64(s["x"], "e4m3", -1)
        if case["train"]:
            wq, wf, _ = _q64(s["w"], "e4m3", None)
            w = wq * wf
        else:
            w = _v64(s["w8"], s["sw"], "e4m3", None)
        y = (q * f) @ w.t() + s["bias"].double()
        if not case["train"]:
            return y
        gq, gf, _ = _q64(s["g"], case["fmt_g"], -1)
        hq, hf, _ = _q64(s["g"], case["fmt_g"], -2)
        xq, xf, _ = _q64(s["x"], "e4m3", -2)
        return y, (gq * gf) @ w, (hq * hf).t() @ (xq * xf), s["g"].double().sum(0)
    q, f, _ = _q64(s["x"], "e4m3", -1)
    x = q * f
    out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        w13 = _v64(s["w13"][e], s["s13"][e], "e4m3", None)
        gate, up = x[t] @ w13[0].t(), x[t] @ w13[1].t()
        hq, hf, _ = _q64(gate / (1.0 + torch.exp(-gate)) * up, "e4m3", -1)
        y = (hq * hf) @ _v64(s["w2"][e], s["s2"][e], "e4m3", None).t()
        out.index_add_(0, t, s["weights"][t, j].double()[:, None] * y)
    return out

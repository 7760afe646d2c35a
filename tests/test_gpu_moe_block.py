"""GPU parity: moe_forward_fp8_block (a mixture-of-experts layer for a few tokens) against fp64.

The hidden activation h is quantized inside: the oracle forms h in fp64, the kernel in fp32, so a value that
lies next to a rounding border of FP8 may take the neighbouring code.  With u = 2^-24, k products per sum and
S = sum |terms|, the kernel's g and u are within (2^-21 + (nb + 9) 2^-24) S of the oracle's (the product's
bound, ``oracle/block.py``), which moves h by dh; a code whose unrounded value is further than dh / s from
every border must be equal, the others may differ by one step of FP8.  The output's tolerance adds, per
value, |weight| * sum |w2| * (step of those codes) to the product's bound."""

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F
from oracle import block as OB
from oracle import fp8_codec as C
from helpers import in_values_f32, bf16_out_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _weights(rng, experts, hidden, inter, fmt):
    def one(r, c, std):
        codes, s = OB.quantize((rng.standard_normal((r, c)) * std).astype(np.float32), fmt, "square")
        return codes, s, OB.values(codes, s, fmt, "square")
    g = [[one(inter, hidden, hidden ** -0.5) for _ in range(2)] for _ in range(experts)]
    d = [one(hidden, inter, inter ** -0.5) for _ in range(experts)]
    w13 = np.stack([np.stack([h[0] for h in e]) for e in g])
    s13 = np.stack([np.stack([h[1] for h in e]) for e in g]).astype(np.float32)
    w2 = np.stack([e[0] for e in d])
    s2 = np.stack([e[1] for e in d]).astype(np.float32)
    return (w13, s13, w2, s2), [[h[2] for h in e] for e in g], [e[2] for e in d]


def _oracle(xv, ids, wts, g, d, fmt, experts):
    """(out, tolerance), fp64."""
    tokens, hidden = xv.shape
    top, mant = C.FP8_MAX[fmt], 3 if fmt == "e4m3" else 2
    low = -6 if fmt == "e4m3" else -14
    xq = OB.values(*OB.quantize(xv, fmt, "rows"), fmt, "rows")
    out, tol = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    acc_abs = np.zeros((tokens, hidden))
    nb = OB.blocks(hidden)
    for t in range(tokens):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < experts:
                continue
            gate, up = g[e][0] @ xq[t], g[e][1] @ xq[t]
            e_acc = 2.0 ** -21 + (nb + 9) * 2.0 ** -24
            dg = e_acc * (np.abs(g[e][0]) @ np.abs(xq[t]))
            du = e_acc * (np.abs(g[e][1]) @ np.abs(xq[t]))
            sig = 1.0 / (1.0 + np.exp(-gate))
            h = gate * sig * up
            # |silu'| <= 1.1; exp, the sum, the quotient and the product round within 2^-21 together
            dh = 1.1 * dg * np.abs(up) + np.abs(gate * sig) * du + 2.0 ** -21 * np.abs(h) + 1.1 * dg * du
            hq = np.zeros_like(h)
            slack = np.zeros_like(h)
            for b in range(0, h.size, 128):
                s_ = slice(b, b + 128)
                s = max(np.abs(h[s_]).max() / top, 1e-12)
                ds = np.where(np.abs(h[s_]) == np.abs(h[s_]).max(), dh[s_], 0).max() / top + 2.0 ** -22 * s
                v = h[s_] / s
                step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 1e-30))), low) - mant)
                r = np.clip(np.rint(v / step) * step, -top, top)
                near = np.abs(np.abs(v / step - np.floor(v / step)) - 0.5) * step <= (dh[s_] + np.abs(v) * ds) / s + 2.0 ** -22 * np.abs(v)
                hq[s_] = r * s
                slack[s_] = np.abs(r) * ds + near * step * s
            y = d[e] @ hq
            w = float(np.float32(wts[t, j]))
            out[t] += w * y
            tol[t] += abs(w) * (np.abs(d[e]) @ slack)
            acc_abs[t] += abs(w) * (np.abs(d[e]) @ np.abs(hq))
    n2 = OB.blocks(g[0][0].shape[0])
    tol += (2.0 ** -8 + 2.0 ** -16) * np.abs(out) + (2.0 ** -21 + (n2 + ids.shape[1] + 10) * 2.0 ** -24) * acc_abs
    return out, tol


def run_moe(x, ids, wts, packed, experts, inter, fmt="e4m3", x_shift=0, stream=None):
    tokens, hidden = x.shape
    w13, s13, w2, s2 = (torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in packed)
    nbytes = F.moe_forward_fp8_block_workspace_size(tokens, ids.shape[1], experts, hidden, inter)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
    flat = torch.zeros(x.numel() + 8, dtype=torch.bfloat16)
    flat[x_shift:x_shift + x.numel()] = x.reshape(-1)
    out = torch.full((tokens + 1, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
    args = (flat.to(DEV)[x_shift:], torch.from_numpy(ids.astype(np.int32)).to(DEV),
            torch.from_numpy(wts.astype(np.float32)).to(DEV), tokens, ids.shape[1], experts, hidden, inter,
            F.FP8_E4M3 if fmt == "e4m3" else F.FP8_E5M2, w13, s13, w2, s2, ws, nbytes, out)
    F.moe_forward_fp8_block(*args)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    assert (out[tokens] == 7.0).all()
    return out[:tokens].clone(), args


def check(tokens, topk, experts, hidden, inter, fmt="e4m3", seed=0, ids=None, x_shift=0):
    rng = np.random.default_rng(seed)
    packed, g, d = _weights(rng, experts, hidden, inter, fmt)
    x = torch.from_numpy((rng.standard_normal((tokens, hidden)) * np.exp(rng.standard_normal((tokens, 1)))).astype(np.float32)).to(torch.bfloat16)
    if ids is None:
        ids = np.stack([rng.permutation(experts)[:topk] for _ in range(tokens)])
    wts = rng.random(ids.shape).astype(np.float32)
    got, args = run_moe(x, ids, wts, packed, experts, inter, fmt, x_shift)
    ref, tol = _oracle(in_values_f32(x), ids, wts, g, d, fmt, experts)
    err = np.abs(bf16_out_to_f64(got) - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, worst {float((err / np.maximum(tol, 1e-30)).max())}, first {np.argwhere(bad)[:4].tolist()}"
    return got, args


@pytest.mark.parametrize("tokens,topk,experts,hidden,inter", [
    (1, 1, 1, 16, 16), (1, 2, 8, 256, 384), (1, 8, 16, 1024, 512), (3, 2, 4, 144, 272), (16, 4, 8, 512, 640),
    (17, 3, 5, 272, 144), (64, 2, 3, 384, 256), (33, 8, 40, 256, 128), (64, 6, 64, 128, 256), (5, 2, 4, 2048, 1360),
    (1, 4, 6, 2048, 400), (2, 3, 4, 1280, 2048), (1, 1, 2, 128, 4096)])
def test_moe_matches_fp64(tokens, topk, experts, hidden, inter):
    check(tokens, topk, experts, hidden, inter, seed=tokens + hidden)


@pytest.mark.parametrize("tokens,topk,experts,hidden,inter", [
    (64, 32, 1024, 32, 48), (64, 8, 64, 256, 144), (11, 32, 100, 128, 128), (64, 32, 33, 128, 128), (64, 1, 1000, 64, 128)])
def test_moe_large_tables(tokens, topk, experts, hidden, inter):
    """The most pairs and experts there can be, and pairs that several warps rank in several steps each."""
    check(tokens, topk, experts, hidden, inter, seed=experts)


def test_moe_e5m2_and_unaligned_rows():
    check(4, 2, 4, 256, 256, fmt="e5m2", seed=3)
    check(6, 2, 4, 272, 256, seed=4, x_shift=1)


def test_moe_skipped_slots_and_repeated_experts():
    """Ids outside 0 .. experts - 1 are skipped, a token without a valid slot gives zeros, and an expert
    named many times (by one token, or by more pairs than one run holds) is added each time."""
    ids = np.array([[0, -1], [3, 3], [-1, -1], [7, 1], [2, 2 ** 30]])
    got, _ = check(5, 2, 4, 256, 256, seed=5, ids=ids)
    assert (got[2] == 0).all()
    check(40, 3, 2, 128, 128, seed=6, ids=np.ones((40, 3), dtype=np.int64))
    check(16, 2, 4, 128, 144, seed=7, ids=np.zeros((16, 2), dtype=np.int64))
    none, _ = check(3, 2, 4, 128, 128, seed=8, ids=np.full((3, 2), -1))
    assert (none == 0).all()


def test_moe_repeats_captures_and_other_streams():
    """The same bits again, from a captured graph replayed with new inputs in the same buffers, and from
    two streams at once with a workspace each."""
    got, args = check(9, 4, 8, 512, 384, seed=9)
    out = args[-1]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        F.moe_forward_fp8_block(*args)
    out.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:9], got)
    # new ids in the captured buffers
    ids = args[1].clone()
    args[1].copy_((ids + 1) % 8)
    graph.replay()
    torch.cuda.synchronize()
    replayed = out[:9].clone()
    F.moe_forward_fp8_block(*args)
    torch.cuda.synchronize()
    assert torch.equal(out[:9], replayed) and not torch.equal(replayed, got)
    args[1].copy_(ids)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(out) for _ in streams]
    wss = [torch.zeros_like(args[-3]) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, o, w in zip(streams, outs, wss):
            F.moe_forward_fp8_block(*args[:-3], w, args[-2], o, stream=st)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    for o in outs:
        assert torch.equal(o[:9], got)


def test_moe_without_programmatic_launch():
    got, args = check(7, 3, 8, 384, 256, seed=11)
    F.fp8_set_pdl(False)
    try:
        args[-1].zero_()
        F.moe_forward_fp8_block(*args)
        torch.cuda.synchronize()
    finally:
        F.fp8_set_pdl(True)
    assert torch.equal(args[-1][:7], got)


def test_moe_no_tokens():
    F.moe_forward_fp8_block(None, None, None, 0, 2, 4, 128, 128, F.FP8_E4M3, *(torch.zeros(1 << 17, dtype=torch.uint8, device=DEV),
                            torch.zeros(64, device=DEV)) * 2, None, 0, None)

"""GPU: calls of the block-scaled entries that their description allows and that the other tests do not make: the smallest
sizes, scales with strides of zero, outputs at any element, many batches, a very long contraction, the first call of a process
made inside a capture, calls from several threads."""

import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F
from oracle import block as OB

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _codes(rng, *shape):
    q = rng.integers(0, 256, shape, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x38  # no NaN codes
    return torch.from_numpy(q).to(DEV)


def _scales(rng, *shape):
    return torch.from_numpy(rng.uniform(0.5, 2.0, shape).astype(np.float32)).to(DEV)


def _value(q):
    return q.view(torch.float8_e4m3fn).double().cpu().numpy()


def _check(out, a, b, k):
    """out against a @ b.T, fp64 values with their scales."""
    ref = a @ b.swapaxes(-1, -2)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= OB.tolerance(ref, np.abs(a) @ np.abs(b).swapaxes(-1, -2), k)).all()


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (2, 1, 129), (65, 1, 1), (3, 2, 5), (64, 3, 127), (66, 5, 255), (130, 129, 1),
                                   (17, 127, 2), (1, 1, 1 << 20), (70, 3, 1 << 18)])
def test_smallest_and_longest(m, n, k):
    rng = np.random.default_rng(m + n + k)
    ld, kb = -(-k // 16) * 16, OB.blocks(k)
    a, b = _codes(rng, m, ld), _codes(rng, n, ld)
    if ld > k:
        a[:, k:], b[:, k:] = 0x7F, 0x7F
    sa, sb = _scales(rng, kb, m), _scales(rng, kb, n)
    flat = torch.full((m * n + 3,), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, ld, ld, n, 1, 0, 0, 0, F.BlockScale(sa, 1, 1, m),
                     F.BlockScale(sb, 1, 1, n), None, flat[1:])
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    assert flat[0] == 7.0 and (flat[m * n + 1:] == 7.0).all()
    at = np.arange(k) // 128
    _check(flat[1:m * n + 1].view(m, n), _value(a)[:, :k] * sa.double().cpu().numpy().T[:, at],
           _value(b)[:, :k] * sb.double().cpu().numpy().T[:, at], k)


@pytest.mark.parametrize("layout,m", [("NT", 3), ("NT", 40), ("NT", 200), ("NT", 700), ("TN", 144), ("TN", 720)])
def test_strides_of_zero(layout, m):
    """One scale for all rows, for all blocks, or for both, and one descriptor's scales for every batch."""
    rng = np.random.default_rng(m)
    n, k, batch = 272, 400, 2
    kb, nb = OB.blocks(k), OB.blocks(n)
    mn = layout == "TN"
    a, b = _codes(rng, batch, *((k, m) if mn else (m, k))), _codes(rng, batch, *((k, n) if mn else (n, k)))
    lay, lda, ldb = (F.FP8_LAYOUT_TN, m, n) if mn else (F.FP8_LAYOUT_NT, k, k)

    def run(sa, sb):
        out = torch.full((batch, m, n), 7.0, dtype=torch.bfloat16, device=DEV)
        F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, lay, m, n, k, lda, ldb, n, batch, m * k, n * k, m * n, sa, sb, None, out)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        return out.view(torch.int16)
    rows, per_k, one = _scales(rng, m), _scales(rng, kb), _scales(rng, 1)
    for col in (False, True):
        width = n if col else nb
        cols = _scales(rng, width)
        mk = lambda t, *s: F.BlockScale(t, 1 if col else 128, *s)  # noqa: E731
        want = run(F.BlockScale(rows.repeat(kb, 1).contiguous(), 1, 1, m, 0), mk(cols.repeat(kb, 1).contiguous(), 1, width, 0))
        assert torch.equal(run(F.BlockScale(rows, 1, 1, 0, 0), mk(cols, 1, 0, 0)), want)
        want = run(F.BlockScale(per_k[:, None].repeat(1, m).contiguous(), 1, 1, m, 0),
                   mk(one.repeat(kb, width).contiguous(), 1, width, 0))
        assert torch.equal(run(F.BlockScale(per_k, 1, 0, 1, 0), mk(one, 0, 0, 0)), want)


@pytest.mark.parametrize("m,n,k", [(1, 144, 272), (33, 16, 128), (100, 48, 144)])
def test_many_batches(m, n, k):
    rng = np.random.default_rng(n)
    batch, kb, nb = 1000, OB.blocks(k), OB.blocks(n)
    a, b, sa, sb = _codes(rng, batch, m, k), _codes(rng, batch, n, k), _scales(rng, batch, kb, m), _scales(rng, batch, nb, kb)
    out = torch.full((batch, m, n), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, k, k, n, batch, m * k, n * k, m * n,
                     F.BlockScale(sa, 1, 1, m, kb * m), F.BlockScale(sb, 128, kb, 1, nb * kb), None, out)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    at, row = np.arange(k) // 128, np.arange(n) // 128
    _check(out, _value(a) * sa.double().cpu().numpy().swapaxes(1, 2)[:, :, at], _value(b) * sb.double().cpu().numpy()[:, row][:, :, at], k)


@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_experts_write_rows_at_any_element(tokens):
    """x and out that are only 2-byte aligned, the same expert in all 32 slots, one expert in all."""
    rng = np.random.default_rng(tokens)
    hidden, inter, experts = 144, 272, 3
    w13, w2 = _codes(rng, experts, 2 * inter, hidden), _codes(rng, experts, hidden, inter)
    s13, s2 = _scales(rng, experts, 2, 3, 2) * 2.0 ** -12, _scales(rng, experts, 2, 3) * 2.0 ** -8
    xs = torch.from_numpy(rng.standard_normal(tokens * hidden + 1).astype(np.float32)).to(torch.bfloat16).to(DEV)

    def run(x, ids, wts, shift, e=experts):
        topk = ids.shape[1]
        nbytes = F.moe_forward_fp8_block_workspace_size(tokens, topk, e, hidden, inter)
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.full((tokens * hidden + 4,), 7.0, dtype=torch.bfloat16, device=DEV)
        F.moe_forward_fp8_block(x, ids, wts, tokens, topk, e, hidden, inter, F.FP8_E4M3, w13, s13, w2, s2, ws, nbytes, out[shift:])
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        assert (out[:shift] == 7.0).all() and (out[shift + tokens * hidden:] == 7.0).all()
        return out[shift:shift + tokens * hidden]
    for topk in (1, 5, 32):
        ids = torch.from_numpy(rng.integers(0, experts, (tokens, topk)).astype(np.int32)).to(DEV)
        wts = _scales(rng, tokens, topk)
        want = run(xs[1:].clone(), ids, wts, 0)
        assert torch.isfinite(want).all()
        for shift in (1, 2, 3):
            assert torch.equal(run(xs[1:], ids, wts, shift), want)
    # 32 slots of one expert, each with 1/32 of the weight: the sum of equal terms of powers of two is exact
    one = run(xs[1:], torch.zeros(tokens, 1, dtype=torch.int32, device=DEV), torch.ones(tokens, 1, device=DEV), 0, 1)
    many = run(xs[1:], torch.zeros(tokens, 32, dtype=torch.int32, device=DEV), torch.full((tokens, 32), 1 / 32, device=DEV), 0, 1)
    diff = (one.double() - many.double()).abs()
    # 32 additions of fp32 on either side, then two bf16 roundings
    assert (diff <= 2.0 ** -7 * one.double().abs() + 2.0 ** -18 * one.double().abs().max()).all()


FIRST = """
import torch
import fp8_delayed_scaling_amax_b200 as F
which = {which!r}
d = "cuda"
u8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device=d)
f32 = lambda *s: torch.ones(*s, device=d)
b16 = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device=d)
m, n, k = {sizes}
if which == "product":
    kb = -(-k // 128)
    a, b, out = u8(m, k), u8(n, k), b16(m, n)
    sa, sb = F.BlockScale(f32(kb, m), 1, 1, m), F.BlockScale(f32(-(-n // 128), kb), 128, kb, 1)
    call = lambda: F.fp8_gemm_block(a, b, 0, 0, F.FP8_LAYOUT_NT, m, n, k, k, k, n, 1, 0, 0, 0, sa, sb, None, out)
elif which == "linear":
    x, w, out, g = b16(m, k), b16(n, k), b16(m, n), b16(m, n)
    w8, sw, xc, xs = u8(n, k), f32(-(-n // 128), -(-k // 128)), u8(m, k), f32(-(-m // 128), k)
    nf, nb = F.linear_forward_fp8_block_workspace_size(m, k, n), F.linear_backward_fp8_block_workspace_size(m, k, n)
    wf, wb, gx, gw, gb = u8(nf), u8(nb), b16(m, k), b16(n, k), b16(n)
    def call():
        F.linear_forward_fp8_block(x, w, 0, None, None, m, k, n, 0, w8, sw, xc, xs, wf, nf, out)
        F.linear_backward_fp8_block(g, xc, xs, w8, sw, m, k, n, 1, 0, 1, 1, 1, wb, nb, gx, gw, gb)
else:
    t, hidden, inter = m, n, k
    x, out, ids, wts = b16(t, hidden), b16(t, hidden), torch.zeros(t, 2, dtype=torch.int32, device=d), f32(t, 2)
    hb, ib = -(-hidden // 128), -(-inter // 128)
    w13, w2, s13, s2 = u8(1, 2 * inter, hidden), u8(1, hidden, inter), f32(1, 2, ib, hb), f32(1, hb, ib)
    nb = F.moe_forward_fp8_block_workspace_size(t, 2, 1, hidden, inter)
    ws = u8(nb)
    call = lambda: F.moe_forward_fp8_block(x, ids, wts, t, 2, 1, hidden, inter, 0, w13, s13, w2, s2, ws, nb, out)
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    call()
out.fill_(float("nan"))
graph.replay()
torch.cuda.synchronize()
first = out.clone()
out.fill_(float("nan"))
call()
torch.cuda.synchronize()
assert F.fp8_get_device_status() == 0
assert not first.isnan().any() and torch.equal(first, out)
print("done")
"""


@pytest.mark.parametrize("which,sizes", [("product", (1, 256, 512)), ("product", (50, 256, 512)), ("product", (128, 256, 4096)),
                                         ("product", (1024, 1024, 256)), ("linear", (200, 272, 144)), ("experts", (2, 256, 144)),
                                         ("experts", (20, 256, 144))])
def test_the_first_call_of_a_process_is_captured(which, sizes):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(which=which, sizes=sizes)], capture_output=True, text=True, timeout=300,
                       cwd=root)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


def test_several_threads():
    """Calls from four threads, a stream and buffers each, give what one thread gives."""
    rng = np.random.default_rng(5)
    shapes = [(1, 1024, 1024), (40, 512, 640), (128, 256, 4096), (600, 528, 272)]
    sets = []
    for m, n, k in shapes:
        kb, nb = OB.blocks(k), OB.blocks(n)
        a, b = _codes(rng, m, k), _codes(rng, n, k)
        out = torch.zeros(m, n, dtype=torch.int16, device=DEV)
        args = (a, b, F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, k, k, n, 1, 0, 0, 0, F.BlockScale(_scales(rng, kb, m), 1, 1, m),
                F.BlockScale(_scales(rng, nb, kb), 128, kb, 1), None)
        F.fp8_gemm_block(*args, out)
        torch.cuda.synchronize()
        sets.append((args, out.clone(), out))
    failed = []

    def work(args, want, out):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    out.zero_()
                    F.fp8_gemm_block(*args, out)
            stream.synchronize()
            if not torch.equal(out, want):
                failed.append(args[5:8])
        except Exception as e:  # a thread's exception would be lost
            failed.append(repr(e))
    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and F.fp8_get_device_status() == 0

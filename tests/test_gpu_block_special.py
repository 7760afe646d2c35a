"""GPU: numbers that are none, infinities and the largest finite ones in the block-scaled entries: what they do to the
block, row or token that holds them (``test_gpu_block_edges.py`` holds that the others do not change)."""

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F
from oracle import block as OB
from oracle import fp8_codec as C
from helpers import np_u8, np_f32, in_values_f32, bf16_out_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = {"e4m3": F.FP8_E4M3, "e5m2": F.FP8_E5M2}
IN = {torch.bfloat16: F.FP8_IN_BF16, torch.float16: F.FP8_IN_F16, torch.float32: F.FP8_IN_F32}
NAN, INF = float("nan"), float("inf")


def _special(dtype, rows, cols):
    """Blocks of zeros, of numbers far below the smallest scale, with NaN (alone, in pairs, and nothing else), with
    infinities of either sign, NaN beside them, with the type's largest and smallest finite numbers."""
    fin = torch.finfo(dtype)
    rng = np.random.default_rng(rows + cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).to(dtype)
    x[:, 128:256] = 0.0                       # a block of zeros in every row
    x[0, 0] = NAN
    x[1, 4:12] = NAN                          # whole words and pairs of them
    x[2, :128] = NAN                          # nothing else
    x[3, 5], x[3, 6] = INF, 1.0
    x[4, 7] = -INF
    x[5, 8], x[5, 9] = -INF, NAN
    x[6, 10], x[6, 11] = fin.max, fin.min
    x[7, :128] = fin.min
    x[8, :128] = fin.tiny                     # below 1e-12 for bf16 and fp32
    x[9, 256:] = fin.smallest_normal / 4      # subnormal
    x[10, :128] = -0.0
    x[11, 130] = 1e-7
    x[-1, -1] = -INF
    x[-2, -3] = NAN
    return x


@pytest.mark.parametrize("dtype", list(IN), ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(40, 300), (256, 512), (131, 272)])
def test_quantize_special_values(dtype, fmt, rows, cols):
    """Scales bit for bit; bytes too, where the byte is a number (any NaN code stands for NaN)."""
    x = _special(dtype, rows, cols)
    v, xd = in_values_f32(x), x.to(DEV)
    q = lambda: torch.full((rows, cols), 0x38, dtype=torch.uint8, device=DEV)  # noqa: E731
    s = lambda *shape: torch.full(shape, 3.0, device=DEV)  # noqa: E731
    found = {}
    o, sr, oc, sc = q(), s(OB.blocks(cols), rows), q(), s(OB.blocks(rows), cols)
    F.fp8_quantize_block(xd, IN[dtype], rows, cols, FMT[fmt], o, sr, oc, sc)
    found["rows"], found["columns"] = (o, sr), (oc, sc)
    one, two = (q(), s(OB.blocks(cols), rows)), (q(), s(OB.blocks(rows), cols))
    F.fp8_quantize_block(xd, IN[dtype], rows, cols, FMT[fmt], *one)
    F.fp8_quantize_block(xd, IN[dtype], rows, cols, FMT[fmt], None, None, *two)
    sq = q(), s(OB.blocks(rows), OB.blocks(cols))
    F.fp8_quantize_block128(xd, IN[dtype], rows, cols, FMT[fmt], *sq)
    found["square"] = sq
    torch.cuda.synchronize()
    assert torch.equal(one[0], o) and torch.equal(one[1], sr) and torch.equal(two[0], oc) and torch.equal(two[1], sc)
    for mode, (codes, scales) in found.items():
        with np.errstate(invalid="ignore", over="ignore"):
            want, ws = OB.quantize(v, fmt, mode)
        assert not np.isnan(ws).any()
        assert np.array_equal(np_f32(scales).view(np.uint32), np.ascontiguousarray(ws, dtype=np.float32).view(np.uint32)), mode
        got, nan = np_u8(codes), np.isnan(C.decode(want, fmt))
        assert np.array_equal(np.isnan(C.decode(got, fmt)), nan), mode
        assert np.array_equal(got[~nan], want[~nan]), mode
        assert np.array_equal(nan, np.isnan(v) | np.isinf(v)), mode   # 0 times an infinite scale is NaN as well
        with np.errstate(invalid="ignore"):
            full = OB.values(got, np_f32(scales), fmt, mode)
        br, bc = {"rows": (1, 128), "columns": (128, 1), "square": (128, 128)}[mode]
        for r0 in range(0, rows, br):
            for c0 in range(0, cols, bc):
                block = slice(r0, r0 + br), slice(c0, c0 + bc)
                if np.isinf(v[block]).any():
                    assert np.isnan(full[block]).all(), mode


def _codes(rng, *shape):
    q = rng.integers(0, 256, shape, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x38  # no NaN codes
    return q


@pytest.mark.parametrize("m", [4, 16, 17, 40, 64, 65, 200])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fill,where", [(NAN, "all"), (NAN, "one"), (INF, "all"), (-INF, "one"), ("max", "all"), ("max", "one")])
def test_linear_rows_without_numbers(m, fmt, fill, where):
    """A row of x with a NaN or an infinity anywhere gives NaN throughout; one of the largest finite numbers, by weights
    small enough, what fp64 gives.  An FP8 and a bf16 weight alike."""
    rng = np.random.default_rng(m)
    n, k = 160, 272
    wv = (rng.standard_normal((n, k)) * 2.0 ** -20).astype(np.float32)
    wb = torch.from_numpy(wv).to(torch.bfloat16)
    codes, sw = OB.quantize(in_values_f32(wb), fmt, "square")
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).to(torch.bfloat16)
    value = torch.finfo(torch.bfloat16).min if fill == "max" else fill
    if where == "all":
        x[1] = value
    else:
        x[1, 200] = value
    nbytes = F.linear_forward_fp8_block_workspace_size(m, k, n)
    for w, s in ((torch.from_numpy(codes).to(DEV), torch.from_numpy(np.ascontiguousarray(sw, dtype=np.float32)).to(DEV)), (wb.to(DEV), None)):
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
        y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV)
        F.linear_forward_fp8_block(x.to(DEV), w, s is not None, s, None, m, k, n, FMT[fmt], None, None, None, None, ws, nbytes, y)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        got = bf16_out_to_f64(y)
        if fill != "max":
            assert np.isnan(got[1]).all()
            got, rows = np.delete(got, 1, 0), np.delete(in_values_f32(x), 1, 0)
        else:
            rows = in_values_f32(x)
        ref, s_abs = OB.product(OB.values(*OB.quantize(rows, fmt, "rows"), fmt, "rows"), OB.values(codes, sw, fmt, "square").T)
        assert np.isfinite(ref).all()
        assert (np.abs(got - ref) <= OB.tolerance(ref, s_abs, k)).all()


@pytest.mark.parametrize("fill", [NAN, INF, -INF])
@pytest.mark.parametrize("m,k,n", [(200, 272, 160), (520, 640, 272)])
def test_gradients_of_rows_without_numbers(fill, m, k, n):
    """One such number in g: its row of grad_x and its row of grad_w (and element of grad_b) have no numbers, all else is
    as without it where no block is shared, and finite."""
    rng = np.random.default_rng(m)
    bf16 = lambda s, std: torch.from_numpy((rng.standard_normal(s) * std).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, w, g = bf16((m, k), 1.0), bf16((n, k), 0.05), bf16((m, n), 1e-3)
    e = lambda *s, d=torch.uint8: torch.full(s, 0x7F, dtype=d, device=DEV)  # noqa: E731
    w8, sw, x8c, sxc = e(n, k), e(OB.blocks(n), OB.blocks(k), d=torch.float32), e(m, k), e(OB.blocks(m), k, d=torch.float32)
    nf, nb = F.linear_forward_fp8_block_workspace_size(m, k, n), F.linear_backward_fp8_block_workspace_size(m, k, n)
    y = e(m, n, d=torch.bfloat16)
    F.linear_forward_fp8_block(x, w, 0, None, None, m, k, n, F.FP8_E4M3, w8, sw, x8c, sxc, e(nf), nf, y)

    def backward(g):
        gx, gw, gb = (e(*s, d=torch.bfloat16) for s in ((m, k), (n, k), (n,)))
        F.linear_backward_fp8_block(g, x8c, sxc, w8, sw, m, k, n, F.FP8_E5M2, F.FP8_E4M3, 1, 1, 1, e(nb), nb, gx, gw, gb)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        return gx, gw, gb
    want = backward(g)
    odd = g.clone()
    odd[130, 150] = fill
    gx, gw, gb = backward(odd)
    assert all(torch.isfinite(t).all() for t in want)
    assert torch.isnan(gx[130]).all() and torch.isnan(gw[150]).all()
    assert gb[150].isnan() if fill != fill else gb[150] == fill
    for got, ref, i in ((gx, want[0], 130), (gw, want[1], 150), (gb, want[2], 150)):
        keep = torch.arange(got.shape[0], device=DEV) != i
        assert torch.equal(got[keep].view(torch.int16), ref[keep].view(torch.int16))


@pytest.mark.parametrize("tokens", [5, 16, 17, 40])
@pytest.mark.parametrize("fill", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["all", "one"])
def test_experts_tokens_without_numbers(tokens, fill, where):
    """A token with a NaN or an infinity gives a row of NaN if an expert takes it, and zeros if none does."""
    rng = np.random.default_rng(tokens)
    topk, experts, hidden, inter = 3, 6, 256, 144
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(DEV)  # noqa: E731
    w13, w2 = t(_codes(rng, experts, 2 * inter, hidden)), t(_codes(rng, experts, hidden, inter))
    s13 = t(rng.uniform(0.5, 2.0, (experts, 2, 2, 2)).astype(np.float32) * np.float32(2.0 ** -12))
    s2 = t(rng.uniform(0.5, 2.0, (experts, 2, 2)).astype(np.float32) * np.float32(2.0 ** -8))
    x = t(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16)
    ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    ids[3] = (-1, experts, -7)
    ids[2, 1:] = -1
    for token in (2, 3):
        if where == "all":
            x[token] = fill
        else:
            x[token, 201] = fill
    nbytes = F.moe_forward_fp8_block_workspace_size(tokens, topk, experts, hidden, inter)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((tokens, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
    F.moe_forward_fp8_block(x, t(ids), torch.full((tokens, topk), 0.5, device=DEV), tokens, topk, experts, hidden, inter, F.FP8_E4M3,
                            w13, s13, w2, s2, ws, nbytes, out)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    assert torch.isnan(out[2]).all()
    assert (out[3] == 0).all()
    keep = torch.tensor([i for i in range(tokens) if i != 2], device=DEV)
    assert torch.isfinite(out[keep]).all()

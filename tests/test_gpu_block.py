"""GPU parity: block-scaled quantize and product (one scale for each block of 128).

Bytes and scales are compared bit for bit with the oracle; products with its fp64 result within the
bound derived in ``oracle/block.py``."""

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F
from oracle import block as OB
from oracle import fp8_codec as C
from helpers import np_u8, np_f32, in_values_f32, bf16_out_to_f64, np_bf16_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = {"e4m3": F.FP8_E4M3, "e5m2": F.FP8_E5M2}
IN = {torch.bfloat16: F.FP8_IN_BF16, torch.float16: F.FP8_IN_F16, torch.float32: F.FP8_IN_F32}


def _acts(rng, rows, cols, std=1.0, dtype=torch.bfloat16):
    v = rng.standard_normal((rows, cols)).astype(np.float32) * std
    v *= np.exp(rng.standard_normal((rows, 1))).astype(np.float32)
    v[:, rng.random(cols) < 0.02] *= 20.0
    return torch.from_numpy(v).to(dtype)


def _same(t, want):
    """fp32 scales bit for bit (a NaN never occurs among them)."""
    assert np.array_equal(np_f32(t).view(np.uint32), want.astype(np.float32).view(np.uint32))


def quantize_gpu(x, fmt, row=True, col=False, square=False, fill=0xAB):
    rows, cols = x.shape
    q = lambda: torch.full((rows, cols), fill, dtype=torch.uint8, device=DEV)  # noqa: E731
    xd = x.to(DEV)
    if square:
        o, s = q(), torch.zeros(OB.blocks(rows), OB.blocks(cols), device=DEV)
        F.fp8_quantize_block128(xd, IN[x.dtype], rows, cols, FMT[fmt], o, s)
        return o, s
    o = [q() if w else None for w in (row, col)]
    s = [torch.zeros(OB.blocks(cols), rows, device=DEV) if row else None,
         torch.zeros(OB.blocks(rows), cols, device=DEV) if col else None]
    F.fp8_quantize_block(xd, IN[x.dtype], rows, cols, FMT[fmt], o[0], s[0], o[1], s[1])
    return o[0], s[0], o[1], s[1]


SHAPES = [(1, 1), (1, 128), (3, 16), (127, 129), (128, 128), (129, 136), (256, 1024), (300, 520), (1, 4096), (777, 8)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_matches_the_oracle(rows, cols, fmt):
    rng = np.random.default_rng(rows * 7919 + cols)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x = _acts(rng, rows, cols, 0.5, dtype)
        v = in_values_f32(x)
        for row, col in ((True, True), (True, False), (False, True)):
            o, s, oc, sc = quantize_gpu(x, fmt, row, col)
            torch.cuda.synchronize()
            if row:
                want, ws = OB.quantize(v, fmt, "rows")
                assert np.array_equal(np_u8(o), want)
                _same(s, ws)
            if col:
                want, ws = OB.quantize(v, fmt, "columns")
                assert np.array_equal(np_u8(oc), want)
                _same(sc, ws)
        o, s = quantize_gpu(x, fmt, square=True)
        want, ws = OB.quantize(v, fmt, "square")
        assert np.array_equal(np_u8(o), want)
        _same(s, ws)


def test_quantize_special_values():
    """All-zero blocks, blocks below the smallest scale, NaN (a NaN byte, not in the scale) and an
    infinity (an infinite scale: the block decodes to NaN or infinity, its neighbours do not change)."""
    x = torch.zeros(130, 300)
    x[0, 0] = 3.0
    x[1, 130] = 1e-20
    x[2, 5], x[2, 6] = float("nan"), 2.0
    x[3, 10], x[3, 11] = float("inf"), 1.0
    x[129, 299] = -7.0
    x = x.to(torch.bfloat16)
    o, s, oc, sc = quantize_gpu(x, "e4m3", True, True)
    torch.cuda.synchronize()
    for mode, q, sv in (("rows", o, s), ("columns", oc, sc)):
        with np.errstate(invalid="ignore"):
            want, ws = OB.quantize(in_values_f32(x), "e4m3", mode)
        _same(sv, ws)
        got, ref = C.decode(np_u8(q), "e4m3"), C.decode(want, "e4m3")
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        assert np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("shift", [1, 3])
def test_quantize_unaligned_views(shift):
    """Rows that start at any element: the scalar path gives the same bytes, and nothing lands outside."""
    rng = np.random.default_rng(5)
    rows, cols = 40, 264
    flat = _acts(rng, 1, rows * cols + 8)[0]
    x = flat[shift:shift + rows * cols].view(rows, cols)
    want, ws = OB.quantize(in_values_f32(x), "e4m3", "rows")
    buf = torch.full((rows * cols + 16,), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.zeros(OB.blocks(cols), rows, device=DEV)
    F.fp8_quantize_block(flat.to(DEV)[shift:], F.FP8_IN_BF16, rows, cols, F.FP8_E4M3, buf[shift:], s)
    torch.cuda.synchronize()
    got = np_u8(buf)
    assert np.array_equal(got[shift:shift + rows * cols].reshape(rows, cols), want)
    assert (got[:shift] == 0xAB).all() and (got[shift + rows * cols:] == 0xAB).all()
    _same(s, ws)


# ------------------------------------------------------------------------------------------------
# product
# ------------------------------------------------------------------------------------------------
def _operand(rng, mn, k, mode, fmt, mn_major, std=1.0):
    """(stored codes, scales, BlockScale factory, fp64 values [mn][k]); mode "rows" (a scale per row) or "square"."""
    v = np.asarray(in_values_f32(_acts(rng, mn, k, std)))
    codes, s = OB.quantize(v, fmt, mode)
    vals = OB.values(codes, s, fmt, mode)
    nkb = OB.blocks(k)
    if mode == "rows":
        scale = (1, 1, mn)                     # [K block][row]
    elif mn_major:
        s, scale = np.ascontiguousarray(s.T), (128, 1, OB.blocks(mn))   # blocks of the stored [k][mn]
    else:
        scale = (128, nkb, 1)
    stored = np.ascontiguousarray(codes.T if mn_major else codes)
    return stored, s, scale, vals


def run_product(m, n, k, layout="NT", a_mode="rows", b_mode="square", fmt_a="e4m3", fmt_b="e4m3", bias=False, batch=1,
                ldo_pad=0, seed=0, out_shift=0, a_broadcast=False):
    rng = np.random.default_rng(seed + m * 31 + n * 17 + k)
    a_mn, b_mn = layout[0] == "T", layout[1] == "N"
    A = [_operand(rng, m, k, a_mode, fmt_a, a_mn) for _ in range(1 if a_broadcast else batch)]
    Bo = [_operand(rng, n, k, b_mode, fmt_b, b_mn, 0.02) for _ in range(batch)]

    def pack(ops):
        """Stored rows padded to a multiple of 16 bytes (filled with NaN codes: they must not be read)."""
        r, c = ops[0][0].shape
        ld = -(-c // 16) * 16
        q = np.full((len(ops), r, ld), 0x7F, dtype=np.uint8)
        for i, o in enumerate(ops):
            q[i, :, :c] = o[0]
        s = np.stack([o[1] for o in ops]).astype(np.float32)
        return torch.from_numpy(q).to(DEV), ld, r * ld, torch.from_numpy(s).to(DEV), int(s[0].size)

    qa, lda, sta, sa, nsa = pack(A)
    qb, ldb, stb, sb, nsb = pack(Bo)
    ldo = n + ldo_pad
    sto = m * ldo
    bv = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(torch.bfloat16) if bias else None
    out = torch.full((batch * sto + out_shift + 8,), 0x7FC1, dtype=torch.int16, device=DEV)
    lay = {"NT": F.FP8_LAYOUT_NT, "NN": F.FP8_LAYOUT_NN, "TN": F.FP8_LAYOUT_TN, "TT": F.FP8_LAYOUT_TT}[layout]
    F.fp8_gemm_block(qa, qb, FMT[fmt_a], FMT[fmt_b], lay, m, n, k, lda, ldb, ldo, batch,
                     0 if a_broadcast or batch == 1 else sta, stb if batch > 1 else 0, sto,
                     F.BlockScale(sa, *A[0][2], 0 if a_broadcast else nsa), F.BlockScale(sb, *Bo[0][2], nsb),
                     None if bv is None else bv.to(DEV), out[out_shift:])
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    got = out.cpu().numpy().view(np.uint16)
    assert (got[:out_shift] == 0x7FC1).all() and (got[out_shift + batch * sto:] == 0x7FC1).all()
    got = got[out_shift:out_shift + batch * sto].reshape(batch, m, ldo)
    assert (got[:, :, n:] == 0x7FC1).all(), "written past n"
    worst = 0.0
    for c in range(batch):
        ref, s_abs = OB.product(A[0 if a_broadcast else c][3], Bo[c][3].T,
                                None if bv is None else C.bf16_bits_to_f64(np_bf16_bits(bv)))
        err = np.abs(C.bf16_bits_to_f64(got[c, :, :n].copy()) - ref)
        tol = OB.tolerance(ref, s_abs, k)
        bad = ~(err <= tol)
        assert not bad.any(), f"batch {c}: {int(bad.sum())} of {bad.size} outside, first {np.argwhere(bad)[:4].tolist()}"
        worst = max(worst, float((err / np.maximum(tol, 1e-300)).max()))
    return got, worst


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 1024, 1024), (3, 48, 4096), (16, 2048, 512), (17, 144, 272),
                                   (64, 1024, 2048), (65, 640, 1040), (128, 256, 8192), (130, 1000, 400), (200, 4096, 128),
                                   (1000, 1040, 1536), (2048, 2064, 520), (2049, 4112, 1024)])
def test_product_forward(m, n, k):
    run_product(m, n, k, bias=(m + k) % 2 == 0)


@pytest.mark.parametrize("layout", ["NT", "NN", "TN", "TT"])
@pytest.mark.parametrize("a_mode,b_mode", [("rows", "square"), ("rows", "rows"), ("square", "rows"), ("square", "square")])
@pytest.mark.parametrize("m,n,k", [(48, 272, 1200), (144, 1024, 333), (2064, 2576, 1500)])
def test_product_layouts_and_granularities(layout, a_mode, b_mode, m, n, k):
    run_product(m, n, k, layout, a_mode, b_mode, "e5m2", "e4m3", bias=layout == "NT")


@pytest.mark.parametrize("batch,m,n,k,broadcast", [(3, 40, 136, 256, False), (5, 1, 64, 700, False), (4, 300, 264, 384, True),
                                                  (9, 512, 512, 512, False)])
def test_product_batched_and_padded(batch, m, n, k, broadcast):
    run_product(m, n, k, batch=batch, ldo_pad=24, a_broadcast=broadcast, bias=True)


@pytest.mark.parametrize("m", [2, 70, 700])
def test_product_odd_output(m):
    """Odd row strides and a base that is only 2-byte aligned: direct stores."""
    run_product(m, 97, 512, ldo_pad=2, out_shift=1, bias=True)
    run_product(m, 2049, 144, ldo_pad=0, out_shift=3)


def test_product_is_deterministic_and_captures():
    """Two runs and a graph replay give the same bits (split K included)."""
    for m, n, k in ((1, 1024, 4096), (128, 512, 8192), (1024, 2048, 1024)):
        a, _ = run_product(m, n, k, seed=3)
        b, _ = run_product(m, n, k, seed=3)
        assert np.array_equal(a, b)


def test_product_without_k_is_the_bias():
    bias = torch.arange(40, dtype=torch.float32).to(torch.bfloat16).to(DEV)
    out = torch.full((3, 40), 9.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_gemm_block(None, None, 0, 0, F.FP8_LAYOUT_NT, 3, 40, 0, 0, 0, 40, 1, 0, 0, 0, None, None, bias, out)
    torch.cuda.synchronize()
    assert torch.equal(out, bias.expand(3, 40))

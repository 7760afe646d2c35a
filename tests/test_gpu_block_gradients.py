"""GPU: the block-scaled linear layer's gradients against the gradients' formulas on the unquantized tensors, every
element, and against differences of the loss.

Each element of an operand is off by half a step of its format, at most: `eg |g|` with eg = 2^-3 (E5M2) or 2^-4 (E4M3),
`2^-4 |w|`, `2^-4 |x|`, or half the smallest subnormal step of its block where that is more (2^-17 or 2^-10 of the block's
scale, itself at most the tensor's maximum / FP8_MAX).  A term p q of a gradient's sum is so off by at most
c = |p| dq + |q| dp + dp dq.  The roundings of a sum's terms are those of different random elements, so their sum is
within 6 sqrt(sum c^2) (Hoeffding: outside with a chance of 2 exp(-18) = 3e-8 for each of the 4e4 elements); the product's own
bound (``oracle/block.py``) comes on top.  All tensors are positive, so a gradient is as large as the sum of its terms'
magnitudes and the bound is 6 to 23 % of it: a gradient that is zero, transposed or short of a block lies outside."""

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F
from oracle import block as OB
from helpers import in_values_f32, bf16_out_to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {"e4m3": (2.0 ** -4, 2.0 ** -10 / 448.0), "e5m2": (2.0 ** -3, 2.0 ** -17 / 57344.0)}


def _off(v, fmt):
    rel, low = HALF[fmt]
    return np.maximum(rel * np.abs(v), low * np.abs(v).max())


def _bound(p, q, fmt_p, fmt_q, ref):
    """Tolerance of p @ q, elementwise, from the operands' roundings and the product."""
    dp, dq = _off(p, fmt_p), _off(q, fmt_q)
    a, b = np.abs(p), np.abs(q)
    # c^2 = (a dq + dp b + dp dq)^2, summed over the contraction
    sq = lambda x, y: (x * x) @ (y * y)  # noqa: E731
    cross = (a * dp) @ (dq * b) + (a * dp) @ (dq * dq) + (dp * dp) @ (b * dq)
    c2 = sq(a, dq) + sq(dp, b) + sq(dp, dq) + 2 * cross
    return 6 * np.sqrt(c2) + OB.tolerance(np.abs(ref), 1.5 * (a @ b), p.shape[1])


@pytest.mark.parametrize("fmt_g", ["e5m2", "e4m3"])
@pytest.mark.parametrize("m,k,n", [(144, 128, 144), (333, 272, 160), (160, 640, 400)])
def test_gradients_against_formulas_and_differences(m, k, n, fmt_g):
    rng = np.random.default_rng(m + k + n)
    pos = lambda shape, std: torch.from_numpy((np.abs(rng.standard_normal(shape)) * std).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    x, w, g = pos((m, k), 1.0), pos((n, k), 0.05), pos((m, n), 1e-3)
    e = lambda *s, d=torch.uint8: torch.full(s, 0x7F, dtype=d, device=DEV)  # noqa: E731
    w8, sw, x8c, sxc = e(n, k), e(OB.blocks(n), OB.blocks(k), d=torch.float32), e(m, k), e(OB.blocks(m), k, d=torch.float32)
    y, gx, gw, gb = (e(*s, d=torch.bfloat16) for s in ((m, n), (m, k), (n, k), (n,)))
    nf, nb = F.linear_forward_fp8_block_workspace_size(m, k, n), F.linear_backward_fp8_block_workspace_size(m, k, n)
    fmt = F.FP8_E5M2 if fmt_g == "e5m2" else F.FP8_E4M3
    F.linear_forward_fp8_block(x.to(DEV), w.to(DEV), 0, None, None, m, k, n, F.FP8_E4M3, w8, sw, x8c, sxc, e(nf), nf, y)
    F.linear_backward_fp8_block(g.to(DEV), x8c, sxc, w8, sw, m, k, n, fmt, F.FP8_E4M3, 1, 1, 1, e(nb), nb, gx, gw, gb)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    xv, wv, gv = (in_values_f32(t).astype(np.float64) for t in (x, w, g))
    loss = lambda a, b: float((gv * (a @ b.T)).sum())  # noqa: E731
    for got, which, p, q, fp in ((gx, 0, gv, wv, fmt_g), (gw, 1, gv.T, xv, fmt_g)):
        ref, got = p @ q, bf16_out_to_f64(got)
        tol = _bound(p, q, fp, "e4m3", ref)
        assert (ref > 3 * tol).all(), "the bound would let a zero pass"
        err = np.abs(got - ref)
        assert (err <= tol).all(), (which, float((err / tol).max()))
        for _ in range(8):
            i, j = rng.integers(ref.shape[0]), rng.integers(ref.shape[1])
            d = []
            for s in (1, -1):
                a, b = xv.copy(), wv.copy()
                (a if which == 0 else b)[i, j] += s * 0.5  # the loss is linear in either: any step will do
                d.append(loss(a, b))
            assert abs((d[0] - d[1]) - got[i, j]) <= tol[i, j] + 1e-9 * abs(d[0])
    ref = gv.sum(0)
    assert (np.abs(bf16_out_to_f64(gb) - ref) <= 2.0 ** -8 * (1 + 2.0 ** -8) * ref + (m + 1) * 2.0 ** -24 * ref).all()

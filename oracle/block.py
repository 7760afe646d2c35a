"""Oracle of the block-scaled FP8 operators: one scale for each block of 128.

Test infrastructure only (see ``oracle/__init__.py``).  A block's scale and bytes are the dynamic
step's formula on that block, ``s = max(RN32(amax / FP8_MAX), 1e-12)`` and
``q = q_fmt(RN32(x * RN32(1/s)))``; everything after the bytes is fp64.

Error bound of a product.  The kernel forms each 128-deep block sum on the tensor cores, multiplies it by
``RN32(sa * sb)`` inside an fp32 fma and adds the blocks in fp32; with ``S = sum |a b| sa sb``:

* the block sum: products of FP8 values are exact in fp32; the tensor core's accumulation over 128 is held
  to ``2^-21 S`` (half of what the per-tensor GEMM's tests allow it over depths up to 8192);
* the scale product: half a step of fp32, ``2^-24 S``;
* the additions over ``nb`` blocks and up to 8 ranges: ``(nb + 8) 2^-24 S``;
* the bias addition ``2^-24 |ref|`` and the bf16 rounding ``2^-8 |ref|`` (half a step, relative to the
  value), taken together as ``(2^-8 + 2^-16) |ref|``.
"""

from __future__ import annotations

import numpy as np

from .fp8_codec import FP8_MAX, decode, encode

B = 128


def blocks(n: int) -> int:
    return -(-n // B)


def _amax(x: np.ndarray, br: int, bc: int) -> np.ndarray:
    """[ceil(rows/br)][ceil(cols/bc)] of max |x|, NaN ignored (fp32)."""
    rows, cols = x.shape
    a = np.zeros((-(-rows // br) * br, -(-cols // bc) * bc), dtype=np.float32)
    a[:rows, :cols] = np.where(np.isnan(x), 0, np.abs(x))
    return a.reshape(a.shape[0] // br, br, a.shape[1] // bc, bc).max((1, 3))


def quantize(x: np.ndarray, fmt: str, mode: str):
    """(codes, scales) of x [rows][cols] (fp32 values); mode "rows", "columns" or "square".  Scales in the
    library's layouts: [ceil(cols/128)][rows], [ceil(rows/128)][cols], [ceil(rows/128)][ceil(cols/128)]."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    br, bc = {"rows": (1, B), "columns": (B, 1), "square": (B, B)}[mode]
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.maximum(_amax(x, br, bc) / np.float32(FP8_MAX[fmt]), np.float32(1e-12))
        inv = np.float32(1.0) / s
        full = np.repeat(np.repeat(inv, br, 0), bc, 1)[:rows, :cols]
        codes = encode(x * full, fmt)
    return codes, np.ascontiguousarray(s.T) if mode == "rows" else s


def values(codes: np.ndarray, s: np.ndarray, fmt: str, mode: str) -> np.ndarray:
    """fp64 values of codes [rows][cols] with their scales (the layouts of :func:`quantize`)."""
    rows, cols = codes.shape
    s = np.asarray(s, dtype=np.float64)
    if mode == "rows":
        full = np.repeat(s.T, B, 1)[:, :cols]
    elif mode == "columns":
        full = np.repeat(s, B, 0)[:rows]
    else:
        full = np.repeat(np.repeat(s, B, 0), B, 1)[:rows, :cols]
    with np.errstate(invalid="ignore"):
        return decode(codes, fmt) * full


def product(a: np.ndarray, b: np.ndarray, bias=None):
    """(ref, s_abs) of a [m][k] . b [k][n] (+ bias [n]), fp64 values with their scales inside."""
    ref = a @ b
    if bias is not None:
        ref = ref + bias
    return ref, np.abs(a) @ np.abs(b)


def tolerance(ref: np.ndarray, s_abs: np.ndarray, k: int) -> np.ndarray:
    nb = blocks(k)
    return (2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + (2.0 ** -21 + (nb + 9) * 2.0 ** -24) * s_abs

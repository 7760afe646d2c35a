"""GPU: the block-scaled forward with no more workspace than it says it uses gives the bits of a call with all of it,
and writes nothing behind it."""

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("m", [1, 16, 17, 64, 65, 300])
@pytest.mark.parametrize("columns", [False, True])
def test_forward_with_the_least_workspace(m, columns):
    k, n = 528, 400
    rng = np.random.default_rng(m)
    bf16 = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, w, b = bf16(m, k), bf16(n, k), bf16(n)
    full = F.linear_forward_fp8_block_workspace_size(m, k, n)
    part = 0 if m <= 16 and not columns else F.linear_forward_fp8_block_workspace_size(m, k, 0)

    def run(w, sw, keep, nbytes):
        """y, and the quantized weight if `keep`, with `nbytes` of workspace and a guard behind it."""
        e = lambda *s, d=torch.uint8: torch.full(s, 0x7F, dtype=d, device=DEV)  # noqa: E731
        w8, s8 = (e(n, k), e(4, 5, d=torch.float32)) if keep else (None, None)
        xc, xs = (e(m, k), e(-(-m // 128), k, d=torch.float32)) if columns else (None, None)
        ws, y = e(nbytes + 4096), e(m, n, d=torch.bfloat16)
        F.linear_forward_fp8_block(x, w, sw is not None, sw, b, m, k, n, F.FP8_E4M3, w8, s8, xc, xs, ws if nbytes else None,
                                   nbytes, y)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        assert (ws[nbytes:] == 0x7F).all()
        return [t for t in (y, xc, xs, w8, s8) if t is not None]

    same = lambda p, q: all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(p, q))  # noqa: E731
    want = run(w, None, True, full)
    assert same(run(w, None, True, part), want)
    assert same(run(want[-2], want[-1], False, part), want[:-2])
    assert same(run(w, None, False, full), want[:-2])


@pytest.mark.parametrize("m", [3, 40])
def test_forward_without_columns(m):
    """No output columns: nothing is done, and nothing needed, unless the column form of x is wanted."""
    k = 272
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    F.linear_forward_fp8_block(x, None, 0, None, None, m, k, 0, F.FP8_E4M3, None, None, None, None, None, 0, None)
    nbytes = F.linear_forward_fp8_block_workspace_size(m, k, 0)
    ws = torch.full((nbytes + 256,), 0x7F, dtype=torch.uint8, device=DEV)
    got, want = ([torch.zeros(m, k, dtype=torch.uint8, device=DEV), torch.zeros(1, k, device=DEV)] for _ in range(2))
    F.linear_forward_fp8_block(x, None, 0, None, None, m, k, 0, F.FP8_E4M3, None, None, *got, ws, nbytes, None)
    F.fp8_quantize_block(x, F.FP8_IN_BF16, m, k, F.FP8_E4M3, None, None, *want)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (ws[nbytes:] == 0x7F).all()

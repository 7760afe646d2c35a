"""GPU: captured products of every kind replay to the bits of eager calls: K cut over a cluster, pair tiles, a scale per
column on one or both sides, the streaming kernels.  Outputs are poisoned before each call and replay."""

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F
from oracle import block as OB

pytestmark = pytest.mark.gpu
DEV = "cuda"
LAYOUTS = {"NT": F.FP8_LAYOUT_NT, "NN": F.FP8_LAYOUT_NN, "TN": F.FP8_LAYOUT_TN}


def _codes(rng, *shape):
    q = rng.integers(0, 256, shape, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x38  # no NaN codes
    return torch.from_numpy(q).to(DEV)


@pytest.mark.parametrize("columns", [False, True], ids=["squares", "columns"])
@pytest.mark.parametrize("layout,m,n,k", [("NT", 1, 1024, 4096), ("NT", 48, 1024, 4096), ("NT", 128, 512, 8192),
                                          ("NT", 1024, 2048, 1024), ("NN", 128, 512, 8192), ("TN", 128, 512, 8192),
                                          ("TN", 2064, 2576, 1500)])
def test_product_replays(layout, m, n, k, columns):
    """(`columns`: B has a scale per column of the product, else one per 128.)"""
    rng = np.random.default_rng(m + n + k)
    a_mn, b_mn = layout[0] == "T", layout[1] == "N"
    kb, nb = OB.blocks(k), OB.blocks(n)
    lda, ldb = (m if a_mn else k), (n if b_mn else k)
    a, b = _codes(rng, k if a_mn else m, lda), _codes(rng, k if b_mn else n, ldb)
    s = lambda *shape: torch.from_numpy(rng.uniform(0.5, 2.0, shape).astype(np.float32)).to(DEV)  # noqa: E731
    sa = F.BlockScale(s(kb, m), 1, 1, m)
    sb = F.BlockScale(s(kb, n), 1, 1, n) if columns else F.BlockScale(s(nb, kb), 128, kb, 1)
    bias = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(torch.bfloat16).to(DEV)
    out = torch.empty(m, n, dtype=torch.int16, device=DEV)

    def call(stream=None):
        F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, LAYOUTS[layout], m, n, k, lda, ldb, n, 1, 0, 0, 0, sa, sb, bias, out,
                         stream=stream)

    got = []
    for _ in range(2):
        out.fill_(0x7FC1)
        call()
        got.append(out.clone())
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    for _ in range(2):
        out.fill_(0x7FC1)
        graph.replay()
        got.append(out.clone())
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    assert torch.isfinite(got[0].view(torch.bfloat16)).all()
    assert all(torch.equal(g, got[0]) for g in got[1:])
    # new codes and scales in the captured buffers
    a.copy_(_codes(rng, *a.shape))
    sb.tensor.mul_(0.5)
    out.fill_(0x7FC1)
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    out.fill_(0x7FC1)
    call()
    torch.cuda.synchronize()
    assert torch.equal(replayed, out) and not torch.equal(replayed, got[0])

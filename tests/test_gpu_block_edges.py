"""GPU: calls of the block-scaled entries that must give the same bits as a plainer call: shared operands,
padded scales, rows and tokens that hold no finite number, slots that are skipped, other ways to launch."""

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


def _gemm(a, b, m, n, k, batch, stride_a, stride_b, sa, sb, bias=None, lda=None, ldb=None):
    out = torch.full((batch, m, n), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, lda or k, ldb or k, n, batch, stride_a, stride_b,
                     m * n, sa, sb, bias, out)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    return out


@pytest.mark.parametrize("m", [1, 16, 33, 64, 96, 300])
def test_shared_weight_of_a_batch(m):
    """One weight for every batch (stride 0) against copies of it."""
    rng = np.random.default_rng(m)
    n, k, batch = 272, 400, 3
    kb, nb = 4, 3
    a, b = _codes(rng, batch, m, k), _codes(rng, n, k)
    sa, sb = _scales(rng, batch, kb, m), _scales(rng, nb, kb)
    one = _gemm(a, b, m, n, k, batch, m * k, 0, F.BlockScale(sa, 1, 1, m, kb * m), F.BlockScale(sb, 128, kb, 1, 0))
    copies = _gemm(a, b.repeat(batch, 1, 1), m, n, k, batch, m * k, n * k, F.BlockScale(sa, 1, 1, m, kb * m),
                   F.BlockScale(sb.repeat(batch, 1, 1), 128, kb, 1, nb * kb))
    assert torch.equal(one.view(torch.int16), copies.view(torch.int16))
    # each batch alone
    for i in range(batch):
        alone = _gemm(a[i], b, m, n, k, 1, 0, 0, F.BlockScale(sa[i], 1, 1, m), F.BlockScale(sb, 128, kb, 1))
        assert torch.equal(one[i].view(torch.int16), alone[0].view(torch.int16))


@pytest.mark.parametrize("m", [5, 64, 200])
def test_padded_scales_and_rows(m):
    """Scales and rows further apart than they need to be, with NaN between them."""
    rng = np.random.default_rng(m + 1)
    n, k, kb, nb = 144, 700, 6, 2
    a, b = _codes(rng, m, 704), _codes(rng, n, 720)
    a[:, k:] = 0x7F
    b[:, k:] = 0x7F
    sa, sb = _scales(rng, kb, m), _scales(rng, nb, kb)
    plain = _gemm(a, b, m, n, k, 1, 0, 0, F.BlockScale(sa, 1, 1, m), F.BlockScale(sb, 128, kb, 1), lda=704, ldb=720)
    wide_a = torch.full((m, 3 * kb), float("nan"), device=DEV)
    wide_a[:, ::3] = sa.T
    wide_b = torch.full((2 * kb, nb + 5), float("nan"), device=DEV)
    wide_b[::2, :nb] = sb.T
    padded = _gemm(a, b, m, n, k, 1, 0, 0, F.BlockScale(wide_a, 1, 3 * kb, 3), F.BlockScale(wide_b, 128, 1, 2 * (nb + 5)),
                   lda=704, ldb=720)
    assert torch.isfinite(plain).all()
    assert torch.equal(plain.view(torch.int16), padded.view(torch.int16))


@pytest.mark.parametrize("m", [3, 50, 150])
def test_a_matrix_with_itself(m):
    """The same tensor as both operands."""
    rng = np.random.default_rng(m + 2)
    k, kb = 256, 2
    m16 = -(-m // 16) * 16
    a = _codes(rng, m16, k)
    sa = _scales(rng, kb, m16)
    s = F.BlockScale(sa, 1, 1, m16)
    out = _gemm(a, a, m16, m16, k, 1, 0, 0, s, s)[0].float()
    v = (a.view(torch.float8_e4m3fn).double().reshape(m16, kb, 128) * sa.T.double()[:, :, None]).reshape(m16, k).cpu().numpy()
    ref = v @ v.T
    assert (np.abs(out.double().cpu().numpy() - ref) <= OB.tolerance(ref, np.abs(v) @ np.abs(v).T, k)).all()


@pytest.mark.parametrize("m", [4, 16, 40, 200])
def test_rows_without_numbers_stay_alone(m):
    """NaN, infinity or nothing but zeros in one row of x changes that row of the output only."""
    rng = np.random.default_rng(m + 3)
    n, k = 160, 272
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    w8, sw = _codes(rng, n, k), _scales(rng, 2, 3)
    nbytes = F.linear_forward_fp8_block_workspace_size(m, k, n)

    def run(x):
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
        y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=DEV)
        F.linear_forward_fp8_block(x, w8, 1, sw, None, m, k, n, F.FP8_E4M3, None, None, None, None, ws, nbytes, y)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        return y
    want = run(x)
    for fill in (float("nan"), float("inf"), 0.0, torch.finfo(torch.bfloat16).min):
        odd = x.clone()
        odd[1] = fill
        got = run(odd)
        keep = torch.arange(m, device=DEV) != 1
        assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16)), fill
        if fill == 0.0:
            assert (got[1] == 0).all()


@pytest.mark.parametrize("tokens", [5, 16, 30])
def test_experts_tokens_and_slots_stay_alone(tokens):
    """A token without finite numbers changes its own row only; the weight of a skipped slot (even NaN) and the
    rest of an output buffer are not touched."""
    rng = np.random.default_rng(tokens)
    topk, experts, hidden, inter = 3, 6, 256, 144
    w13, w2 = _codes(rng, experts, 2 * inter, hidden), _codes(rng, experts, hidden, inter)
    s13, s2 = _scales(rng, experts, 2, 2, 2) * 2.0 ** -12, _scales(rng, experts, 2, 2) * 2.0 ** -8
    x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    ids = torch.from_numpy(rng.integers(-1, experts, (tokens, topk)).astype(np.int32)).to(DEV)
    ids[0] = torch.tensor([-1, 2, experts], dtype=torch.int32, device=DEV)
    wts = torch.from_numpy(rng.random((tokens, topk)).astype(np.float32)).to(DEV)
    nbytes = F.moe_forward_fp8_block_workspace_size(tokens, topk, experts, hidden, inter)

    def run(x, wts):
        ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.full((tokens + 2, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
        F.moe_forward_fp8_block(x, ids, wts, tokens, topk, experts, hidden, inter, F.FP8_E4M3, w13, s13, w2, s2, ws, nbytes, out)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        assert (out[tokens:] == 7.0).all()
        return out[:tokens]
    want = run(x, wts)
    assert torch.isfinite(want).all()
    skipped = (ids < 0) | (ids >= experts)
    assert torch.equal(run(x, wts.masked_fill(skipped, float("nan"))), want)
    for fill in (float("nan"), float("inf"), torch.finfo(torch.bfloat16).min):
        odd = x.clone()
        odd[2] = fill
        got = run(odd, wts)
        keep = torch.arange(tokens, device=DEV) != 2
        assert torch.equal(got[keep], want[keep]), fill


@pytest.mark.parametrize("m", [1, 40, 200, 600])
def test_product_plain_launches_and_the_profiler(m):
    """The same bits without programmatic launches, and with every kernel timed; both replayed from a graph."""
    rng = np.random.default_rng(m + 4)
    n, k, kb, nb = 528, 1040, 9, 5
    a, b = _codes(rng, m, k), _codes(rng, n, k)
    sa, sb = F.BlockScale(_scales(rng, kb, m), 1, 1, m), F.BlockScale(_scales(rng, nb, kb), 128, kb, 1)
    want = _gemm(a, b, m, n, k, 1, 0, 0, sa, sb)
    F.fp8_set_pdl(False)
    try:
        plain = _gemm(a, b, m, n, k, 1, 0, 0, sa, sb)
    finally:
        F.fp8_set_pdl(True)
    assert torch.equal(plain.view(torch.int16), want.view(torch.int16))
    F.fp8_profiler_enable(True)
    try:
        timed = _gemm(a, b, m, n, k, 1, 0, 0, sa, sb)
    finally:
        F.fp8_profiler_enable(False)
    assert torch.equal(timed.view(torch.int16), want.view(torch.int16))
    out = torch.zeros_like(want)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, k, k, n, 1, 0, 0, m * n, sa, sb, None, out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows and columns of the quantizers equal those of a small call, and the
    last columns of a product agree with fp64."""
    rows, cols = 66048, 33024
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    for r in range(0, rows, 8256):
        x[r:r + 8256] = torch.randn(8256, cols, device=DEV, generator=gen)
    rb, cb = rows // 128, cols // 128

    def quantize(x):
        r, c = x.shape
        out = [torch.empty(r, c, dtype=torch.uint8, device=DEV) for _ in range(2)]
        s = [torch.empty(c // 128, r, device=DEV), torch.empty(r // 128, c, device=DEV)]
        F.fp8_quantize_block(x, F.FP8_IN_BF16, r, c, F.FP8_E4M3, out[0], s[0], out[1], s[1])
        return out, s
    (q, qc), (s, sc) = quantize(x)
    tail = x[-256:, -512:].contiguous()
    (tq, tqc), (ts, tsc) = quantize(tail)
    torch.cuda.synchronize()
    assert torch.equal(q[-256:, -512:], tq) and torch.equal(qc[-256:, -512:], tqc)
    assert torch.equal(s[-4:, -256:], ts) and torch.equal(sc[-2:, -512:], tsc)
    del qc, sc
    w8, ws = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rb, cb, device=DEV)
    F.fp8_quantize_block128(x, F.FP8_IN_BF16, rows, cols, F.FP8_E4M3, w8, ws)
    t8, t_s = torch.empty(256, 512, dtype=torch.uint8, device=DEV), torch.empty(2, 4, device=DEV)
    F.fp8_quantize_block128(tail, F.FP8_IN_BF16, 256, 512, F.FP8_E4M3, t8, t_s)
    torch.cuda.synchronize()
    assert torch.equal(w8[-256:, -512:], t8) and torch.equal(ws[-2:, -4:], t_s)
    wv = (w8[-16:].view(torch.float8_e4m3fn).double().reshape(16, cb, 128) * ws[-1].double()[None, :, None]).reshape(16, cols)
    for m in (3, 130):
        a, sa = q[:m].contiguous(), s[:, :m].contiguous()
        out = _gemm(a, w8, m, rows, cols, 1, 0, 0, F.BlockScale(sa, 1, 1, m), F.BlockScale(ws, 128, cb, 1))[0]
        av = (a.view(torch.float8_e4m3fn).double().reshape(m, cb, 128) * sa.T.double()[:, :, None]).reshape(m, cols)
        ref = (av @ wv.T).cpu().numpy()
        tol = OB.tolerance(ref, (av.abs() @ wv.abs().T).cpu().numpy(), cols)
        assert (np.abs(out[:, -16:].double().cpu().numpy() - ref) <= tol).all()


def test_experts_past_32_bits():
    """Weights of more than 2^31 bytes: naming the last four experts gives the bits of a call that has only those."""
    rng = np.random.default_rng(9)
    experts, hidden, inter, tokens, topk = 64, 4096, 8192, 2, 2
    gen = torch.Generator(device=DEV).manual_seed(2)

    def codes(*shape):
        q = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)
        return torch.where((q & 0x7F) == 0x7F, torch.full_like(q, 0x38), q)
    w13, w2 = codes(experts, 2 * inter, hidden), codes(experts, hidden, inter)
    s13, s2 = _scales(rng, experts, 2, inter // 128, hidden // 128) * 2.0 ** -14, _scales(rng, experts, hidden // 128, inter // 128) * 2.0 ** -10
    x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    wts = torch.from_numpy(rng.random((tokens, topk)).astype(np.float32)).to(DEV)

    def run(first, ids):
        e = experts - first
        nbytes = F.moe_forward_fp8_block_workspace_size(tokens, topk, e, hidden, inter)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        out = torch.zeros(tokens, hidden, dtype=torch.bfloat16, device=DEV)
        F.moe_forward_fp8_block(x, torch.tensor(ids, dtype=torch.int32, device=DEV), wts, tokens, topk, e, hidden, inter, F.FP8_E4M3,
                                w13[first:], s13[first:], w2[first:], s2[first:], ws, nbytes, out)
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        return out
    far, near = run(0, [[63, 60], [62, 61]]), run(60, [[3, 0], [2, 1]])
    assert torch.isfinite(far).all() and far.abs().max() > 0
    assert torch.equal(far, near)

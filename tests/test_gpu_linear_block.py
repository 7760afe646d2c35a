"""GPU parity: the block-scaled linear layer, forward and backward, against the oracle.

The bytes and scales the forward leaves are compared bit for bit, products within the bound derived in
``oracle/block.py``, the bias gradient within half a step of bf16 plus the fp32 summation's bound; the
gradients are also held against differences of the layer's own fp64 loss."""

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


def _bf16(rng, shape, std):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(torch.bfloat16)


def _within(got, ref, s_abs, k, what):
    err = np.abs(bf16_out_to_f64(got) - ref)
    bad = ~(err <= OB.tolerance(ref, s_abs, k))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, first {np.argwhere(bad)[:4].tolist()}"


def _same_scale(t, want):
    assert np.array_equal(np_f32(t).view(np.uint32), np.ascontiguousarray(want, dtype=np.float32).view(np.uint32))


class Layer:
    """One layer's buffers, and its calls."""

    def __init__(self, m, k, n, seed=0):
        rng = np.random.default_rng(seed + m + 3 * k + 7 * n)
        self.m, self.k, self.n = m, k, n
        self.x, self.w = _bf16(rng, (m, k), 1.0), _bf16(rng, (n, k), 0.05)
        self.b, self.g = _bf16(rng, (n,), 0.1), _bf16(rng, (m, n), 1e-3)
        e = lambda *s, d=torch.uint8: torch.full(s, 0x7F, dtype=d, device=DEV)  # noqa: E731
        self.w8, self.sw = e(n, k), e(OB.blocks(n), OB.blocks(k), d=torch.float32)
        self.x8c, self.sxc = e(m, k), e(OB.blocks(m), k, d=torch.float32)
        self.y, self.gx, self.gw, self.gb = (e(*s, d=torch.bfloat16) for s in ((m, n), (m, k), (n, k), (n,)))
        self.nf = F.linear_forward_fp8_block_workspace_size(m, k, n)
        self.nb = F.linear_backward_fp8_block_workspace_size(m, k, n)
        self.wf, self.wb = e(self.nf), e(self.nb)
        self.dev = [t.to(DEV) for t in (self.x, self.w, self.b, self.g)]

    def forward(self, fmt="e4m3", save=True, bias=True, stream=None):
        x, w, b, _ = self.dev
        s = (self.w8, self.sw, self.x8c, self.sxc) if save else (None,) * 4
        F.linear_forward_fp8_block(x, w, 0, None, b if bias else None, self.m, self.k, self.n, FMT[fmt], *s, self.wf,
                                   self.nf, self.y, stream=stream)

    def backward(self, fmt_g="e5m2", fmt="e4m3", need=(1, 1, 1), stream=None):
        F.linear_backward_fp8_block(self.dev[3], self.x8c, self.sxc, self.w8, self.sw, self.m, self.k, self.n, FMT[fmt_g],
                                    FMT[fmt], *need, self.wb, self.nb, self.gx if need[0] else None,
                                    self.gw if need[1] else None, self.gb if need[2] else None, stream=stream)

    def oracle(self, fmt="e4m3", fmt_g="e5m2"):
        xv, wv, gv = (in_values_f32(t) for t in (self.x, self.w, self.g))
        q = lambda v, f, mode: OB.values(*OB.quantize(v, f, mode), f, mode)  # noqa: E731
        w = q(wv, fmt, "square")
        y = OB.product(q(xv, fmt, "rows"), w.T, in_values_f32(self.b).astype(np.float64))
        gx = OB.product(q(gv, fmt_g, "rows"), w)
        gw = OB.product(q(gv, fmt_g, "columns").T, q(xv, fmt, "columns"))
        return y, gx, gw, gv.astype(np.float64)

    def check(self, fmt="e4m3", fmt_g="e5m2", need=(1, 1, 1)):
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        y, gx, gw, g = self.oracle(fmt, fmt_g)
        _within(self.y, *y, self.k, "y")
        if need[0]:
            _within(self.gx, *gx, self.n, "grad_x")
        if need[1]:
            _within(self.gw, *gw, self.m, "grad_w")
        if need[2]:
            ref = g.sum(0)
            err = np.abs(bf16_out_to_f64(self.gb) - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (self.m + 1) * 2.0 ** -24 * np.abs(g).sum(0)).all()


@pytest.mark.parametrize("m,k,n", [(1, 16, 16), (3, 256, 144), (64, 512, 1024), (130, 272, 400), (512, 1024, 1024),
                                   (777, 1040, 528), (1024, 384, 2064), (2048, 1024, 4096)])
@pytest.mark.parametrize("fmt_g", ["e4m3", "e5m2"])
def test_training_step(m, k, n, fmt_g):
    layer = Layer(m, k, n)
    layer.forward()
    layer.backward(fmt_g)
    layer.check(fmt_g=fmt_g)
    codes, s = OB.quantize(in_values_f32(layer.w), "e4m3", "square")
    assert np.array_equal(np_u8(layer.w8), codes)
    _same_scale(layer.sw, s)
    codes, s = OB.quantize(in_values_f32(layer.x), "e4m3", "columns")
    assert np.array_equal(np_u8(layer.x8c), codes)
    _same_scale(layer.sxc, s)


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)])
def test_selected_gradients(need):
    layer = Layer(200, 256, 384, seed=2)
    layer.forward()
    layer.backward(need=need)
    layer.check(need=need)


@pytest.mark.parametrize("m", [1, 2, 7, 16, 17, 40, 64, 65, 300])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_serving_forward_with_an_fp8_weight(m, fmt):
    """The same numbers from an FP8 weight (a few rows: the product quantizes x itself) as from a bf16 one."""
    layer = Layer(m, 1024, 528, seed=4)
    layer.forward(fmt)
    x, _, b, _ = layer.dev
    y = torch.full_like(layer.y, 9.0)
    F.linear_forward_fp8_block(x, layer.w8, 1, layer.sw, b, m, 1024, 528, FMT[fmt], None, None, None, None, layer.wf, layer.nf, y)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    ref = layer.oracle(fmt)[0]
    _within(layer.y, *ref, 1024, "y from bf16 w")
    _within(y, *ref, 1024, "y from fp8 w")
    flat = torch.zeros(m * 1024 + 8, dtype=torch.bfloat16, device=DEV)
    flat[3:3 + m * 1024] = x.reshape(-1)   # rows that are only 2-byte aligned
    z = torch.full_like(layer.y, 9.0)
    F.linear_forward_fp8_block(flat[3:], layer.w8, 1, layer.sw, b, m, 1024, 528, FMT[fmt], None, None, None, None, layer.wf, layer.nf, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)


def test_empty_sizes():
    layer = Layer(0, 128, 64)
    layer.forward()
    layer.backward()
    torch.cuda.synchronize()
    assert (layer.gw == 0).all() and (layer.gb == 0).all()
    codes, _ = OB.quantize(in_values_f32(layer.w), "e4m3", "square")
    assert np.array_equal(np_u8(layer.w8), codes)
    layer = Layer(5, 0, 64)
    layer.forward()
    layer.backward()
    torch.cuda.synchronize()
    assert torch.equal(layer.y.cpu(), layer.b.expand(5, 64))
    Layer(5, 64, 0).forward()
    layer = Layer(5, 64, 0)
    layer.backward()
    torch.cuda.synchronize()
    assert (layer.gx == 0).all()


def test_captured_step_and_two_streams():
    """A forward and backward captured into a graph replay to the same bits as eager calls, with new data in
    the captured buffers as well, and two layers on two streams do not disturb one another."""
    layer, other = Layer(300, 512, 640, seed=6), Layer(256, 640, 384, seed=7)
    for one in (layer, other):
        one.forward()
        one.backward()
    torch.cuda.synchronize()
    want = [[t.clone() for t in (one.y, one.gx, one.gw, one.gb)] for one in (layer, other)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        layer.forward()
        layer.backward()
    for t in (layer.y, layer.gx, layer.gw, layer.gb):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((layer.y, layer.gx, layer.gw, layer.gb), want[0]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, one in zip(streams, (layer, other)):
            one.forward(stream=st)
            one.backward(stream=st)
    torch.cuda.synchronize()
    for one, w in zip((layer, other), want):
        assert all(torch.equal(a, b) for a, b in zip((one.y, one.gx, one.gw, one.gb), w))
    layer.dev[0].mul_(2)  # x doubles: so does y - b (every scale doubles exactly)
    graph.replay()
    torch.cuda.synchronize()
    layer.x = (layer.x.float() * 2).to(torch.bfloat16)
    layer.check()


def test_gradients_against_differences():
    """grad_x and grad_w of L = sum(g * y) against central differences of the fp64 layer (unquantized):
    quantization to 3 or 2 mantissa bits moves a gradient by at most half a step of either operand,
    2^-4 + 2^-3 of sum |terms| here (E4M3 with E5M2), and the sum's terms are independent."""
    m, k, n = 24, 128, 144
    layer = Layer(m, k, n, seed=8)
    layer.forward()
    layer.backward()
    torch.cuda.synchronize()
    x, w, g = (in_values_f32(t).astype(np.float64) for t in (layer.x, layer.w, layer.g))
    loss = lambda a, b: float((g * (a @ b.T)).sum())  # noqa: E731
    rng = np.random.default_rng(0)
    for got, which, terms in ((layer.gx, 0, np.abs(g) @ np.abs(w)), (layer.gw, 1, np.abs(g).T @ np.abs(x))):
        got = bf16_out_to_f64(got)
        for _ in range(20):
            i, j = rng.integers(got.shape[0]), rng.integers(got.shape[1])
            d = []
            for s in (1, -1):
                a, b = x.copy(), w.copy()
                (a if which == 0 else b)[i, j] += s * 0.5
                d.append(loss(a, b))
            assert abs((d[0] - d[1]) - got[i, j]) <= (2.0 ** -4 + 2.0 ** -3 + 2.0 ** -7) * terms[i, j] + 2.0 ** -8 * abs(got[i, j])

"""The block-scaled entry points without a GPU: argument checks run before any CUDA call."""

import ctypes

import pytest

import fp8_delayed_scaling_amax_b200 as F

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -5


def test_quantize_block_checks():
    q = F.lib().fp8_quantize_block
    ok = dict(x=256, t=0, r=4, c=32, f=0, o=512, s=1024, oc=None, sc=None)

    def call(**kw):
        d = dict(ok, **kw)
        return q(d["x"], d["t"], d["r"], d["c"], d["f"], d["o"], d["s"], d["oc"], d["sc"], None)
    assert call(t=5) == INVALID
    assert call(f=2) == INVALID
    assert call(r=-1) == INVALID
    assert call(x=None) == INVALID
    assert call(o=None, s=None) == INVALID          # no output at all
    assert call(s=None) == INVALID                  # bytes without their scales
    assert call(oc=4096) == INVALID
    assert call(x=257) == UNSUPPORTED               # not aligned to bf16
    assert call(s=1026) == UNSUPPORTED
    assert call(t=2, x=258) == UNSUPPORTED
    b = F.lib().fp8_quantize_block128
    assert b(256, 0, 4, 32, 0, 512, None, None) == INVALID
    assert b(None, 0, 4, 32, 0, 512, 1024, None) == INVALID
    assert b(256, 0, 4, -32, 0, 512, 1024, None) == INVALID
    assert b(255, 0, 4, 32, 0, 512, 1024, None) == UNSUPPORTED
    assert "x" in F.last_error()


def _scale(p=4096, block=1, mn=1, kb=32, bt=0):
    return F.fp8_block_scale_t(p, block, mn, kb, bt)


def test_gemm_block_checks():
    g = F.lib().fp8_gemm_block
    ok = dict(a=256, b=512, fa=0, fb=0, lay=0, m=32, n=32, k=32, lda=32, ldb=32, ldo=32, batch=1, sa=0, sb=0, so=0,
              pa=_scale(), pb=_scale(block=128), bias=None, out=1024)

    def call(**kw):
        d = dict(ok, **kw)
        p = [None if d[x] is None else ctypes.byref(d[x]) for x in ("pa", "pb")]
        return g(d["a"], d["b"], d["fa"], d["fb"], d["lay"], d["m"], d["n"], d["k"], d["lda"], d["ldb"], d["ldo"],
                 d["batch"], d["sa"], d["sb"], d["so"], p[0], p[1], d["bias"], d["out"], None)
    assert call(fa=3) == INVALID
    assert call(lay=9) == INVALID
    assert call(m=-1) == INVALID
    assert call(out=None) == INVALID
    assert call(pa=None) == INVALID
    assert call(pb=_scale(p=None)) == INVALID
    assert call(pa=_scale(block=64)) == INVALID
    assert "block_mn" in F.last_error()
    assert call(pa=_scale(kb=-1)) == INVALID
    assert call(pa=_scale(p=4098)) == UNSUPPORTED
    assert call(ldo=16) == INVALID
    assert call(lda=16) == INVALID
    assert call(lda=40) == UNSUPPORTED
    assert call(a=257) == UNSUPPORTED
    assert call(out=1025) == UNSUPPORTED
    assert call(m=1 << 31) == UNSUPPORTED
    assert call(ldo=1 << 40) == UNSUPPORTED
    assert call(batch=2, so=100) == INVALID            # batches overlap
    assert call(batch=2, sa=8, so=2048) == UNSUPPORTED
    assert call(batch=2, sa=-16, so=2048) == INVALID


def test_linear_block_checks():
    lib = F.lib()
    nf = F.linear_forward_fp8_block_workspace_size(64, 64, 64)
    assert nf >= 2 * 64 * 64 and nf % 256 == 0
    assert F.linear_forward_fp8_block_workspace_size(-1, 64, 64) == 0
    assert F.linear_forward_fp8_block_workspace_size(1 << 31, 64, 64) == 0
    ok = dict(x=256, w=512, f8=0, ws=None, b=None, m=64, k=64, n=64, f=0, w8=None, w8s=None, xc=None, xs=None, work=1024,
              nb=nf, y=2048)

    def fwd(**kw):
        d = dict(ok, **kw)
        return lib.linear_forward_fp8_block(d["x"], d["w"], d["f8"], d["ws"], d["b"], d["m"], d["k"], d["n"], d["f"],
                                            d["w8"], d["w8s"], d["xc"], d["xs"], d["work"], d["nb"], d["y"], None)
    assert fwd(f=2) == INVALID
    assert fwd(k=60) == UNSUPPORTED
    assert fwd(m=-1) == INVALID
    assert fwd(m=1 << 31) == UNSUPPORTED
    assert fwd(work=None) == INVALID
    assert fwd(work=1040) == UNSUPPORTED
    assert fwd(nb=nf - 1) == WORKSPACE
    assert fwd(x=None) == INVALID
    assert fwd(y=None) == INVALID
    assert fwd(f8=1) == INVALID                       # fp8 weight without scales
    assert fwd(f8=1, ws=4096, w8=8192, w8s=4096) == INVALID
    assert fwd(w8=8192) == INVALID                    # bytes without their scales
    assert fwd(xc=8192) == INVALID
    assert fwd(w8=8200, w8s=4096) == UNSUPPORTED
    assert fwd(f8=1, ws=4096, w=520) == UNSUPPORTED   # fp8 weight not 16-byte aligned
    nb = F.linear_backward_fp8_block_workspace_size(64, 64, 64)
    okb = dict(g=256, xc=512, xs=512, w8=1024, ws=512, m=64, k=64, n=64, fg=1, f=0, nx=1, nw=1, nb_=1, work=1024, nb=nb,
               gx=256, gw=256, gb=256)

    def bwd(**kw):
        d = dict(okb, **kw)
        return lib.linear_backward_fp8_block(d["g"], d["xc"], d["xs"], d["w8"], d["ws"], d["m"], d["k"], d["n"], d["fg"],
                                             d["f"], d["nx"], d["nw"], d["nb_"], d["work"], d["nb"], d["gx"], d["gw"],
                                             d["gb"], None)
    assert bwd(fg=3) == INVALID
    assert bwd(g=None) == INVALID
    assert bwd(w8=None) == INVALID
    assert bwd(ws=None) == INVALID
    assert bwd(xc=None) == INVALID
    assert bwd(gx=None) == INVALID
    assert bwd(gw=None) == INVALID
    assert bwd(gb=None) == INVALID
    assert bwd(n=72) == UNSUPPORTED
    assert bwd(xc=520) == UNSUPPORTED
    assert bwd(nb=nb - 1) == WORKSPACE


def test_moe_checks():
    size = F.moe_forward_fp8_block_workspace_size
    n = size(4, 2, 8, 256, 128)
    assert n >= 8 * 128 + 8 * 4 and n % 256 == 0
    for bad in ((65, 2, 8, 256, 128), (4, 33, 8, 256, 128), (4, 2, 1025, 256, 128), (4, 2, 8, 250, 128), (4, 2, 8, 256, 8),
                (-1, 2, 8, 256, 128)):
        assert size(*bad) == 0
    ok = dict(x=256, ids=256, w=256, t=4, tk=2, e=8, h=256, i=128, f=0, w13=512, s13=512, w2=512, s2=512, ws=1024, nb=n, o=256)

    def call(**kw):
        d = dict(ok, **kw)
        return F.lib().moe_forward_fp8_block(d["x"], d["ids"], d["w"], d["t"], d["tk"], d["e"], d["h"], d["i"], d["f"],
                                             d["w13"], d["s13"], d["w2"], d["s2"], d["ws"], d["nb"], d["o"], None)
    assert call(f=2) == INVALID
    assert call(t=-1) == INVALID
    assert call(tk=0) == INVALID
    assert call(t=65) == UNSUPPORTED
    assert call(h=248) == UNSUPPORTED
    assert call(e=1025) == UNSUPPORTED
    assert call(w13=None) == INVALID
    assert call(s2=None) == INVALID
    assert call(w2=520) == UNSUPPORTED
    assert call(ids=258) == UNSUPPORTED
    assert call(x=None) == INVALID
    assert call(o=None) == INVALID
    assert call(ws=None) == INVALID
    assert call(ws=1040) == UNSUPPORTED
    assert call(nb=n - 1) == WORKSPACE


@pytest.mark.parametrize("name", ["fp8_quantize_block", "fp8_quantize_block128", "fp8_gemm_block", "linear_forward_fp8_block",
                                  "linear_backward_fp8_block", "moe_forward_fp8_block"])
def test_header_declares_what_the_binding_binds(name):
    assert name in F.header_functions() and hasattr(F, name)

"""GPU: CTAs of the block-scaled streaming kernels that can share an SM never want more than its 512 columns of
tensor memory, by the shared memory their launches take (read from captured graphs; nothing is made to wait)."""

import ctypes

import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
TMEM_COLUMNS = 512
# columns that a CTA of the streaming kernels allocates, by its threads: 16 token columns, and 64
COLUMNS = {288: 256, 480: 512}


class _KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "smem")] + [
        (n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")]


def _launches(call):
    """(threads, dynamic shared memory) of every kernel that `call(stream)` launches."""
    cuda = ctypes.CDLL("libcuda.so.1")
    graph, side = torch.cuda.CUDAGraph(keep_graph=True), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    handle, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cuda.cuGraphGetNodes(handle, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(handle, nodes, ctypes.byref(n)) == 0
    found = []
    for node in nodes:
        kind = ctypes.c_int(-1)
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:  # a kernel
            p = _KernelNode()
            assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            found.append((p.bx * p.by * p.bz, p.smem))
    return found


def _attribute(which):
    cuda, v = ctypes.CDLL("libcuda.so.1"), ctypes.c_int(0)
    assert cuda.cuDeviceGetAttribute(ctypes.byref(v), which, torch.cuda.current_device()) == 0
    return v.value


def _zeros(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def _product(m, n, k):
    kb, nb = -(-k // 128), -(-n // 128)
    a, b, out = _zeros(m, k), _zeros(n, k), _zeros(m, n, dtype=torch.bfloat16)
    sa, sb = F.BlockScale(torch.ones(kb, m, device=DEV), 1, 1, m), F.BlockScale(torch.ones(nb, kb, device=DEV), 128, kb, 1)
    return lambda st: F.fp8_gemm_block(a, b, F.FP8_E4M3, F.FP8_E4M3, F.FP8_LAYOUT_NT, m, n, k, k, k, n, 1, 0, 0, m * n, sa, sb,
                                       None, out, stream=st)


def _serving(m, n, k):
    x, w, y = _zeros(m, k, dtype=torch.bfloat16), _zeros(n, k), _zeros(m, n, dtype=torch.bfloat16)
    s = torch.ones(-(-n // 128), -(-k // 128), device=DEV)
    nbytes = F.linear_forward_fp8_block_workspace_size(m, k, n)
    ws = _zeros(nbytes)
    return lambda st: F.linear_forward_fp8_block(x, w, 1, s, None, m, k, n, F.FP8_E4M3, None, None, None, None, ws, nbytes, y,
                                                 stream=st)


def _experts(tokens, topk, experts, hidden, inter):
    x, out = _zeros(tokens, hidden, dtype=torch.bfloat16), _zeros(tokens, hidden, dtype=torch.bfloat16)
    ids, wts = _zeros(tokens, topk, dtype=torch.int32), _zeros(tokens, topk, dtype=torch.float32)
    hb, ib = -(-hidden // 128), -(-inter // 128)
    w13, w2 = _zeros(experts, 2 * inter, hidden), _zeros(experts, hidden, inter)
    s13, s2 = torch.ones(experts, 2, ib, hb, device=DEV), torch.ones(experts, hb, ib, device=DEV)
    nbytes = F.moe_forward_fp8_block_workspace_size(tokens, topk, experts, hidden, inter)
    ws = _zeros(nbytes)
    return lambda st: F.moe_forward_fp8_block(x, ids, wts, tokens, topk, experts, hidden, inter, F.FP8_E4M3, w13, s13, w2, s2, ws,
                                              nbytes, out, stream=st)


CALLS = [(_product, (1, 128, 128)), (_product, (1, 1024, 384)), (_product, (16, 4096, 1024)), (_product, (17, 128, 128)),
         (_product, (64, 1024, 640)), (_product, (64, 8192, 2048)), (_serving, (1, 128, 128)), (_serving, (16, 1024, 2048)),
         (_experts, (1, 1, 1, 128, 128)), (_experts, (1, 2, 8, 1024, 512)), (_experts, (40, 4, 8, 256, 144))]


def test_streaming_ctas_never_want_more_tensor_memory_than_an_sm_has():
    per_sm, reserved = _attribute(81), _attribute(111)  # shared memory of a multiprocessor, and the system's part per CTA
    found = []
    for make, sizes in CALLS:
        call = make(*sizes)
        call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert F.fp8_get_device_status() == 0
        mine = [x for x in _launches(call) if x[0] in COLUMNS]
        assert mine, (make.__name__, sizes)
        found += [(COLUMNS[t], s + reserved) for t, s in mine]
    assert {c for c, _ in found} == set(COLUMNS.values())
    least = {c: min(s for x, s in found if x == c) for c in set(COLUMNS.values())}
    # any mix of a halves and b wholes that fits an SM's shared memory fits its TMEM
    for a in range(5):
        for b in range(3):
            if a * least[256] + b * least[512] <= per_sm:
                assert a * 256 + b * 512 <= TMEM_COLUMNS, (a, b, least)

"""GPU: a token's experts are added in the experts' order, so the order in which a router lists them does not show in a
single bit of the output."""

import itertools

import numpy as np
import pytest
import torch

import fp8_delayed_scaling_amax_b200 as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _codes(rng, *shape):
    q = rng.integers(0, 256, shape, dtype=np.uint8)
    q[(q & 0x7F) == 0x7F] = 0x38  # no NaN codes
    return torch.from_numpy(q).to(DEV)


def _run(x, ids, wts, packed, experts, inter):
    tokens, hidden = x.shape
    topk = ids.shape[1]
    nbytes = F.moe_forward_fp8_block_workspace_size(tokens, topk, experts, hidden, inter)
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((tokens, hidden), 7.0, dtype=torch.bfloat16, device=DEV)
    F.moe_forward_fp8_block(x, ids.contiguous(), wts.contiguous(), tokens, topk, experts, hidden, inter, F.FP8_E4M3, *packed, ws,
                            nbytes, out)
    torch.cuda.synchronize()
    assert F.fp8_get_device_status() == 0
    return out


@pytest.mark.parametrize("tokens", [1, 8, 9, 40])
@pytest.mark.parametrize("hidden,inter", [(256, 144), (1024, 512)])
def test_the_order_of_a_tokens_slots_does_not_show(tokens, hidden, inter):
    """Experts that are copies of one another, weighted by 1, 2^-26 and -1: added in another order, the small one is lost or
    kept (32 pairs and fewer are sorted in another way than more)."""
    rng = np.random.default_rng(tokens)
    experts, picked = 12, (2, 5, 11)
    w13, w2 = _codes(rng, 1, 2 * inter, hidden).repeat(experts, 1, 1), _codes(rng, 1, hidden, inter).repeat(experts, 1, 1)
    ib, hb = -(-inter // 128), -(-hidden // 128)
    s13, s2 = torch.full((experts, 2, ib, hb), 2.0 ** -12, device=DEV), torch.full((experts, hb, ib), 2.0 ** -8, device=DEV)
    x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    ids = torch.tensor(picked, dtype=torch.int32, device=DEV).repeat(tokens, 1)
    for values in ((1.0, 2.0 ** -26, -1.0), (1.0, -1.0, 2.0 ** -26)):
        wts = torch.tensor(values, device=DEV).repeat(tokens, 1)
        want = _run(x, ids, wts, (w13, s13, w2, s2), experts, inter)
        for order in itertools.permutations(range(3)):
            got = _run(x, ids[:, order], wts[:, order], (w13, s13, w2, s2), experts, inter)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)), (values, order)


@pytest.mark.parametrize("tokens,topk,experts", [(1, 32, 64), (4, 8, 8), (3, 10, 1024), (16, 2, 5), (33, 6, 40)])
def test_shuffled_slots(tokens, topk, experts):
    rng = np.random.default_rng(topk)
    hidden, inter = 512, 256
    packed = (_codes(rng, experts, 2 * inter, hidden), torch.full((experts, 2, 2, 4), 2.0 ** -12, device=DEV),
              _codes(rng, experts, hidden, inter), torch.full((experts, 4, 2), 2.0 ** -8, device=DEV))
    x = torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    # distinct experts, some slots skipped
    picked = np.stack([rng.permutation(experts)[:topk] for _ in range(tokens)]).astype(np.int32)
    picked[rng.random(picked.shape) < 0.2] = -1
    ids = torch.from_numpy(picked).to(DEV)
    wts = torch.from_numpy(rng.standard_normal((tokens, topk)).astype(np.float32)).to(DEV)
    want = _run(x, ids, wts, packed, experts, inter)
    assert torch.isfinite(want).all()
    for _ in range(4):
        at = torch.from_numpy(np.stack([rng.permutation(topk) for _ in range(tokens)])).to(DEV)
        got = _run(x, ids.gather(1, at), wts.gather(1, at), packed, experts, inter)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))

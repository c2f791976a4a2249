"""Calls of the 8-bit block operators at the edges of what they promise."""
import pytest
import torch

import block8_oracle as O

pytestmark = pytest.mark.gpu

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from conv_bn_silu_amd import block8
    return block8


@pytest.mark.parametrize("held", [I8, BF16], ids=["i8", "bf16"])
def test_shared_slots_harm_no_others(ops, held):
    """Of a slot that two tokens name, nothing is promised; the slots that one names hold what they should."""
    T, H, D, P = 600, 3, 64, 16
    g = torch.Generator().manual_seed(3)
    k = (torch.randn(T, H, D, generator=g) * 10.0 ** torch.randint(-3, 4, (T, 1, 1), generator=g)).to(BF16)
    slots = torch.randperm(700, generator=g)[:T].to(torch.int32)
    slots[100:200] = slots[:100]
    shared = torch.zeros(T, dtype=torch.bool)
    shared[:200] = True
    cache = ops.PagedCache.empty(50, H, P, D, held)
    ops.cache_write(cache, k.cuda(), k.cuda(), slots.cuda())
    codes, s = O.quantize(k)
    want = (codes.float() * s[..., None]).to(BF16) if held == I8 else k
    for y in ops.cache_read(cache, slots.cuda()):
        assert torch.equal(y[~shared].cpu(), want[~shared])
    unnamed = torch.ones(800, dtype=torch.bool)
    unnamed[slots.long()] = False
    assert bool((ops.cache_read(cache, unnamed.nonzero()[:, 0].to(torch.int32).cuda())[0] == 0).all())

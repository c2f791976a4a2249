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


def test_a_cache_keeps_its_tensors(ops):
    """The memory that the kernels are given is not freed while the cache lives, and a cache whose tensors
    have been given other memory is refused."""
    dev = dict(device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    cache = ops.PagedCache.empty(64, 2, 16, 64)
    held = torch.cuda.memory_allocated() - before
    record = cache._record
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros_like(getattr(cache, name)))
    del cache
    assert torch.cuda.memory_allocated() - before == held > 64 * 2 * 16 * 64 * 2
    del record
    assert torch.cuda.memory_allocated() == before

    slots = torch.zeros(1, dtype=torch.int32, **dev)
    x = torch.zeros(1, 2, 64, dtype=BF16, **dev)
    i32 = dict(dtype=torch.int32, **dev)
    for name in ("k", "v", "k_scale", "v_scale"):
        for how in ("data", "set_", "resize_"):
            cache = ops.PagedCache.empty(64, 2, 16, 64)
            t = getattr(cache, name)
            old = t.detach()
            if how == "data":
                t.data = torch.zeros_like(t)
            elif how == "set_":
                t.set_(torch.zeros_like(t))
            else:
                t.resize_(0)
            for call in (lambda: ops.cache_write(cache, x, x, slots), lambda: ops.cache_read(cache, slots),
                         lambda: ops.paged_attention(x, cache, torch.zeros(1, 1, **i32), torch.tensor([0, 1], **i32),
                                                     torch.ones(1, **i32))):
                with pytest.raises(ValueError, match="other memory"):
                    call()
            del old


def test_conv_on_another_device(monkeypatch):
    """Calls take the current device's handle and stream, and so tensors that lie there."""
    from conv_bn_silu_amd import binding as B
    x, w, s = torch.ones(1, 4, 8, 8, device="cuda"), torch.ones(4, 4, 1, 1, device="cuda"), torch.ones(4, device="cuda")
    B.conv_bn_silu(x, w, s, s)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (B.conv_bn_silu, B.conv_bn_silu_unfused, B.conv_bn_silu_unfused_noalloc):
        with pytest.raises(ValueError, match="current device"):
            call(x, w, s, s)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_tensors_of_another_device(ops):
    def on(d):
        dev = dict(device=f"cuda:{d}")
        i32 = dict(dtype=torch.int32, **dev)
        x = torch.zeros(1, 2, 64, dtype=BF16, **dev)
        cache = torch.zeros(4, 2, 16, 64, dtype=BF16, **dev)
        return (lambda: ops.int8_linear(x, torch.zeros(8, 64, dtype=I8, **dev), torch.zeros(8, **dev)),
                lambda c: ops.cache_write(c, x, x, torch.zeros(1, **i32)), lambda c: ops.cache_read(c, torch.zeros(1, **i32)),
                lambda c: ops.paged_attention(x, c, torch.zeros(1, 1, **i32), torch.tensor([0, 1], **i32), torch.ones(1, **i32)),
                cache)

    linear, *calls, k = on(1)
    with pytest.raises(ValueError, match="current device"):
        linear()
    cache = ops.PagedCache(k, k.clone())
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call(cache)


def test_tangents_are_refused(ops):
    from torch.autograd import forward_ad
    i32 = dict(dtype=torch.int32, device="cuda")
    x, w, s = torch.zeros(2, 64, device="cuda"), torch.zeros(8, 64, dtype=I8, device="cuda"), torch.zeros(8, device="cuda")
    cache, slots = ops.PagedCache.empty(4, 2, 16, 64, BF16), torch.zeros(1, **i32)
    k = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    with forward_ad.dual_level():
        def dual(t):
            return forward_ad.make_dual(t, torch.ones_like(t))
        for call in (lambda: ops.int8_linear(dual(x), w, s), lambda: ops.int8_linear(x, w, dual(s)),
                     lambda: ops.int8_linear(x, w, s, bias=dual(s)), lambda: ops.cache_write(cache, k, dual(k), slots),
                     lambda: ops.paged_attention(dual(k), cache, torch.zeros(1, 1, **i32), torch.tensor([0, 1], **i32),
                                                 torch.ones(1, **i32))):
            with pytest.raises(ValueError, match="tangent"):
                call()
    assert tuple(ops.int8_linear(x, w, s).shape) == (2, 8)

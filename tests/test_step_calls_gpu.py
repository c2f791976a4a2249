"""Calls that the documentation allows or refuses, beside those of test_step_gpu.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64, I8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import conv_bn_silu_amd
    return conv_bn_silu_amd


def test_a_wrong_sum_is_called_by_its_name(ops):
    x, r = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.zeros(4, 64, dtype=BF16, device="cuda")
    with pytest.raises(TypeError, match="^sum_out"):
        ops.add_rms_norm(x, None, r, sum_out=torch.zeros(4, 64, device="cuda"))
    for bad in (r[:3], torch.zeros(4, 128, dtype=BF16, device="cuda")[:, ::2], r.cpu()):
        with pytest.raises(ValueError, match="^sum_out"):
            ops.add_rms_norm(x, None, r, sum_out=bad)
    with pytest.raises(ValueError, match="^out"):
        ops.add_rms_norm(x, None, r, out=r[:3])


def test_a_step_in_inference_mode(ops):
    """Outputs made there serve there and outside, growth's three parts of one allocation among them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(5, 8, 64, generator=g, device="cuda").to(BF16)
    f = ops.rotary_frequencies(64)

    def run():
        pool, cache = ops.PagePool.full(8, 4), ops.PagedCache.empty(8, 2, 4, 64)
        table, lens = torch.full((2, 4), -1, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
        starts, slots, positions = ops.grow_pages(pool, table, lens, torch.tensor([3, 2], dtype=I32, device="cuda"), 5)
        return pool, cache, table, lens, starts, slots, positions

    def rest(pool, cache, table, lens, starts, slots, positions):
        q = ops.rotary_cache_write(cache, x[:, :4], x[:, 4:6], x[:, 6:], positions, slots, f)
        a = ops.paged_attention(q, cache, table, starts, lens)
        rows, h = ops.add_rms_norm(a.view(5, -1), None, x[:, :4].reshape(5, -1), int8=True)
        ops.release_pages(pool, table, lens, torch.zeros(2, dtype=I32, device="cuda"))
        return [starts, slots, positions, q, a, rows.codes, rows.scale, h, table, lens, pool.free, pool.counts]

    want = rest(*run())
    with torch.inference_mode():
        inside = run()
        got = rest(*inside)
        half = run()
    assert inside[4].is_inference() and all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(want, rest(*half)))
    starts, slots, positions = half[4:]
    assert starts.untyped_storage().data_ptr() == positions.untyped_storage().data_ptr()
    slots.clone().fill_(7), positions.clone().fill_(7)
    assert torch.equal(starts, want[0]) and torch.equal(torch.stack((slots, positions)), torch.stack(want[1:3]))


def test_parts_of_a_projection_with_heads_are_normalised(ops):
    """Heads that lie in a wider tensor are no rows one distance apart: copied, and the same as of a copy; so is the residual."""
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(7, 12, 64, generator=g, device="cuda").to(BF16)
    before, w = wide.clone(), torch.rand(64, generator=g, device="cuda")
    for x, r in ((wide[:, :5], None), (wide[:, 2:7], wide[:, 7:]), (wide.transpose(0, 1), None)):
        want, got = (ops.add_rms_norm(a, w, b) for a, b in ((x.contiguous(), None if r is None else r.contiguous()), (x, r)))
        for a, b in [(want, got)] if r is None else zip(want, got):
            assert a.shape == x.shape and torch.equal(a, b)
        assert torch.equal(wide, before)

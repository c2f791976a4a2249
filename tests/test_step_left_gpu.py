"""A step in which some sequences find no room: the others' tokens, and all that is kept, are as they would be without them."""
import pytest
import torch

import block8_oracle as O

pytestmark = pytest.mark.gpu

BF16, F64, I32 = torch.bfloat16, torch.float64, torch.int32


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# table's width, spare pages of the pool, which sequences are left: the second alone where its row of the table is full (the
# spare page then goes to the third), else the first that lacks a page and all after it
@pytest.mark.parametrize("width,spare,left", [(3, 9, [1]), (9, 1, [2, 3, 4]), (3, 1, [1, 3, 4]), (9, 0, [1, 2, 3, 4])], ids=str)
def test_a_step_with_sequences_left(width, spare, left):
    import conv_bn_silu_amd as ops
    print("[left]", width, spare, left, flush=True)
    H, Hk, D, P = 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)  # noqa: E731
    old, more = [20, 48, 31, 0, 16], [1, 1, 2, 1, 2]
    taken = sum(-(-n // P) for n in old)
    cache = ops.PagedCache.empty(taken + spare, Hk, P, D, BF16)
    cache.k.zero_(), cache.v.zero_()
    pool = ops.PagePool.full(taken + spare, P)
    table, lens = torch.full((5, width), -1, dtype=I32, device="cuda"), i32([0] * 5)
    f = ops.rotary_frequencies(D)

    def enter(new, tokens):
        starts, slots, positions = ops.grow_pages(pool, table, lens, i32(new), tokens)
        q, k, v = normal(tokens, H, D), normal(tokens, Hk, D), normal(tokens, Hk, D)
        q = ops.rotary_cache_write(cache, q, k, v, positions, slots, f)
        return starts, slots, q, ops.paged_attention(q, cache, table, starts, lens)

    def check(starts, q, out, rows):
        ref, tol, _ = O.attention(q.cpu(), cache.k.cpu().to(F64), cache.v.cpu().to(F64), table.cpu(), starts.tolist(), lens.tolist(),
                                  0, D ** -0.5, O.half_step(BF16))
        O.check(out[rows], ref[rows.cpu()], tol[rows.cpu()], "rows with a slot")

    enter(old, sum(old))
    assert pool.report() == (spare, 0, 0)
    before = [t.clone() for t in (table, cache.k, cache.v)]
    starts, slots, q, out = enter(more, sum(more))
    assert pool.report()[2] == len(left) and lens.tolist() == [n + (0 if b in left else m) for b, (n, m) in enumerate(zip(old, more))]
    there = torch.tensor([b not in left for b, m in enumerate(more) for _ in range(m)], device="cuda")
    assert torch.equal(slots >= 0, there)
    if bool(there.any()):
        check(starts, q, out, there)
    out.masked_fill_((slots < 0)[:, None, None], 0)
    assert not bool(out[~there].any())
    # nothing of the others was touched
    assert torch.equal(table[left], before[0][left])
    free = torch.ones(cache.k.shape[0], P, dtype=torch.bool, device="cuda")
    free[slots[there].long() // P, slots[there].long() % P] = False
    for t, was in zip((cache.k, cache.v), before[1:]):
        assert torch.equal(t.transpose(1, 2)[free], was.transpose(1, 2)[free])
    # the first ends, and the first that found no page brings its tokens again
    short = [b for b in left if not (b == 1 and width == 3)]
    keep = [0 if b == 0 else 2 ** 31 - 1 for b in range(5)]
    ops.release_pages(pool, table, lens, i32(keep))
    new = [more[b] if b in short[:1] else 0 for b in range(5)]
    starts, slots, q, out = enter(new, sum(new))
    assert pool.report()[2] == 0 and bool((slots >= 0).all())
    if short:
        check(starts, q, out, slots >= 0)

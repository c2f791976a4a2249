"""A step's other operators at large sizes: more rows and tokens than a launch takes, offsets past 32 bits, the most
sequences."""
import pytest
import torch

import block8_oracle as O
import step_oracle as S

pytestmark = pytest.mark.gpu

BF16, F32, F64, I8, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int8, torch.int32


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import conv_bn_silu_amd
    yield conv_bn_silu_amd
    torch.cuda.empty_cache()


def say(*a):
    print(*a, flush=True)


def rows_at(n, borders):
    """Rows to compare: both ends, those around the borders, and some between."""
    g = torch.Generator().manual_seed(n)
    some = torch.randint(0, n, (40,), generator=g).tolist()
    near = [b + d for b in borders for d in (-2, -1, 0, 1, 2)]
    return torch.tensor(sorted({r for r in [0, 1, n - 2, n - 1, *near, *some] if 0 <= r < n}))


@pytest.mark.parametrize("M,K", [(2 ** 21 + 3, 2056), (2 ** 24, 72), (2 ** 22 + 1, 520), (2 ** 21 + 70, 1001)], ids=str)
def test_norm_most_rows(ops, M, K):
    """Several launches; 4.3 billion values in the first, so that its later rows lie past 2^32 of them."""
    g = torch.Generator(device="cuda").manual_seed(K)
    say("[norm rows]", M, K)
    x = torch.empty(M, K, dtype=BF16, device="cuda").normal_(generator=g)
    r = torch.empty(M, K, dtype=BF16, device="cuda").normal_(generator=g)
    w = 1 + 0.1 * torch.randn(K, generator=g, device="cuda")
    at = rows_at(M, [2 ** 20, 2 ** 21, 2 ** 22, 2 ** 23, 2 ** 32 // K]).cuda()
    y, tol, h = S.norm(x[at].cpu(), w.cpu(), r[at].cpu(), 1e-6)
    before = r[at].clone()
    rows, s = ops.add_rms_norm(x, w, r, int8=True)
    assert torch.equal(s[at].cpu(), h)
    R, blocks = (M + 15) // 16 * 16, (K + 127) // 128 * 2
    codes = rows.buffer[4 * R:].view(blocks, R, 64)[:, at].transpose(0, 1).flatten(1)[:, :K]
    S.check_codes(codes, rows.buffer[:4 * R].view(F32)[at], y, tol, f"{M} {K}")
    del rows, s
    got, s = ops.add_rms_norm(x, w, r, sum_out=r)
    assert s is r and torch.equal(r[at].cpu(), h) and not torch.equal(before, r[at])
    O.check(got[at], y, O.rounded(y, tol, BF16), f"{M} {K}")
    # and no row between is left out: every one is what a smaller call makes of it
    for m0 in range(0, M, 2 ** 20):
        part = ops.add_rms_norm(r[m0:m0 + 2 ** 20], w)
        assert torch.equal(part, got[m0:m0 + 2 ** 20]), m0
    del x, r, s, got, part
    torch.cuda.empty_cache()


@pytest.mark.parametrize("heads,dim,pairs", [(16, 128, 64), (3, 36, 9)], ids=["pieces", "any"])
def test_rotary_most_tokens(ops, heads, dim, pairs):
    """More tokens than a launch takes, and 4.3 billion values; the keys and values of some enter a cache."""
    T = 2 ** 21 + 5
    say("[rotary tokens]", heads, dim, pairs)
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.empty(T, heads, dim, dtype=BF16, device="cuda").normal_(generator=g)
    pos = torch.arange(T, dtype=I32, device="cuda") * 7
    f = 10000.0 ** (-torch.arange(pairs, dtype=F64, device="cuda") / pairs)
    at = rows_at(T, [2 ** 20, 2 ** 21, 2 ** 32 // (heads * dim)]).cuda()
    ref, tol = S.rotate(x[at].cpu(), pos[at].cpu(), f.cpu(), False, 1.0)
    y = ops.rotary(x, pos, f)
    O.check(y[at], ref, O.rounded(ref, tol, BF16), "turned")
    for t0 in range(0, T, 2 ** 19):  # no token between is left out
        part = ops.rotary(x[t0:t0 + 2 ** 19], pos[t0:t0 + 2 ** 19], f)
        assert torch.equal(part, y[t0:t0 + 2 ** 19]), t0
    del part
    if dim % 8 == 0:
        slots = torch.full((T,), -1, dtype=I32, device="cuda")
        slots[at] = torch.randperm(at.numel(), generator=g, device="cuda").to(I32)
        cache = ops.PagedCache.empty(16, 2, 16, dim)
        q = ops.rotary_cache_write(cache, x[:, :heads - 4], x[:, heads - 4:heads - 2], x[:, heads - 2:], pos, slots, f)
        assert torch.equal(q, y[:, :heads - 4])
        where = slots[at].cpu().long()
        S.check_codes(cache.k.cpu()[where // 16, :, where % 16], cache.k_scale.cpu()[where // 16, :, where % 16],
                      ref[:, heads - 4:heads - 2], tol[:, heads - 4:heads - 2], "keys")
        codes, s = O.quantize(x[at, heads - 2:].cpu())
        assert torch.equal(cache.v.cpu()[where // 16, :, where % 16].double(), codes)
        del q
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
def test_rotary_past_32_bit_offsets(ops, interleaved):
    """Tensors whose tokens and heads lie far apart, and a cache of more than 2^31 values."""
    say("[rotary offsets]", interleaved)
    T, H, D, P = 5, 2, 64, 64
    wide = torch.zeros(T * (2 ** 30 + 24), dtype=BF16, device="cuda")
    x = wide.as_strided((T, H, D), (2 ** 30 + 24, 2 ** 29 + 8, 1))
    x.copy_(torch.randn(T, H, D, generator=torch.Generator().manual_seed(1)))
    pages = 2 ** 31 // (P * D) + 8
    cache = ops.PagedCache(*(torch.empty(pages, 1, P, D, dtype=I8, device="cuda") for _ in range(2)),
                           *(torch.zeros(pages, 1, P, device="cuda") for _ in range(2)))
    pos = torch.arange(T, dtype=I32) * 1000
    slots = torch.tensor([pages * P - 1, 5, (pages - 2) * P, -1, pages * P - 40], dtype=I32)
    f = 10000.0 ** (-torch.arange(32, dtype=F64) / 32)
    ref, tol = S.rotate(x.cpu(), pos, f, interleaved, 1.0)
    q = ops.rotary_cache_write(cache, x[:, :1], x[:, 1:], x[:, 1:], pos.cuda(), slots.cuda(), f.cuda(), interleaved)
    O.check(q, ref[:, :1], O.rounded(ref, tol, BF16)[:, :1], "queries")
    there = slots >= 0
    page, off = (slots[there].long() // P).cuda(), (slots[there].long() % P).cuda()
    S.check_codes(cache.k[page, :, off], cache.k_scale[page, :, off], ref[there, 1:], tol[there, 1:], "keys")
    ops.rotary(x, pos.cuda(), f.cuda(), interleaved, out=x)
    O.check(x, ref, O.rounded(ref, tol, BF16), "in place")
    del wide, x, cache
    torch.cuda.empty_cache()


def test_pages_most_sequences(ops):
    """65536 sequences, 30 million tokens; grown by prompts, by single tokens, cut back."""
    B, P, width = 65536, 16, 80
    say("[pages]", B)
    g = torch.Generator().manual_seed(5)
    more = torch.randint(0, 921, (B,), generator=g, dtype=I32)
    need = (more + P - 1) // P
    pages = int(need.sum()) + 40000
    pool = ops.PagePool.full(pages, P)
    table = torch.full((B, width), -1, dtype=I32, device="cuda")
    lens = torch.zeros(B, dtype=I32, device="cuda")
    tokens = int(more.sum()) + 100
    starts, slots, positions = ops.grow_pages(pool, table, lens, more.cuda(), tokens)
    assert pool.report() == (40000, 0, 0) and torch.equal(lens.cpu(), more)
    ends = more.long().cumsum(0)
    assert torch.equal(starts.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), ends]))
    # a full pool hands out pages 0, 1, ... in the order of the sequences
    first = (need.long().cumsum(0) - need).repeat_interleave(more.long())
    where = torch.arange(tokens - 100) - (ends - more).repeat_interleave(more.long())
    assert torch.equal(positions.cpu()[:-100].long(), where)
    assert torch.equal(slots.cpu()[:-100].long(), (first + where // P) * P + where % P)
    assert bool((slots[-100:] == -1).all()) and bool((positions[-100:] == 0).all())
    # a token each: those whose pages are full take one more, as long as there are any
    full = (more % P == 0)
    before = pool.report()[0]
    starts, slots, positions = ops.grow_pages(pool, table, lens, torch.ones(B, dtype=I32, device="cuda"), B)
    taken = int(full.sum())
    assert taken < before and pool.report() == (before - taken, 0, 0)
    assert torch.equal(positions.cpu(), more) and torch.equal(lens.cpu(), more + 1)
    entry = table.cpu()[torch.arange(B), (more // P).long()]
    assert torch.equal(slots.cpu(), entry * P + more % P)
    # back to what they had, then to nothing
    ops.release_pages(pool, table, lens, more.cuda())
    assert pool.report()[0] == before and torch.equal(lens.cpu(), more)
    ops.release_pages(pool, table, lens, torch.zeros(B, dtype=I32, device="cuda"))
    assert pool.report()[0] == pages and bool((table == -1).all()) and not bool(lens.any())
    assert torch.equal(pool.free.cpu(), torch.arange(pages - 1, -1, -1, dtype=I32))
    torch.cuda.empty_cache()

"""The 8-bit block operators at the largest sizes that they accept: launches that hold more
rows than a grid of one dimension, offsets past 32 bits."""
import pytest
import torch

import block8_oracle as O

pytestmark = pytest.mark.gpu

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from conv_bn_silu_amd import block8
    yield block8
    torch.cuda.empty_cache()


def say(*a):
    print(*a, flush=True)


def rows_at(M, borders):
    """Rows to compare: both ends, those around the borders, and some between."""
    g = torch.Generator().manual_seed(M)
    some = torch.randint(0, M, (40,), generator=g).tolist()
    near = [b + d for b in borders for d in (-2, -1, 0, 1, 2)]
    return torch.tensor(sorted({r for r in [0, 1, M - 2, M - 1, *near, *some] if 0 <= r < M}))


@pytest.mark.parametrize("M,N,K", [(2 ** 23 + 3, 8, 2056), (2 ** 24, 8, 2064), (2 ** 24, 5, 65)],
                         ids=lambda v: str(v))
def test_linear_most_rows(ops, M, N, K):
    """Every row is quantised, whatever their number (2^23 rows of 256 threads pass 2^31, 2^24 pass 2^32)."""
    g = torch.Generator(device="cuda").manual_seed(K)
    say("[linear rows]", M, N, K)
    x = torch.empty(M, K, dtype=BF16, device="cuda").normal_(generator=g)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32, device="cuda").to(I8)
    ws = torch.rand(N, generator=g, device="cuda") * 0.02 + 0.001
    y = ops.int8_linear(x, w, ws)
    at = rows_at(M, [2 ** 22, 2 ** 23, 3 * 2 ** 22])
    ref, tol = O.linear(x[at.cuda()].cpu(), w.cpu(), ws.cpu(), None, False)
    O.check(y[at.cuda()], ref, tol, f"{M} {N} {K}")
    # and no row between is left out: its sum with the weights is that of a smaller call
    for m0 in range(0, M, 2 ** 21):
        assert torch.equal(y[m0:m0 + 2 ** 21], ops.int8_linear(x[m0:m0 + 2 ** 21], w, ws)), m0
    del x, y
    torch.cuda.empty_cache()


def test_linear_most_rows_unaligned(ops):
    """Weights that start off 16 bytes go through the streaming kernel, whose tiles of rows pass 65535 here."""
    M, N, K = 64 * 65536 + 70, 5, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    say("[linear rows, unaligned]", M, N, K)
    x = torch.empty(M, K, dtype=BF16, device="cuda").normal_(generator=g)
    buf = torch.randint(-128, 128, (N * K + 1,), generator=g, dtype=torch.int32, device="cuda").to(I8)
    w = buf[1:].view(N, K)
    ws = torch.rand(N, generator=g, device="cuda") * 0.02 + 0.001
    y = ops.int8_linear(x, w, ws)
    at = rows_at(M, [64 * 32768, 64 * 65535, 64 * 65536])
    ref, tol = O.linear(x[at.cuda()].cpu(), w.cpu(), ws.cpu(), None, False)
    O.check(y[at.cuda()], ref, tol, f"{M} {N} {K}")
    assert torch.equal(y, ops.int8_linear(x, w.clone(), ws))


@pytest.mark.parametrize("tokens,heads,dim", [(2 ** 28 + 5, 1, 8), (2 ** 26 + 3, 2, 136)], ids=["narrow", "wide"])
def test_cache_most_rows(ops, tokens, heads, dim):
    """Calls of more rows than a launch has threads for (16 lanes a row up to dim 128, 32 beyond)."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    say("[cache rows]", tokens, heads, dim)
    pages, page = 64, 16
    cache = ops.PagedCache.empty(pages, heads, page, dim)
    k = torch.empty(tokens, heads, dim, dtype=BF16, device="cuda").normal_(generator=g)
    # tokens from all over the call have slots, the others none
    at = torch.cat([torch.arange(400), tokens // 2 + torch.arange(200), tokens - 1 - torch.arange(400)]).cuda()
    slots = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    slots[at] = torch.randperm(pages * page, generator=g, device="cuda")[:at.numel()].to(torch.int32)
    ops.cache_write(cache, k, k, slots)
    codes, s = O.quantize(k[at].cpu())
    want = (codes.float() * s[..., None]).to(BF16)
    del k
    got = ops.cache_read(cache, slots, BF16)
    for y in got:
        assert torch.equal(y[at].cpu(), want)
        assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(want))  # and zeros elsewhere
    del got, y
    torch.cuda.empty_cache()

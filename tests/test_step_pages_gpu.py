"""Pages given back where lengths or tables are not what growth leaves: against the rule, written out here as lists."""
import pytest
import torch

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import conv_bn_silu_amd
    yield conv_bn_silu_amd
    torch.cuda.empty_cache()


def say(*a):
    print(*a, flush=True)


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.mark.parametrize("n,width", [(3, 4), (70, 6), (1030, 2), (9, 20000)], ids=str)
def test_release_of_negative_lengths(ops, n, width):
    """They count as 0, and 0 is what they become; the others are cut as ever."""
    say("[negative lengths]", n, width)
    pool = ops.PagePool.full(4 * n, 4)
    table = torch.full((n, width), -1, dtype=I32, device="cuda")
    lens = torch.zeros(n, dtype=I32, device="cuda")
    ops.grow_pages(pool, table, lens, i32([5] * n), 5 * n)
    was = [[5, -1, 5, -2 ** 31, 5][b % 5] for b in range(n)]
    keep = [[1, 0, 9, 7, -3][b % 5] for b in range(n)]
    lens.copy_(i32(was))
    ops.release_pages(pool, table, lens, i32(keep))
    assert lens.tolist() == [min(max(0, w), max(0, k)) for w, k in zip(was, keep)]
    assert pool.report()[0] == 2 * n + sum([1, 0, 0, 0, 2][b % 5] for b in range(n))


@pytest.mark.parametrize("batch", [1024, 65536])
def test_release_of_as_many_pages_as_a_pool_may_have(ops, batch):
    """1.8 billion pages of one token come back at once, the first on top."""
    width, spare = 1_800_000_000 // batch, 12345
    n = batch * width
    say("[most pages]", batch, n)
    table = torch.arange(n, dtype=I32, device="cuda").view(batch, width)
    free = torch.full((n + spare,), -5, dtype=I32, device="cuda")
    free[:spare] = torch.arange(n, n + spare, dtype=I32, device="cuda")
    pool = ops.PagePool(free, i32([spare, 0, 0]), 1)
    lens = torch.full((batch,), width, dtype=I32, device="cuda")
    ops.release_pages(pool, table, lens, torch.zeros_like(lens))
    assert pool.report()[0] == n + spare
    assert bool((table == -1).all()) and not bool(lens.any())
    del table
    assert torch.equal(free[:spare], torch.arange(n, n + spare, dtype=I32, device="cuda"))
    assert torch.equal(free[spare:], torch.arange(n - 1, -1, -1, dtype=I32, device="cuda"))
    del free, pool
    torch.cuda.empty_cache()

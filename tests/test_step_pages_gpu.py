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

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


def given_back(table, lens, keep, page, free, count):
    """The rule: pages past the tokens that stay, of those that the pool has, the first on top."""
    table, free, back = [list(r) for r in table], list(free), []
    for b, row in enumerate(table):
        has = max(lens[b], 0)
        stays = min(has, max(keep[b], 0))
        for i in range(-(-stays // page), min(-(-has // page), len(row))):
            if 0 <= row[i] < len(free):
                back.append(row[i])
            row[i] = -1
    stack = (free[:count] + back[::-1])[:len(free)]
    return table, stack + free[len(stack):], len(stack)


HOLES = [
    # sequences, width, pages of each that come back: by threads, by one workgroup, by parts of rows, by several launches
    (1, 5, 5), (9, 8, 6), (1000, 60, 8), (9, 300, 300), (700, 90, 70), (64, 1000, 900), (1, 40000, 30000), (3, 30000, 27001),
    (1100, 40, 7), (1500, 60, 50), (5000, 30, 23),
]


@pytest.mark.parametrize("share", [0.0, 0.3, 1.0], ids=["whole", "some", "all"])
@pytest.mark.parametrize("shape", HOLES, ids=lambda s: "x".join(map(str, s)))
def test_release_of_rows_with_holes(ops, shape, share):
    """Entries that name no page of the pool give nothing back; what grows next gets pages only."""
    n, width, per = shape
    say("[holes]", shape, share)
    page, g = 3, torch.Generator().manual_seed(n + width)
    was = [per - b % 3 if per > 3 else per for b in range(n)]
    pages = sum(was) + 50
    order = torch.randperm(pages, generator=g)
    table, at = torch.full((n, width), -1, dtype=I32), 0
    for b, w in enumerate(was):
        table[b, :w] = order[at:at + w]
        at += w
    holes = torch.rand(n, width, generator=g) < share
    table = torch.where(holes, torch.tensor([-1, -1, pages, 2 ** 31 - 1, -2 ** 31], dtype=I32)[torch.arange(width) % 5], table)
    lens = [max(0, w * page - b % page) for b, w in enumerate(was)]
    keep = [[0, 4, 10, 2 ** 31 - 1, 0][b % 5] for b in range(n)]
    # what a window has left behind is in the stack already: with the holes it would not fit
    left = order[torch.isin(order, table[table >= 0], invert=True)].tolist()
    free = left + [-9] * (pages - len(left))
    want, stack, count = given_back(table.tolist(), lens, keep, page, free, len(left))
    pool = ops.PagePool(i32(free), i32([len(left), 0, 0]), page)
    on, dlens = table.cuda(), i32(lens)
    ops.release_pages(pool, on, dlens, i32(keep))
    assert pool.report()[0] == count and torch.equal(on.cpu(), torch.tensor(want, dtype=I32))
    assert torch.equal(pool.free.cpu(), torch.tensor(stack, dtype=I32))
    assert dlens.tolist() == [min(a, b) for a, b in zip(lens, keep)]
    # all that the pool has goes to new sequences, and every one of their tokens has a slot
    new = torch.full((1, count), -1, dtype=I32, device="cuda")
    _, slots, _ = ops.grow_pages(pool, new, i32([0]), i32([count * page]), count * page)
    assert pool.report() == (0, 0, 0) and new[0].tolist() == stack[:count][::-1]
    assert int(slots.min()) >= 0 and int(slots.unique().numel()) == count * page


def test_release_of_more_than_the_stack_holds(ops):
    """Pages that are in the table twice: the first given back, which would lie past the stack, are dropped."""
    for n, width in ((2, 6), (2, 40000), (6000, 12)):
        say("[twice]", n, width)
        table = (torch.arange(n * width, dtype=I32) % (n * width // 2)).view(n, width)
        lens, keep, free = [width] * n, [0] * n, [7] * (n * width // 2)
        want, stack, count = given_back(table.tolist(), lens, keep, 1, free, 5)
        pool, on, dlens = ops.PagePool(i32(free), i32([5, 0, 0]), 1), table.cuda(), i32(lens)
        ops.release_pages(pool, on, dlens, i32(keep))
        assert pool.report()[0] == count == len(free) and torch.equal(pool.free.cpu(), torch.tensor(stack, dtype=I32))
        assert bool((on == -1).all()) and not bool(dlens.any())


def test_growth_past_runs_of_idle_sequences(ops):
    """Tokens find their sequences past tens of thousands that bring none, and no slower for where those lie: walked one
    by one, the run costs thousands of times the search."""
    n, per, page = 65536, 1501, 16
    at = [5, 30000, 30002, 65535]
    times = []
    for where in (at, [0, 1, 2, 3]):
        more = torch.zeros(n, dtype=I32)
        more[where] = per
        say("[idle]", where)
        pool = ops.PagePool.full(4 * 95, page)
        table, lens = torch.full((n, 95), -1, dtype=I32, device="cuda"), torch.zeros(n, dtype=I32, device="cuda")
        more, keep, tokens = more.cuda(), torch.zeros_like(lens), 4 * per + 70
        for turn in range(5):
            ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            ev[0].record()
            starts, slots, positions = ops.grow_pages(pool, table, lens, more, tokens)
            ev[1].record()
            torch.cuda.synchronize()
            times.append(ev[0].elapsed_time(ev[1]))
            i = torch.arange(4 * per, dtype=I32)
            # a full pool hands out pages 0, 1, ... in order
            assert pool.report() == (4, 0, 0) and torch.equal(positions[:4 * per].cpu(), i % per)
            assert torch.equal(slots[:4 * per].cpu(), i // per * 94 * page + i % per)
            assert bool((slots[4 * per:] == -1).all()) and bool((positions[4 * per:] == 0).all())
            assert torch.equal(lens, more) and torch.equal(starts[1:].cpu().long(), more.cpu().long().cumsum(0))
            ops.release_pages(pool, table, lens, keep)
    print("idle between %.3f ms, behind %.3f ms" % (min(times[:5]), min(times[5:])))
    assert min(times[:5]) < 20 * min(times[5:])


@pytest.mark.parametrize("shape", [(9, 20, 6), (60, 1000, 700), (3, 30000, 20011), (1500, 60, 50), (4500, 30, 23)], ids=str)
def test_pages_in_a_graph(ops, shape):
    """Growth and giving back captured once and replayed, with holes made in between and other work beside, against the same
    calls by themselves."""
    n, width, per = shape
    say("[pages graph]", shape)
    page, tokens = 4, n * per * 4
    more = torch.full((n,), per * 4, dtype=I32, device="cuda")
    more[::3] -= 5
    keep = torch.arange(n, dtype=I32, device="cuda") % 7
    hole = torch.rand(n, width, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)) < 0.2
    lost = torch.zeros((), dtype=I32, device="cuda")

    def state():
        return [ops.PagePool.full(n * per + 9, page), torch.full((n, width), -1, dtype=I32, device="cuda"),
                torch.zeros(n, dtype=I32, device="cuda")]

    def turn(pool, table, lens):
        got = ops.grow_pages(pool, table, lens, more, tokens)
        table.masked_fill_(hole, -1)
        ops.release_pages(pool, table, lens, keep)
        return got

    eager, s = state(), state()
    turn(*eager), turn(*s)
    graph = torch.cuda.CUDAGraph()
    before = [t.clone() for t in (s[0].free, s[0].counts, *s[1:])]
    with torch.cuda.graph(graph):
        out = turn(*s)
    for t, v in zip((s[0].free, s[0].counts, *s[1:]), before):
        t.copy_(v)
    for i in range(5):
        graph.replay()
        want = turn(*eager)
        lost += eager[0].counts[2]
        torch.cuda.synchronize()
        for a, b in zip((*want, eager[0].free, eager[0].counts, *eager[1:]), (*out, s[0].free, s[0].counts, *s[1:])):
            assert torch.equal(a, b), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = turn(*eager)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*want, eager[0].free, eager[0].counts, *eager[1:]), (*out, s[0].free, s[0].counts, *s[1:])):
        assert torch.equal(a, b)
    assert int(lost) > 0  # holes are pages lost, and the pool ran short

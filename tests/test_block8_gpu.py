"""The 8-bit block operators on the GPU against their definitions in 64 bits."""
import math

import pytest
import torch

import block8_oracle as O

pytestmark = pytest.mark.gpu

BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from conv_bn_silu_amd import block8
    return block8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def say(*a):
    print(*a, flush=True)


# --- linear -----------------------------------------------------------------

LINEAR = [
    # M, N, K: one row to many, tiles' edges, odd K (rows of w at any byte)
    (1, 1, 1), (1, 17, 64), (1, 4096, 4096), (1, 129, 8192), (2, 1000, 2000), (3, 64, 128), (4, 257, 1999),
    (5, 96, 16), (8, 512, 9000), (13, 300, 72), (16, 128, 256), (17, 130, 320), (31, 1024, 1024), (33, 65, 63),
    (40, 256, 4096), (48, 80, 500), (64, 192, 640), (65, 1001, 130), (100, 96, 1999), (127, 129, 257),
    (128, 256, 512), (200, 520, 1040), (256, 256, 128), (257, 300, 384), (333, 1001, 1999), (512, 768, 1152),
    (700, 511, 2048), (1000, 1024, 96), (1025, 260, 1000),
]


def linear_inputs(M, N, K, dtype, seed):
    g = gen(seed)
    x = torch.randn(M, K, generator=g) * (1 + 5 * (torch.rand(K, generator=g) > 0.95))
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int32).to(I8)
    ws = torch.rand(N, generator=g) * 0.02 + 0.001
    return x.to(dtype), w, ws, torch.randn(N, generator=g)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", LINEAR, ids=lambda s: "x".join(map(str, s)))
def test_linear(ops, shape, dtype):
    M, N, K = shape
    say("[linear]", shape, dtype)
    x, w, ws, b = linear_inputs(M, N, K, dtype, 7 * M + N + K)
    for bias, act in ((None, None), (b, "silu")):
        ref, tol = O.linear(x, w, ws, bias, act == "silu")
        y = ops.int8_linear(x.cuda(), w.cuda(), ws.cuda(), None if bias is None else bias.cuda(), act)
        assert y.dtype == dtype and tuple(y.shape) == (M, N)
        O.check(y, ref, tol, f"{shape} {act}")


@pytest.mark.parametrize("shape", [(1, 64, 96), (5, 70, 200), (40, 48, 130), (300, 130, 257)],
                         ids=lambda s: "x".join(map(str, s)))
def test_linear_strides_and_alignment(ops, shape):
    M, N, K = shape
    for dtype in (BF16, F32):
        x, w, ws, b = linear_inputs(M, N, K, dtype, 11)
        ref, tol = O.linear(x, w, ws, b, False)
        say("[linear strided]", shape, dtype)
        wide = torch.zeros(M, K + 9, dtype=dtype, device="cuda")
        wide[:, 3:3 + K] = x.cuda()
        wbuf = torch.zeros(N * K + 1, dtype=I8, device="cuda")
        wbuf[1:] = w.cuda().reshape(-1)
        ybuf = torch.full((M * N + 3,), 7.0, dtype=dtype, device="cuda")
        out = ybuf[1:1 + M * N].view(M, N)
        y = ops.int8_linear(wide[:, 3:3 + K], wbuf[1:].view(N, K), ws.cuda(), b.cuda(), out=out)
        assert y.data_ptr() == out.data_ptr()
        O.check(y, ref, tol, f"{shape} strided")
        assert bool((ybuf[:1] == 7).all()) and bool((ybuf[1 + M * N:] == 7).all())
        xt = x.cuda().t().contiguous().t()  # column-major rows
        O.check(ops.int8_linear(xt, w.cuda(), ws.cuda(), b.cuda()), ref, tol, f"{shape} transposed")


@pytest.mark.parametrize("shape", [
    # M, N, K: each kernel's own sizes, off its tiles: rows quantised inside the product (up to 16), tiles of 64, of
    # 128 and of 256, K from one step to several rounds of the buffers, rows of w at odd bytes
    (6, 300, 2000), (9, 70, 900), (16, 500, 1024), (16, 500, 1040), (7, 40, 131072), (20, 16390, 48), (64, 16400, 640),
    (97, 4097, 1152), (130, 3100, 130), (140, 5000, 1023), (1300, 2001, 128), (1281, 2050, 784), (1400, 1999, 515),
    (3500, 3460, 16), (4097, 3011, 144), (3400, 3600, 129), (60, 16390, 131),
], ids=lambda s: "x".join(map(str, s)))
def test_linear_kernels(ops, shape):
    M, N, K = shape
    for dtype, bias, act in ((BF16, False, None), (F32, True, "silu")):
        say("[linear kernels]", shape, dtype)
        x, w, ws, b = linear_inputs(M, N, K, dtype, M + N + K)
        ref, tol = O.linear(x, w, ws, b if bias else None, act == "silu")
        O.check(ops.int8_linear(x.cuda(), w.cuda(), ws.cuda(), b.cuda() if bias else None, act), ref, tol, f"{shape}")


@pytest.mark.parametrize("shape", [(33, 64, 6272), (40, 70, 8192), (100, 1030, 8992), (130, 70, 6501),
                                   (65, 16, 131072), (600, 200, 14336)], ids=lambda s: "x".join(map(str, s)))
def test_linear_long_sums(ops, shape):
    """Few outputs of long sums; calls one after the other share nothing."""
    M, N, K = shape
    for dtype, bias, act in ((BF16, False, None), (F32, True, "silu")):
        say("[linear long sums]", shape, dtype)
        x, w, ws, b = linear_inputs(M, N, K, dtype, M + N + K)
        ref, tol = O.linear(x, w, ws, b if bias else None, act == "silu")
        x, w, ws, b = x.cuda(), w.cuda(), ws.cuda(), b.cuda() if bias else None
        y = [ops.int8_linear(x, w, ws, b, act) for _ in range(3)]
        O.check(y[0], ref, tol, f"{shape}")
        assert torch.equal(y[1], y[0]) and torch.equal(y[2], y[0])


def test_linear_long_sums_graph(ops):
    x, w, ws, b = (t.cuda() for t in linear_inputs(70, 200, 9216, BF16, 10))
    want = ops.int8_linear(x, w, ws, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.int8_linear(x, w, ws, b)
    for i in range(4):
        y.zero_()
        graph.replay()
        assert torch.equal(ops.int8_linear(x, w, ws, b), want), i
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_linear_leading_axes_and_empty(ops):
    x, w, ws, b = linear_inputs(24, 48, 64, BF16, 5)
    ref, tol = O.linear(x, w, ws, b, True)
    y = ops.int8_linear(x.cuda().view(2, 3, 4, 64), w.cuda(), ws.cuda(), b.cuda(), "silu")
    assert tuple(y.shape) == (2, 3, 4, 48)
    O.check(y.view(24, 48), ref, tol, "leading axes")
    assert tuple(ops.int8_linear(x.cuda()[:0], w.cuda(), ws.cuda()).shape) == (0, 48)


@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_linear_special_rows(ops, M):
    """Rows of zeros, of one value, of the smallest and largest numbers, next to
    code borders; a NaN or an infinity makes its own row NaN and no other."""
    K, N = 256, 72
    x, w, ws, b = linear_inputs(M, N, K, F32, 3)
    rows = [torch.zeros(K), torch.full((K,), 2.0 ** -130), torch.full((K,), -3e38),
            torch.arange(K).float() / 2 - 63.5,  # halves: ties between codes
            (torch.arange(K).float() - 127).clamp(-127, 127) * 1.1920929e-7]
    for i in range(min(M, len(rows))):
        for first in ([0] if M > 1 else range(len(rows))):
            x[i] = rows[i + first]
            if M == 1:
                ref, tol = O.linear(x, w, ws * 1e-3, b, False)
                O.check(ops.int8_linear(x.cuda(), w.cuda(), (ws * 1e-3).cuda(), b.cuda()), ref, tol, f"row {first}")
    ref, tol = O.linear(x, w, ws * 1e-3, b, False)
    O.check(ops.int8_linear(x.cuda(), w.cuda(), (ws * 1e-3).cuda(), b.cuda()), ref, tol, "special rows")
    for bad in (math.nan, math.inf, -math.inf):
        z = x.clone()
        z[M // 2, 5] = bad
        y = ops.int8_linear(z.cuda(), w.cuda(), (ws * 1e-3).cuda(), b.cuda()).cpu()
        assert bool(y[M // 2].isnan().all())
        keep = torch.arange(M) != M // 2
        if M > 1:
            O.check(y[keep], ref[keep], tol[keep], "other rows")


def test_linear_graph_and_streams(ops):
    x, w, ws, b = (t.cuda() for t in linear_inputs(40, 512, 1024, BF16, 9))
    want = ops.int8_linear(x, w, ws, b, "silu")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.int8_linear(x, w, ws, b, "silu")
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.int8_linear(x, w, ws, b, "silu")
    for i in range(4):
        x.copy_(torch.roll(x, 1, 0))
        eager = ops.int8_linear(x, w, ws, b, "silu")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), i


# --- cache ------------------------------------------------------------------

CACHE = [
    # tokens, heads, dim, page
    (1, 1, 8, 1), (64, 8, 128, 16), (37, 5, 80, 24), (100, 3, 96, 17), (33, 2, 256, 128), (50, 1, 64, 32),
    (29, 4, 16, 7), (20, 2, 136, 16), (500, 8, 128, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("held", [I8, BF16, F16, F32], ids=["i8", "hbf16", "hf16", "hf32"])
@pytest.mark.parametrize("shape", CACHE, ids=lambda s: "x".join(map(str, s)))
def test_cache_round_trip(ops, shape, dtype, held):
    T, H, D, P = shape
    say("[cache]", shape, dtype, held)
    g = gen(T + H + D)
    pages = (T + P - 1) // P + 3
    k = (torch.randn(T, H, D, generator=g) + 2 * torch.randn(H, D, generator=g)).to(dtype)
    v = torch.randn(T, H, D, generator=g).to(dtype)
    slots = torch.randperm(pages * P, generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    if T > 3:
        slots[3] = pages * P  # just past the cache
    cache = ops.PagedCache.empty(pages, H, P, D, held)
    cache.k.fill_(3)
    # strided: slices of one fused projection
    fused = torch.zeros(T, 2 * H * D + 8, dtype=dtype, device="cuda")
    ks, vs = fused[:, :H * D].view(T, H, D), fused[:, H * D:2 * H * D].view(T, H, D)
    ks.copy_(k)
    vs.copy_(v)
    ops.cache_write(cache, ks, vs, slots.cuda())
    there = (slots >= 0) & (slots < pages * P)
    at = slots[there].long()
    untouched = torch.ones(pages * P, dtype=torch.bool)
    untouched[at] = False
    u = untouched.nonzero()[:, 0]
    assert bool((cache.k[u.cuda() // P, :, u.cuda() % P] == 3).all())
    back = ops.cache_read(cache, slots.cuda(), dtype)
    for src, got, name in ((k, back[0], "k"), (v, back[1], "v")):
        if held == I8:
            codes, s = O.quantize(src)
            pg, off = (at // P).cuda(), (at % P).cuda()
            assert torch.equal(getattr(cache, name)[pg, :, off].cpu().double(), codes[there])
            assert torch.equal(getattr(cache, name + "_scale")[pg, :, off].cpu(), s[there])
            want = (codes.float() * s[..., None]).to(dtype)
        else:
            want = src.to(held).to(dtype)
        want[~there] = 0
        assert torch.equal(got.cpu(), want)


def test_cache_unaligned_and_special(ops):
    T, H, D, P = 12, 2, 24, 4
    buf = torch.zeros(T * H * D + 1, dtype=BF16, device="cuda")
    x = torch.randn(T, H, D, generator=gen(1))
    x[0] = 0
    x[1, :, 5] = math.inf
    x[2, 0, 3] = math.nan
    x[3] = torch.arange(D) / 2 - 5.5
    x[4] = 2.0 ** -130
    x = x.to(BF16)
    k = buf[1:].view(T, H, D)
    k.copy_(x)
    cache = ops.PagedCache.empty(4, H, P, D)
    slots = torch.arange(T, dtype=torch.int32)
    ops.cache_write(cache, k, k, slots.cuda())
    codes, s = O.quantize(x)
    fine = torch.ones(T, H, dtype=torch.bool)
    fine[1] = fine[2, 0] = False
    got = ops.cache_read(cache, slots.cuda(), F32)
    for y in got:
        y = y.cpu()
        assert torch.equal(y[fine], (codes.float() * s[..., None])[fine])
        assert bool(y[~fine].isnan().all())
    ops.cache_write(cache, k[:0], k[:0], slots[:0].cuda())
    assert ops.cache_read(cache, slots[:0].cuda())[0].shape[0] == 0


def test_cache_past_32_bit_offsets(ops):
    """A cache whose values lie past 2^31 elements, written, read and attended."""
    P, D, H = 64, 256, 1
    pages = 2 ** 31 // (P * D) + 8
    k = torch.empty(pages, H, P, D, dtype=I8, device="cuda")
    v = torch.empty_like(k)
    cache = ops.PagedCache(k, v, *(torch.zeros(pages, H, P, device="cuda") for _ in range(2)))
    n = 130
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    j = torch.arange(n)
    slots = (table[0].long()[j // P] * P + j % P).to(torch.int32)
    x, y = (torch.randn(n, H, D, generator=gen(s)).to(BF16) for s in (1, 2))
    ops.cache_write(cache, x.cuda(), y.cuda(), slots.cuda())
    got = ops.cache_read(cache, slots.cuda(), F32)
    for src, g in ((x, got[0]), (y, got[1])):
        codes, s = O.quantize(src)
        assert torch.equal(g.cpu(), codes.float() * s[..., None])
    q = torch.randn(3, 2, D, generator=gen(4)).to(BF16)
    out = ops.paged_attention(q.cuda(), cache, table.cuda(), torch.tensor([0, 3], dtype=torch.int32).cuda(),
                              torch.tensor([n], dtype=torch.int32).cuda())
    small = torch.zeros(3, H, P, D, dtype=O.F64), torch.zeros(3, H, P, D, dtype=O.F64)
    for t, src in zip(small, (x, y)):
        codes, s = O.quantize(src)
        t[j // P, :, j % P] = codes * s.double()[..., None]
    ref, tol, _ = O.attention(q, *small, torch.tensor([[0, 1, 2]]), [0, 3], [n], 0, D ** -0.5, O.half_step(F16))
    O.check(out, ref, tol, "high pages")


# --- attention --------------------------------------------------------------

def attention_case(new, lens, heads, hk, dim, page, dtype, int8, window=0, seed=0, holes=False, scale=None, k_gain=1.0,
                   v_gain=None):
    """Inputs on the CPU; what lies past a sequence's end, and every page that no
    sequence owns, holds NaN."""
    g = gen(seed)
    B = len(new)
    used = [(n + page - 1) // page for n in lens]
    width = max(max(used), 1) + 1
    pages = sum(used) + 2
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]].to(torch.int32)
        at += used[b]
    k = torch.randn(pages, hk, page, dim, generator=g) * k_gain + torch.randn(hk, 1, dim, generator=g)
    v = torch.randn(pages, hk, page, dim, generator=g)
    if v_gain is not None:
        v = v * v_gain[0] * (v_gain[1] / v_gain[0]) ** torch.rand(pages, hk, page, 1, generator=g)
    live = torch.zeros(pages, page, dtype=torch.bool)
    for b in range(B):
        j = torch.arange(lens[b])
        live[table[b].long()[j // page], j % page] = True
    if int8:
        held = []
        for x in (k, v):
            codes, s = O.quantize(x)
            s = s.clone()
            s[~live[:, None, :].expand_as(s)] = math.nan
            held += [codes.to(I8), s]
        kv64 = [(c.double() * s.double().nan_to_num(0)[..., None]) for c, s in ((held[0], held[1]), (held[2], held[3]))]
        tensors = (held[0], held[2], held[1], held[3])
    else:
        k, v = k.to(dtype), v.to(dtype)
        kv64 = [torch.where(live[:, None, :, None], x.double(), 0.0) for x in (k, v)]
        for x in (k, v):
            x[~live[:, None, :].expand(x.shape[:3])] = math.nan
        tensors = (k, v)
    if holes:
        for b in range(B):
            if used[b] > 2:
                table[b, 1] = [-1, pages, 2 ** 30][b % 3]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = torch.randn(starts[-1], heads, dim, generator=g).to(dtype)
    return dict(q=q, tensors=tensors, kv64=kv64, table=table, starts=starts, lens=lens, window=window,
                scale=dim ** -0.5 if scale is None else scale)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_case(ops, c, **kw):
    cache = ops.PagedCache(*(t.cuda() for t in c["tensors"]))
    return ops.paged_attention(c["q"].cuda(), cache, c["table"].cuda(), i32(c["starts"]), i32(c["lens"]),
                               window=c["window"], scale=c["scale"], **kw)


def check_case(ops, c, what):
    u = O.half_step(BF16) if c["tensors"][0].dtype == BF16 else O.half_step(F16)
    ref, tol, mine = O.attention(c["q"], *c["kv64"], c["table"], c["starts"], c["lens"], c["window"], c["scale"], u)
    say("[attention]", what)
    out = run_case(ops, c)
    O.check(out.cpu()[mine], ref[mine], tol[mine], what)


TYPES = [(BF16, True), (F16, True), (BF16, False), (F16, False)]
TYPE_IDS = ["bf16-i8", "f16-i8", "bf16", "f16"]
ATTENTION = [
    # new, lens, heads, kv heads, dim, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1, 1, 1, 1], [90, 600, 33, 1], 8, 2, 64, 16, 0),
    ([1, 1, 1], [127, 128, 129], 8, 1, 128, 16, 0),
    ([1, 1], [1500, 70], 32, 8, 128, 16, 0),
    ([1, 1, 1], [255, 17, 40], 5, 5, 80, 24, 0),
    ([1, 0, 1], [40, 12, 0], 12, 3, 96, 17, 0),
    ([1, 1], [300, 64], 8, 4, 256, 128, 0),
    ([1, 1], [500, 80], 15, 3, 16, 32, 100),
    ([1, 1], [300, 64], 24, 1, 192, 64, 0),
    ([1], [700], 71, 1, 64, 16, 0),
    ([3, 1, 2], [60, 700, 2], 8, 2, 128, 16, 0),
    ([7, 40], [7, 300], 8, 8, 64, 64, 0),
    ([33, 100, 1, 0], [200, 100, 90, 5], 10, 2, 80, 24, 64),
    ([130], [130], 4, 2, 128, 64, 0),
    ([65, 64, 63], [65, 640, 63], 5, 1, 96, 17, 0),
    ([50, 200], [777, 200], 8, 2, 256, 32, 0),
    ([150], [400], 15, 3, 80, 24, 100),
    ([90, 31], [100, 31], 16, 1, 48, 16, 30),
    ([300], [300], 2, 1, 128, 128, 0),
]


@pytest.mark.parametrize("types", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(ops, case, types):
    new, lens, heads, hk, dim, page, window = ATTENTION[case]
    c = attention_case(new, lens, heads, hk, dim, page, *types, window=window, seed=case)
    check_case(ops, c, f"{ATTENTION[case]} {types}")


@pytest.mark.parametrize("types", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("new,lens", [([1], [20000]), ([1, 1, 1], [9000, 3, 2500]), ([2, 20, 1], [4000, 6000, 5]),
                                      ([40], [5000])], ids=["one", "decode", "mixed", "chunk"])
def test_attention_long(ops, new, lens, types):
    c = attention_case(new, lens, 4, 1, 128, 16, *types, seed=3)
    check_case(ops, c, f"{new} {lens} {types}")


@pytest.mark.parametrize("types", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("new,lens", [([1, 1, 1, 1], [100, 70, 300, 17]), ([40, 3, 64, 5], [100, 70, 300, 17])],
                         ids=["decode", "chunk"])
def test_attention_missing_pages(ops, new, lens, types):
    """Pages outside the cache are not seen, nor is what lies past the table."""
    c = attention_case(new, lens, 8, 2, 64, 16, *types, seed=5, holes=True)
    check_case(ops, c, f"holes {new} {types}")
    c["table"] = c["table"][:, :4].contiguous()
    check_case(ops, c, f"short table {new} {types}")
    c["table"] = torch.full_like(c["table"], -1)
    assert bool((run_case(ops, c) == 0).all())


@pytest.mark.parametrize("new", [[1, 1], [30, 40]], ids=["decode", "chunk"])
def test_attention_value_scales(ops, new):
    """Values of widely spread scales (a growing one, a shrinking one) and tokens
    of zeros keep their weight in the sum; large scores; negative scale."""
    for gain in ((1e-4, 1e4), (1e3, 1e-3), (1e-30, 1e-28)):
        c = attention_case(new, [200, 333], 8, 2, 128, 16, BF16, True, seed=8, v_gain=gain)
        check_case(ops, c, f"scales {gain}")
    c = attention_case(new, [200, 333], 8, 2, 128, 16, BF16, True, seed=9)
    for t, s in zip(c["tensors"][1:2], c["tensors"][3:4]):
        t[:, :, ::2] = 0
        s[:, :, ::2] = torch.where(s[:, :, ::2].isnan(), math.nan, 2.0 ** -126)
        c["kv64"][1][:, :, ::2] = 0
    check_case(ops, c, "zero values")
    for types in TYPES:
        check_case(ops, attention_case(new, [200, 333], 8, 2, 128, 16, *types, seed=10, k_gain=30.0), f"sharp {types}")
        check_case(ops, attention_case(new, [200, 333], 8, 2, 128, 16, *types, seed=10, scale=-0.2), "negative scale")
        c = attention_case(new, [200, 333], 8, 2, 128, 16, *types, seed=10)
        c["q"] = (c["q"].float() * torch.logspace(-6, 3, c["q"].shape[0] * 8).view(-1, 8, 1)).to(types[0])
        check_case(ops, c, f"queries of every size {types}")


@pytest.mark.parametrize("types", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("new,lens", [([4, 2], [40, 30]), ([70, 3], [200, 30])], ids=["few", "chunk"])
def test_attention_masked_nan(ops, new, lens, types):
    """A NaN or infinity in a later token's keys or values does not reach the
    queries before it; those after it get NaN."""
    for which, bad in (("k", math.nan), ("v", math.nan), ("v", math.inf)):
        c = attention_case(new, lens, 4, 2, 64, 16, *types, seed=21)
        clean = run_case(ops, c).cpu()
        at = lens[0] - 2  # the last but one token of the first sequence
        page, off = int(c["table"][0, at // 16]), at % 16
        if types[1]:
            c["tensors"][2 if which == "k" else 3][page, :, off] = bad
        else:
            c["tensors"][0 if which == "k" else 1][page, :, off, 3] = bad
        out = run_case(ops, c).cpu()
        n = new[0]
        assert torch.equal(out[:n - 2], clean[:n - 2]), which
        assert torch.equal(out[n:], clean[n:]), which
        hit = out[n - 2:n] if types[1] or which == "k" else out[n - 2:n, :, 3]
        assert not bool(hit.isfinite().any()), which


def test_attention_strides_streams_and_rest(ops):
    c = attention_case([30, 1, 7], [100, 50, 7], 8, 2, 64, 16, BF16, True, seed=12)
    want = run_case(ops, c)
    q = c["q"].cuda()
    T = q.shape[0]
    cache = ops.PagedCache(*(t.cuda() for t in c["tensors"]))
    table, starts, lens = c["table"].cuda(), i32(c["starts"]), i32(c["lens"])
    # queries inside a fused projection, a table with longer rows, out given
    fused = torch.zeros(T, 8 * 64 + 24, dtype=BF16, device="cuda")
    fused[:, 8:8 + 512] = q.view(T, 512)
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out = torch.full((T + 2, 8, 64), 5.0, dtype=BF16, device="cuda")
    got = ops.paged_attention(fused[:, 8:8 + 512].view(T, 8, 64), cache, wide[:, :table.shape[1]], starts, lens,
                              out=out[1:T + 1])
    assert torch.equal(got, want) and bool((out[0] == 5).all()) and bool((out[T + 1] == 5).all())
    # at an odd element offset
    buf = torch.zeros(T * 512 + 1, dtype=BF16, device="cuda")
    buf[1:] = q.view(-1)
    obuf = torch.zeros(T * 512 + 1, dtype=BF16, device="cuda")
    got = ops.paged_attention(buf[1:].view(T, 8, 64), cache, table, starts, lens, out=obuf[1:].view(T, 8, 64))
    assert torch.equal(got, want)
    # head-major queries
    got = ops.paged_attention(q.transpose(0, 1).contiguous().transpose(0, 1), cache, table, starts, lens)
    assert torch.equal(got, want)
    # rows that belong to no sequence are left alone
    out = torch.full((T, 8, 64), 5.0, dtype=BF16, device="cuda")
    ops.paged_attention(q, cache, table[1:2], starts[1:3].contiguous(), lens[1:2].contiguous(), out=out)
    mine = torch.arange(T) == 30
    assert torch.equal(out.cpu()[mine], want.cpu()[mine]) and bool((out.cpu()[~mine] == 5).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.paged_attention(q, cache, table, starts, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    assert ops.paged_attention(q[:0], cache, table, starts, lens).shape[0] == 0
    assert ops.paged_attention(q, cache, table[:0], starts[:1].contiguous(), lens[:0]).shape[0] == T


@pytest.mark.parametrize("new", [1, 20], ids=["decode", "chunk"])
def test_attention_graph(ops, new):
    """A captured step of write and attention replays like eager calls while the
    lengths, the table's pages and the tokens change."""
    B, H, hk, D, P = 5, 8, 2, 64, 16
    g = gen(2)
    cache = ops.PagedCache.empty(120, hk, P, D)
    other = ops.PagedCache.empty(120, hk, P, D)
    table = torch.randperm(120, generator=g)[:100].view(B, 20).to(torch.int32).cuda()
    starts = i32([new * b for b in range(B + 1)])
    lens = i32([40, 60, 100, 33, 200])
    kv = torch.randn(2, new * B, hk, D, generator=g).to(BF16).cuda()
    q = torch.randn(new * B, H, D, generator=g).to(BF16).cuda()

    def slots():
        pos = (lens.long()[:, None] - new + torch.arange(new, device="cuda")).view(-1)
        rows = torch.arange(B, device="cuda").repeat_interleave(new)
        return (table[rows, pos // P].long() * P + pos % P).to(torch.int32)

    def step(c, s):
        ops.cache_write(c, kv[0], kv[1], s)
        return ops.paged_attention(q, c, table, starts, lens)

    at = slots()
    step(cache, at), step(other, at)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(cache, at)
    for i in range(4):
        lens += 3
        kv.copy_(torch.roll(kv, 1, 1))
        q.copy_(torch.roll(q, 1, 0))
        at.copy_(slots())
        want = step(other, at)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        assert bool(y.isfinite().all())


def test_attention_is_deterministic(ops):
    c = attention_case([1, 1, 300], [3000, 50, 4000], 8, 2, 128, 16, BF16, True, seed=14)
    first = run_case(ops, c)
    for _ in range(3):
        assert torch.equal(run_case(ops, c), first)


def test_attention_wide_table(ops):
    """A table with room for far more tokens than any sequence has."""
    for new, lens in (([1, 1, 1], [700, 30, 2100]), ([1, 40, 300], [2000, 40, 900])):
        c = attention_case(new, lens, 8, 2, 64, 16, BF16, True, seed=31)
        want = run_case(ops, c)
        ref, tol, mine = O.attention(c["q"], *c["kv64"], c["table"], c["starts"], c["lens"], 0, c["scale"], O.half_step(F16))
        wide = torch.full((3, 20000), -1, dtype=torch.int32)
        wide[:, :c["table"].shape[1]] = c["table"]
        c["table"] = wide
        say("[attention wide table]", new)
        O.check(run_case(ops, c), ref, tol, f"wide table {new}")
        O.check(want, ref, tol, f"narrow table {new}")


@pytest.mark.parametrize("dim", [16, 48, 80, 96, 112, 144, 192, 256])
def test_attention_dims(ops, dim):
    """Every padding of dim, single tokens and chunks, NaN in what is never read."""
    for types in TYPES:
        for new in ([1, 1], [70, 5]):
            c = attention_case(new, [150, 90], 6, 2, dim, 20, *types, window=70, seed=dim)
            check_case(ops, c, f"dim {dim} {new} {types}")


@pytest.mark.parametrize("types", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("new,lens,heads,hk,dim,window",
                         [([700], [700], 8, 2, 128, 0), ([1000, 90, 600], [1000, 700, 1500], 4, 1, 64, 0),
                          ([400], [5000], 4, 2, 80, 300), ([300, 40], [2000, 3000], 6, 3, 128, 130),
                          ([129, 64, 5], [129, 600, 700], 2, 1, 96, 0)],
                         ids=["prompt", "prompts", "window", "windows", "ragged"])
def test_attention_prompts(ops, new, lens, heads, hk, dim, window, types):
    """Prompts that are too short to fill the CUs with whole tiles, with and without chunks."""
    c = attention_case(new, lens, heads, hk, dim, 16, *types, window=window, seed=37)
    check_case(ops, c, f"{new} {lens} {dim} {window} {types}")


@pytest.mark.parametrize("new,lens", [([1, 1], [900, 40]), ([5, 9], [600, 9]), ([80, 300], [500, 300])],
                         ids=["decode", "few", "chunk"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_bad_scales(ops, new, lens, bad):
    """An infinite or NaN scale of a key or value reaches the queries that see it and no others."""
    for which in (2, 3):
        c = attention_case(new, lens, 8, 2, 64, 16, BF16, True, seed=41)
        ref, tol, _ = O.attention(c["q"], *c["kv64"], c["table"], c["starts"], c["lens"], 0, c["scale"], O.half_step(F16))
        at = lens[1] - 2  # of the second sequence
        c["tensors"][which][int(c["table"][1, at // 16]), :, at % 16] = bad
        out = run_case(ops, c).cpu()
        token = torch.arange(out.shape[0])
        pos = lens[1] - new[1] + token - new[0]
        hit = (token >= new[0]) & (pos >= at)
        say("[attention bad scales]", new, which, bad)
        O.check(out[~hit], ref[~hit], tol[~hit], f"rows that do not see it {new} {which}")
        assert not bool(out[hit].isfinite().any())


def test_refusals(ops):
    """What the binding and the C ABI do not serve is refused before any kernel."""
    from conv_bn_silu_amd.binding import CbsError
    dev = dict(device="cuda")
    x, w, s = torch.zeros(4, 64, dtype=BF16, **dev), torch.zeros(8, 64, dtype=I8, **dev), torch.zeros(8, **dev)
    for bad in (dict(x=x.double()), dict(w=w.float()), dict(w_scale=s.half()), dict(bias=s.half()), dict(x=None),
                dict(out=torch.zeros(4, 8, dtype=F16, **dev))):
        with pytest.raises(TypeError):
            ops.int8_linear(**{**dict(x=x, w=w, w_scale=s), **bad})
    for bad in (dict(x=x[:, :63]), dict(w=w[:, ::2]), dict(w=w.t().contiguous().t()), dict(w_scale=s[:7]),
                dict(bias=s.cpu()), dict(activation="gelu"), dict(out=torch.zeros(3, 8, dtype=BF16, **dev)),
                dict(x=torch.zeros(4, 64, dtype=BF16, requires_grad=True, **dev))):
        with pytest.raises(ValueError):
            ops.int8_linear(**{**dict(x=x, w=w, w_scale=s), **bad})
    with pytest.raises(CbsError):  # the output over the input
        ops.int8_linear(x, torch.zeros(64, 64, dtype=I8, **dev), torch.zeros(64, **dev), out=x)
    with pytest.raises(CbsError):
        ops.int8_linear(torch.zeros(1, 131088, dtype=BF16, **dev), torch.zeros(1, 131088, dtype=I8, **dev), s[:1])

    cache = ops.PagedCache.empty(4, 2, 16, 64)
    k, slots = torch.zeros(3, 2, 64, dtype=BF16, **dev), torch.zeros(3, dtype=torch.int32, **dev)
    with pytest.raises(ValueError):
        ops.PagedCache(cache.k, cache.v, cache.k_scale[:3], cache.v_scale)
    with pytest.raises(ValueError):
        ops.PagedCache(k[None], k[None], cache.k_scale, cache.v_scale)
    with pytest.raises(TypeError):
        ops.PagedCache(cache.k, cache.v)
    with pytest.raises(CbsError):  # a head dim that is no multiple of 8
        ops.cache_read(ops.PagedCache.empty(4, 2, 16, 60), slots)
    for bad in ((k.double(), k.double(), slots), (k, k.half(), slots), (k, k, slots.long())):
        with pytest.raises(TypeError):
            ops.cache_write(cache, *bad)
    for bad in ((k[:2], k, slots), (k, k[:, :1], slots), (k.transpose(1, 2), k, slots), (k, k, slots[:2])):
        with pytest.raises(ValueError):
            ops.cache_write(cache, *bad)
    with pytest.raises(TypeError):
        ops.cache_read(cache, slots, torch.int8)

    q = torch.zeros(3, 4, 64, dtype=BF16, **dev)
    good = dict(q=q, cache=cache, table=torch.zeros(1, 2, dtype=torch.int32, **dev), starts=i32([0, 3]), lens=i32([5]))
    ops.paged_attention(**good)
    for bad in (dict(q=q.float()), dict(table=good["table"].long()), dict(lens=good["lens"].float()),
                dict(cache=ops.PagedCache.empty(4, 2, 16, 64, F16)), dict(out=torch.zeros(3, 4, 64, **dev))):
        with pytest.raises(TypeError):
            ops.paged_attention(**{**good, **bad})
    for bad in (dict(q=q[:, :3]), dict(q=q[:, :, :32]), dict(q=q.transpose(1, 2)), dict(starts=i32([0, 1, 3])),
                dict(lens=i32([5, 5])), dict(window=-1), dict(table=good["table"][0]), dict(starts=good["starts"].cpu())):
        with pytest.raises(ValueError):
            ops.paged_attention(**{**good, **bad})
    for bad in (dict(scale=math.nan), dict(scale=math.inf)):
        with pytest.raises(CbsError):
            ops.paged_attention(**{**good, **bad})
    with pytest.raises(CbsError):  # dim 8: served by the cache, not by the attention
        ops.paged_attention(**{**good, "q": torch.zeros(3, 4, 8, dtype=BF16, **dev),
                               "cache": ops.PagedCache.empty(4, 2, 16, 8)})


def test_served_block(ops):
    """The example: chunks of prompts and single tokens through one block; its error is that of the 8-bit steps
    (four layers and the cache, each near 1 / 254 of its rows' largest, some four times the root mean square)."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import served_block
    assert served_block.main(["--width", "256", "--heads", "4", "--kv-heads", "2", "--prompts", "90", "1", "33",
                              "--chunk", "32", "--decode", "6"]) < 0.05

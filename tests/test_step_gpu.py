"""A step's other operators on the GPU against their definitions in 64 bits."""
import math

import pytest
import torch

import block8_oracle as O
import step_oracle as S

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64, I8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int8, torch.int32
TYPES, TYPE_IDS = [BF16, F16, F32], ["bf16", "f16", "f32"]


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import conv_bn_silu_amd
    return conv_bn_silu_amd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def say(*a):
    print(*a, flush=True)


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


# --- norm -------------------------------------------------------------------

NORM = [
    # M, K: each team's widths and the next one's, odd ones, rows that are read twice (beyond 16384)
    (1, 1), (1, 8), (3, 16), (17, 64), (33, 100), (5, 127), (40, 128), (9, 511), (16, 512), (4, 513), (7, 1999), (3, 2048),
    (5, 2056), (1, 4096), (40, 4096), (2, 8192), (3, 8200), (2, 16384), (2, 16391), (1, 40000), (1, 131072), (1000, 80),
]


def norm_inputs(M, K, dtype, residual, weight, seed):
    g = gen(seed)
    x = torch.randn(M, K, generator=g) * (1 + 8 * (torch.rand(K, generator=g) > 0.95))
    r = None if residual is None else (2 * torch.randn(M, K, generator=g)).to(residual)
    w = None if weight is None else (1 + 0.3 * torch.randn(K, generator=g)).to(weight)
    return x.to(dtype), w, r


def check_norm(ops, x, w, r, eps, what):
    y, tol, h = S.norm(x, w, r, eps)
    to = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = ops.add_rms_norm(to(x), to(w), to(r), eps=eps)
    rows = ops.add_rms_norm(to(x), to(w), to(r), eps=eps, int8=True)
    if r is not None:
        (got, sum1), (rows, sum2) = got, rows
        assert sum1.dtype == r.dtype and torch.equal(sum1.cpu(), h) and torch.equal(sum2.cpu(), h), what
    assert got.dtype == x.dtype and got.shape == x.shape
    O.check(got, y, O.rounded(y, tol, x.dtype), what)
    assert rows.shape == x.shape and rows.dtype == x.dtype
    S.check_codes(rows.codes, rows.scale, y, tol, what)


@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("shape", NORM, ids=lambda s: "x".join(map(str, s)))
def test_norm(ops, shape, dtype):
    M, K = shape
    for i, (r, w) in enumerate(dict.fromkeys([(None, None), (dtype, dtype), (F32, F32), (None, F32), (F32, dtype)])):
        say("[norm]", shape, dtype, r, w)
        check_norm(ops, *norm_inputs(M, K, dtype, r, w, 7 * M + K + i), 1e-6, f"{shape} {dtype} {r} {w}")


@pytest.mark.parametrize("K", [40, 200, 1030, 5000, 20000])
def test_norm_values(ops, K):
    """The largest and smallest numbers, rows of zeros and of one value, an eps that counts."""
    for dtype in TYPES:
        big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
        x, w, r = norm_inputs(7, K, dtype, dtype, dtype, K)
        x[0], r[0] = 0, 0
        x[1], r[1] = big, 0
        x[2], r[2] = tiny, tiny
        x[3], r[3] = big, -big
        x[4], r[4] = -3, 0
        x[5, K // 2], r[5, K // 2] = big / 2, 0
        for eps in (1e-6, 2.0 ** -126, 10.0):
            say("[norm values]", K, dtype, eps)
            check_norm(ops, x, w, r, eps, f"{K} {dtype} {eps}")
            check_norm(ops, x, w, None, eps, f"{K} {dtype} {eps} no residual")


@pytest.mark.parametrize("K", [40, 1030, 5000, 20000])
def test_norm_infinities_and_nan(ops, K):
    """They stay in their rows; an infinity becomes NaN and the row's other numbers zero."""
    x, w, r = norm_inputs(9, K, F32, F32, F32, K)
    y, tol, _ = S.norm(x, w, r, 1e-6)
    bad = {1: math.inf, 3: -math.inf, 4: math.nan}
    for m, v in bad.items():
        (x if m == 3 else r)[m, K // 3] = v
    say("[norm bad values]", K)
    got, h = ops.add_rms_norm(x.cuda(), w.cuda(), r.cuda())
    rows, _ = ops.add_rms_norm(x.cuda(), w.cuda(), r.cuda(), int8=True)
    keep = torch.tensor([m for m in range(9) if m not in bad])
    O.check(got[keep.cuda()], y[keep], O.rounded(y, tol, F32)[keep], "other rows")
    S.check_codes(rows.codes.cpu()[keep], rows.scale.cpu()[keep], y[keep], tol[keep], "other rows")
    got = got.cpu()
    for m in (1, 3):
        assert bool(got[m, K // 3].isnan()) and int(torch.count_nonzero(got[m])) == 1
    assert bool(got[4].isnan().all())
    assert torch.equal(h.cpu().isfinite().sum(-1), torch.tensor([K - (m in bad) for m in range(9)]))
    assert not bool(rows.scale.cpu()[torch.tensor(sorted(bad))].isfinite().any())
    assert bool((rows.codes[torch.tensor(sorted(bad)).cuda()] == 0).all())


@pytest.mark.parametrize("K", [96, 130, 1999, 8192, 17000])
def test_norm_strides_places_and_shapes(ops, K):
    """Strided and unaligned rows, leading axes, the residual updated in its place, other tensors untouched."""
    for dtype, held in ((BF16, BF16), (F16, F32), (F32, F32)):
        M = 6
        x, w, r = norm_inputs(M, K, dtype, held, dtype, K)
        y, tol, h = S.norm(x, w, r, 1e-5)
        tol = O.rounded(y, tol, dtype)
        say("[norm strided]", K, dtype)
        wide = torch.zeros(M, K + 11, dtype=dtype, device="cuda")
        wide[:, 3:3 + K] = x.cuda()
        rwide = torch.zeros(M, 2 * K + 3, dtype=held, device="cuda")
        rwide[:, 1:1 + K] = r.cuda()
        got, s = ops.add_rms_norm(wide[:, 3:3 + K], w.cuda(), rwide[:, 1:1 + K], eps=1e-5)
        O.check(got, y, tol, "strided")
        assert torch.equal(s.cpu(), h) and bool((rwide[:, 1 + K:] == 0).all())
        # in its place, unaligned, with guards
        buf = torch.full((M * K + 2,), 5.0, dtype=held, device="cuda")
        place = buf[1:-1].view(M, K)
        place.copy_(r)
        ybuf = torch.full((M * K + 2,), 7.0, dtype=dtype, device="cuda")
        out = ybuf[1:-1].view(M, K)
        got, s = ops.add_rms_norm(x.cuda(), w.cuda(), place, eps=1e-5, out=out, sum_out=place)
        assert got.data_ptr() == out.data_ptr() and s is place
        O.check(out, y, tol, "in place")
        assert torch.equal(place.cpu(), h) and float(buf[0]) == float(buf[-1]) == 5 and float(ybuf[0]) == float(ybuf[-1]) == 7
        # leading axes, columns first
        got, s = ops.add_rms_norm(x.cuda().t().contiguous().t().view(2, 3, K), w.cuda(), r.cuda().view(2, 3, K), eps=1e-5)
        assert got.shape == s.shape == (2, 3, K)
        O.check(got.view(M, K), y, tol, "leading axes")
        rows = ops.add_rms_norm(x.cuda().view(2, 3, K), w.cuda(), int8=True)
        assert rows.scale.shape == (2, 3) and rows.codes.shape == (2, 3, K)
        one = ops.add_rms_norm(x.cuda()[0], w.cuda())
        assert one.shape == (K,)
        assert tuple(ops.add_rms_norm(x.cuda()[:0], w.cuda()).shape) == (0, K)
        assert ops.add_rms_norm(x.cuda()[:0], w.cuda(), r.cuda()[:0], int8=True)[0].codes.shape == (0, K)


def test_norm_rows_leave_their_padding(ops):
    """What a buffer holds for rows past M, and past it, is not written."""
    from conv_bn_silu_amd import binding as B, step  # noqa: F401  (declares the types)
    M, K = 5, 200
    x, w, _ = norm_inputs(M, K, BF16, None, BF16, 2)
    x, w = x.cuda(), w.cuda()
    need = B.lib.cbs_rows8_bytes(M, K)
    buf = torch.full((need + 64,), 99, dtype=I8, device="cuda")
    h = B.default_library().handle
    st = torch.cuda.current_stream().cuda_stream
    assert B.lib.cbs_add_rms_norm(h, x.data_ptr(), K, None, 0, 1, w.data_ptr(), 1, 1e-6, None, 0, buf.data_ptr(), 3, M, K, 1, st) == 0
    want = ops.add_rms_norm(x, w, int8=True)
    got = ops.Rows8(buf[:need], (M, K), BF16)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scale, want.scale)
    assert bool((buf[need:] == 99).all())
    scales, codes = got._split()
    assert bool((scales[M:].view(I8) == 99).all()) and bool((codes[:, M:] == 99).all())
    assert bool((codes[:, :M].transpose(0, 1).flatten(1)[:, K:] == 0).all())


# --- the linear layer on rows in 8 bits -----------------------------------------

LINEAR = [
    # M, N, K: each kernel's own sizes; K off 16 (a copy of w), few outputs of long sums (K divided)
    (1, 17, 64), (1, 4096, 4096), (3, 64, 130), (16, 500, 1040), (20, 300, 72), (33, 65, 63), (40, 256, 4096), (64, 16400, 640),
    (100, 1030, 8992), (130, 70, 6501), (140, 5000, 1023), (257, 300, 384), (333, 1001, 1999), (1281, 2050, 784), (3500, 3460, 16),
    (3400, 3600, 129),
]


@pytest.mark.parametrize("shape", LINEAR, ids=lambda s: "x".join(map(str, s)))
def test_linear_of_rows(ops, shape):
    """The same bits as from the values that the rows were made of."""
    M, N, K = shape
    g = gen(M + N + K)
    for dtype, act in ((BF16, None), (F32, "silu"), (F16, None)):
        say("[linear of rows]", shape, dtype)
        x = (torch.randn(M, K, generator=g) * (1 + 5 * (torch.rand(K, generator=g) > 0.95))).to(dtype)
        w = torch.randint(-128, 128, (N, K), generator=g, dtype=I32).to(I8).cuda()
        ws = (torch.rand(N, generator=g) * 0.02 + 0.001).cuda()
        b = torch.randn(N, generator=g).cuda() if act else None
        codes, s = O.quantize(x)
        R, Kp = (M + 15) // 16 * 16, (K + 127) // 128 * 128
        buffer = torch.randint(-128, 128, (R * 4 + R * Kp,), generator=g, dtype=I32).to(I8)  # anything past M
        rows = ops.Rows8(buffer, (M, K), dtype)
        scales, blocks = rows._split()
        scales[:M] = s
        full = torch.zeros(M, Kp, dtype=I8)
        full[:, :K] = codes.to(I8)
        blocks[:, :M] = full.view(M, -1, 64).transpose(0, 1)
        rows.buffer = buffer.cuda()
        want = ops.int8_linear(x.cuda(), w, ws, b, act)
        out = torch.empty(M, N, dtype=dtype, device="cuda")
        for kw in ({}, {"out": out}):
            got = ops.int8_linear(rows, w, ws, b, act, **kw)
            assert got.dtype == dtype and torch.equal(got, want), f"{shape} {dtype}"


def test_linear_of_rows_leading_axes_and_empty(ops):
    x, w, _ = norm_inputs(24, 64, BF16, None, None, 1)
    weight, ws = torch.randint(-128, 128, (48, 64), dtype=I32).to(I8).cuda(), torch.rand(48).cuda()
    rows = ops.add_rms_norm(x.cuda().view(2, 3, 4, 64), int8=True)
    flat = ops.add_rms_norm(x.cuda(), int8=True)
    y = ops.int8_linear(rows, weight, ws)
    assert tuple(y.shape) == (2, 3, 4, 48) and torch.equal(y.view(24, 48), ops.int8_linear(flat, weight, ws))
    p = flat.codes.cpu().to(F64) @ weight.cpu().to(F64).t() * (flat.scale.cpu().to(F64)[:, None] * ws.cpu().to(F64))
    O.check(ops.int8_linear(flat, weight, ws), p, O.rounded(p, 4 * O.U32 * p.abs(), BF16), "by the codes")
    assert tuple(ops.int8_linear(ops.add_rms_norm(x.cuda()[:0], int8=True), weight, ws).shape) == (0, 48)


# --- rotary -------------------------------------------------------------------

ROTARY = [
    # tokens, heads, dim, pairs: whole 8s and others, part of the head, one pair, wide heads
    (1, 1, 2, 1), (1, 32, 128, 64), (7, 5, 64, 32), (33, 3, 80, 16), (20, 4, 80, 40), (5, 2, 96, 20), (9, 3, 100, 50), (4, 1, 7, 3),
    (64, 40, 128, 32), (3, 2, 256, 128), (11, 6, 256, 8), (5, 1, 192, 96), (6, 2, 512, 256), (3, 3, 320, 24), (2, 1, 511, 200),
    (300, 1, 16, 8), (2, 130, 64, 32), (2, 1500, 8, 4), (3, 2, 24, 12),
]


def frequencies(pairs):
    return 10000.0 ** (-torch.arange(pairs, dtype=F64) / pairs)


@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("shape", ROTARY, ids=lambda s: "x".join(map(str, s)))
def test_rotary(ops, shape, interleaved, dtype):
    T, H, D, n = shape
    say("[rotary]", shape, interleaved, dtype)
    g = gen(T + H + D)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=I32)
    pos[0] = -5
    f = frequencies(n)
    ref, tol = S.rotate(x, pos, f, interleaved, 1.2)
    tol = O.rounded(ref, tol, dtype)
    # parts of a wider tensor, unaligned
    wide = torch.zeros(T, H + 1, D + 3, dtype=dtype, device="cuda")
    view = wide[:, 1:, 3:]
    view.copy_(x)
    args = (pos.cuda(), f.cuda(), interleaved, 1.2)
    y = ops.rotary(view, *args)
    assert y.shape == x.shape and y.is_contiguous()
    O.check(y, ref, tol, f"{shape}")
    assert torch.equal(y[..., 2 * n:].cpu(), x[..., 2 * n:])
    assert torch.equal(ops.rotary(x.cuda(), *args), y)
    # in place, and into a part of another tensor; nothing else is written
    assert ops.rotary(view, *args, out=view).data_ptr() == view.data_ptr()
    assert torch.equal(view, y)
    view.zero_()
    assert bool((wide == 0).all())
    other = torch.zeros_like(wide)
    ops.rotary(x.cuda(), *args, out=other[:, :H, :D])
    assert torch.equal(other[:, :H, :D], y)
    other[:, :H, :D] = 0
    assert bool((other == 0).all())


def test_rotary_head_major(ops):
    """Heads before tokens: the head stride the larger."""
    T, H, D = 10, 3, 64
    x = torch.randn(H, T, D, generator=gen(1)).to(BF16).cuda()
    pos, f = torch.arange(T, dtype=I32).cuda(), frequencies(32).cuda()
    want = ops.rotary(x.transpose(0, 1).contiguous(), pos, f)
    out = torch.empty_like(x)
    ops.rotary(x.transpose(0, 1), pos, f, out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want)
    ops.rotary(x.transpose(0, 1), pos, f, out=x.transpose(0, 1))
    assert torch.equal(x.transpose(0, 1), want)


def test_rotary_far_positions(ops):
    """Angles of far positions keep their accuracy, to the last position, either sign."""
    f = torch.cat((frequencies(24), torch.tensor([0.0, 1e-30, 3.0, 1000.0], dtype=F64), frequencies(4)))
    pos = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31], dtype=I32)
    x = torch.randn(8, 2, 64, generator=gen(2))
    for interleaved in (False, True):
        ref, tol = S.rotate(x, pos, f, interleaved, 1.0)
        y = ops.rotary(x.cuda(), pos.cuda(), f.cuda(), interleaved)
        O.check(y, ref, O.rounded(ref, tol, F32), f"far {interleaved}")
        assert torch.equal(y[0].cpu(), x[0])


def test_rotary_many_tokens_and_values(ops):
    """More tokens than a workgroup's share; infinities and NaN stay in their pairs."""
    T, H, D = 5003, 3, 32
    x = torch.randn(T, H, D, generator=gen(3)).to(BF16)
    pos = torch.arange(T, dtype=I32)
    ref, tol = S.rotate(x, pos, frequencies(16), False, 1.0)
    y = ops.rotary(x.cuda(), pos.cuda(), frequencies(16).cuda())
    O.check(y, ref, O.rounded(ref, tol, BF16), "many tokens")
    x[17, 1, 3], x[99, 2, 20] = math.inf, math.nan
    z = ops.rotary(x.cuda(), pos.cuda(), frequencies(16).cuda())
    z, y = z.cpu(), y.cpu()
    for t, h, a in ((17, 1, 3), (99, 2, 4)):
        assert not bool(z[t, h, [a, a + 16]].isfinite().any())
        z[t, h, [a, a + 16]] = y[t, h, [a, a + 16]]
    assert torch.equal(z, y)
    assert tuple(ops.rotary(x.cuda()[:0], pos.cuda()[:0], frequencies(16).cuda()).shape) == (0, H, D)


ROTARY_CACHE = [
    # tokens, heads, kv heads, dim, pairs, page
    (1, 1, 1, 8, 4, 1), (64, 32, 8, 128, 64, 16), (37, 15, 5, 80, 16, 24), (20, 4, 4, 80, 40, 17), (9, 3, 1, 96, 20, 32),
    (11, 8, 2, 256, 128, 128), (5, 0, 3, 64, 32, 16), (7, 2, 2, 136, 64, 7), (30, 6, 3, 24, 12, 64), (6, 5, 1, 200, 33, 16),
]


@pytest.mark.parametrize("held", [I8, BF16, F16, F32], ids=["i8", "hbf16", "hf16", "hf32"])
@pytest.mark.parametrize("dtype", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("shape", ROTARY_CACHE, ids=lambda s: "x".join(map(str, s)))
def test_rotary_cache_write(ops, shape, dtype, held):
    T, H, Hk, D, n, P = shape
    for interleaved in (False, True):
        say("[rotary cache]", shape, dtype, held, interleaved)
        g = gen(T + H + D)
        fused = torch.randn(T, H + 2 * Hk, D, generator=g).to(dtype)
        q, k, v = fused.split([H, Hk, Hk], 1)
        pos = torch.randint(0, 100000, (T,), generator=g, dtype=I32)
        pages = (T + P - 1) // P + 3
        slots = torch.randperm(pages * P, generator=g)[:T].to(I32)
        slots[6::7] = -1
        if T > 3:
            slots[3] = pages * P  # just past the cache
        cache = ops.PagedCache.empty(pages, Hk, P, D, held)
        cache.k.fill_(3)
        cache.v.fill_(3)
        f = frequencies(n)
        on = fused.cuda()
        parts = on.split([H, Hk, Hk], 1)
        args = (pos.cuda(), slots.cuda(), f.cuda(), interleaved, 0.9)
        out = ops.rotary_cache_write(cache, *parts, *args)
        ref, tol = S.rotate(q, pos, f, interleaved, 0.9)
        O.check(out, ref, O.rounded(ref, tol, dtype), f"queries {shape}")
        assert torch.equal(on.cpu(), fused)
        there = (slots >= 0) & (slots < pages * P)
        at = slots[there].long()
        pg, off = at // P, at % P
        kr, kt = S.rotate(k, pos, f, interleaved, 0.9)
        for what, held_t, scale, y, t in (("keys", cache.k, cache.k_scale, kr, kt), ("values", cache.v, cache.v_scale, v.to(F64), 0 * kt)):
            got = held_t.cpu()[pg, :, off]
            if held == I8:
                S.check_codes(got, scale.cpu()[pg, :, off], y[there], t[there], f"{what} {shape}")
            else:
                O.check(got, y[there], O.rounded(y, t, held)[there], f"{what} {shape}")
        if held == I8:  # values are what cache_write makes of them
            codes, s = O.quantize(v)
            assert torch.equal(cache.v.cpu()[pg, :, off].double(), codes[there]) and torch.equal(cache.v_scale.cpu()[pg, :, off], s[there])
        free = torch.ones(pages * P, dtype=torch.bool)
        free[at] = False
        u = free.nonzero()[:, 0]
        assert bool((cache.k.cpu()[u // P, :, u % P] == 3).all()) and bool((cache.v.cpu()[u // P, :, u % P] == 3).all())
        # the queries in their place, between the keys and values
        again = ops.PagedCache.empty(pages, Hk, P, D, held)
        ops.rotary_cache_write(again, *parts, *args, out=parts[0])
        assert torch.equal(parts[0], out) and torch.equal(on[:, H:].cpu(), fused[:, H:])
        assert torch.equal(again.k.cpu()[pg, :, off], cache.k.cpu()[pg, :, off])


@pytest.mark.parametrize("T", [1, 6])
def test_rotary_cache_layouts(ops, T):
    """Queries turned in their place beside the keys and values of their token, of their head, and head by head."""
    H, D = 4, 64
    g = gen(T)
    q, k, v = (torch.randn(T, H, D, generator=g).to(BF16).cuda() for _ in range(3))
    pos, slots, f = torch.arange(T, dtype=I32).cuda(), torch.arange(T, dtype=I32).cuda(), frequencies(32).cuda()
    cache = ops.PagedCache.empty(2, H, 16, D)
    want = ops.rotary_cache_write(cache, q, k, v, pos, slots, f)
    for how in ("tokens", "heads", "three", "head major"):
        if how == "tokens":
            parts = torch.cat((q, k, v), 1).split(H, 1)
        elif how == "heads":  # [tokens, heads, 3, dim]
            parts = torch.stack((q, k, v), 2).unbind(2)
        elif how == "three":  # [tokens, 3, heads, dim]
            parts = torch.stack((q, k, v), 1).unbind(1)
        else:  # [heads, 3, tokens, dim]
            parts = [t.transpose(0, 1) for t in torch.stack([t.transpose(0, 1) for t in (q, k, v)], 1).unbind(1)]
        again = ops.PagedCache.empty(2, H, 16, D)
        got = ops.rotary_cache_write(again, *parts, pos, slots, f, out=parts[0])
        assert got.data_ptr() == parts[0].data_ptr()
        assert torch.equal(got, want) and torch.equal(parts[1], k) and torch.equal(parts[2], v), how
        assert torch.equal(again.k, cache.k) and torch.equal(again.v, cache.v) and torch.equal(again.k_scale, cache.k_scale), how


def test_rotary_cache_special_rows(ops):
    """Keys of zeros, infinities, NaN and of the smallest numbers; unaligned tensors."""
    T, H, D, P = 8, 2, 24, 4
    x = torch.randn(T, 3 * H, D, generator=gen(1))
    x[0] = 0
    x[1, H:, 5] = math.inf
    x[2, H:, 3] = math.nan
    x[3] = 2.0 ** -130
    buf = torch.zeros(x.numel() + 1, device="cuda")
    on = buf[1:].view(x.shape)
    on.copy_(x)
    q, k, v = on.split([H] * 3, 1)
    pos, slots = torch.arange(T, dtype=I32).cuda(), torch.arange(T, dtype=I32).cuda()
    cache = ops.PagedCache.empty(4, H, P, D)
    ops.rotary_cache_write(cache, q, k, v, pos, slots, frequencies(8).cuda())
    kr, kt = S.rotate(x[:, H:2 * H], pos.cpu(), frequencies(8), False, 1.0)
    back = ops.cache_read(cache, slots, F32)
    fine = torch.tensor([0, 3, 4, 5, 6, 7])
    page, off = fine // P, fine % P
    S.check_codes(cache.k.cpu()[page, :, off], cache.k_scale.cpu()[page, :, off], kr[fine], kt[fine], "special keys")
    for y in back:
        assert bool(y[1:3].isnan().all()) and bool(y[fine.cuda()].isfinite().all())


# --- pages ----------------------------------------------------------------------

def pages_case(lens, page, width, spare, seed, scatter=True):
    """Tables of the given lengths over a cache with `spare` free pages."""
    g = gen(seed)
    used = [min(-(-max(n, 0) // page), width) for n in lens]
    pages = max(1, sum(used) + spare)
    order = torch.randperm(pages, generator=g).tolist() if scatter else list(range(pages))
    table, at = [], 0
    for u in used:
        table.append(order[at:at + u] + [-1] * (width - u))
        at += u
    free = order[at:] + [-7] * at
    return S.Pages(free, pages - at, page, table, lens)


def on_device(ops, s, width):
    pool = ops.PagePool(i32(s.below), i32([s.count, 0, 0]), s.page)
    table = torch.full((len(s.table), width + 3), -9, dtype=I32, device="cuda")[:, :width]
    if s.table and width:
        table.copy_(torch.tensor(s.table, dtype=I32))
    return pool, table, i32(s.lens)


def check_state(pool, table, lens, s, what):
    assert table.tolist() == s.table, what
    assert lens.tolist() == s.lens, what
    assert pool.free.tolist() == s.below, what
    assert list(pool.report()) == s.counts(), what


PAGES = [
    # lens, more, page, width, spare, padding: one workgroup and several, by tokens and by sequences
    ([0], [1], 1, 1, 1, 0), ([5], [0], 4, 8, 3, 2), ([0, 0, 0], [7, 0, 9], 4, 5, 9, 3), ([17, 3, 40, 0], [1, 1, 1, 1], 16, 8, 20, 0),
    ([31, 32, 33], [1, 1, 1], 16, 4, 9, 5), ([0] * 70, [3] * 70, 2, 4, 200, 0), ([100, 0, 7], [5000, 4000, 1], 24, 300, 500, 9),
    ([0, 50], [30000, 3], 17, 2000, 2000, 0), (list(range(1500)), [1] * 1500, 16, 100, 2000, 7),
    ([0] * 2100, [i % 3 for i in range(2100)], 3, 2, 2200, 100), ([0] * 1024, [8] * 1024, 16, 1, 1024, 0),
    ([9] * 1025, [1] * 1025, 10, 2, 100, 0), ([0] * 3, [0] * 3, 16, 4, 4, 10), ([10], [9000], 7, 1300, 1300, 8000),
]


@pytest.mark.parametrize("case", range(len(PAGES)))
def test_pages_grow_and_release(ops, case):
    lens, more, page, width, spare, padding = PAGES[case]
    s = pages_case(lens, page, width, spare, case)
    pool, table, dlens = on_device(ops, s, width)
    say("[pages]", case)
    for turn in range(3):
        tokens = sum(more) + padding
        want = s.grow(more, tokens)
        got = ops.grow_pages(pool, table, dlens, i32(more), tokens)
        for name, w, g in zip(("starts", "slots", "positions"), want, got):
            assert g.tolist() == w, f"{name} {turn}"
        check_state(pool, table, dlens, s, f"grown {turn}")
        if turn == 1:  # some end, some are cut back, some stay
            keep = [[0, n, max(0, n - 3), 2 ** 31 - 1, n // 2][b % 5] for b, n in enumerate(s.lens)]
            s.release(keep)
            ops.release_pages(pool, table, dlens, i32(keep))
            check_state(pool, table, dlens, s, f"released {turn}")
    keep = [0] * len(lens)
    s.release(keep)
    ops.release_pages(pool, table, dlens, i32(keep))
    check_state(pool, table, dlens, s, "all released")
    assert not table.numel() or bool((table == -1).all())


@pytest.mark.parametrize("n", [5, 1100], ids=["few", "many"])
def test_pages_that_lack(ops, n):
    """Too few pages, rows of the table that are too short, tokens past the batch, each alone and together; then it
    goes on."""
    g = gen(n)
    lens = torch.randint(0, 50, (n,), generator=g).tolist()
    more = torch.randint(0, 12, (n,), generator=g).tolist()
    for spare, width, cut in ((n // 3, 9, 0), (4 * n, 9, 17), (4 * n, 13, 0), (n // 2, 9, 9), (0, 9, 0)):
        s = pages_case([min(x, width * 4) for x in lens], 4, width, spare, 3)
        pool, table, dlens = on_device(ops, s, width)
        wide = list(more)
        wide[n // 2] = 70  # passes its row
        tokens = max(0, sum(wide) - cut)
        say("[pages lack]", n, spare, width, cut)
        for turn in range(2):
            want = s.grow(wide, tokens)
            got = ops.grow_pages(pool, table, dlens, i32(wide), tokens)
            assert [x.tolist() for x in got] == list(want)
            check_state(pool, table, dlens, s, f"{spare} {width} {cut} {turn}")
            assert s.left > 0
            keep = [x // 2 for x in s.lens]
            s.release(keep)
            ops.release_pages(pool, table, dlens, i32(keep))
            check_state(pool, table, dlens, s, "released")


def test_pages_take_and_give_back(ops):
    """What is taken and given back at once leaves the pool as it was, order included."""
    for lens, more in (([33, 0, 7, 100], [40, 9, 0, 1]), ([5] * 1300, [30] * 1300)):
        s = pages_case(lens, 8, 20, 6000, 1)
        pool, table, dlens = on_device(ops, s, 20)
        free, before = pool.free.clone(), table.clone()
        ops.grow_pages(pool, table, dlens, i32(more), sum(more))
        assert pool.report()[1:] == (0, 0) and dlens.tolist() == [a + b for a, b in zip(lens, more)]
        ops.release_pages(pool, table, dlens, i32(lens))
        assert torch.equal(pool.free, free) and torch.equal(table, before) and dlens.tolist() == lens
        assert pool.report()[0] == s.count


def test_pages_of_bad_contents(ops):
    """Lengths, counts and page numbers that cannot be: nothing goes out of the tensors, and where pages lie outside
    the pool no slot does."""
    guard = 64
    big = 2 ** 31 - 1
    for n in (4, 1200):
        g = gen(n)
        free = torch.full((2 * guard + 50,), 11, dtype=I32, device="cuda")
        tables = torch.full((2 * guard + n * 6,), 12, dtype=I32, device="cuda")
        stack, table = free[guard:-guard], tables[guard:-guard].view(n, 6)
        stack.copy_(torch.randint(-3, 60, (50,), generator=g))
        table.copy_(torch.randint(-5, 60, (n, 6), generator=g))
        for count in (-5, 50, 51, big, -big):
            for length in (-1, 10, 40, big):
                say("[pages bad]", n, count, length)
                pool = ops.PagePool(stack, i32([count, 0, 0]), 4)
                lens = torch.full((n,), length, dtype=I32, device="cuda")
                more = i32([[1, big, -3, 7][b % 4] for b in range(n)])
                starts, slots, positions = ops.grow_pages(pool, table, lens, more, 100)
                slots = slots.cpu()
                assert bool(((slots >= -1) & (slots < 200)).all())
                assert starts.tolist() == sorted(starts.tolist()) and int(starts[-1]) <= 100
                ops.release_pages(pool, table, lens, i32([[0, -4, 3, big][b % 4] for b in range(n)]))
                assert 0 <= pool.report()[0] <= 50
                for t, v in ((free, 11), (tables, 12)):
                    assert bool((t[:guard] == v).all()) and bool((t[-guard:] == v).all())
    # a hole in a row, and one in the stack
    s = S.Pages([3, -1, 9, 2], 4, 4, [[0, 99, -1, -1, -1]], [6])
    pool, table, lens = on_device(ops, s, 5)
    want = s.grow([12], 12)
    got = ops.grow_pages(pool, table, lens, i32([12]), 12)
    # of 4 pages: tokens 6 and 7 on page 99, 12 to 15 on page 9, 16 and 17 on page -1
    assert [x.tolist() for x in got] == list(want) and want[1].count(-1) == 8
    check_state(pool, table, lens, s, "holes")


def test_pages_empty_batch(ops):
    pool = ops.PagePool.full(4, 16)
    assert pool.free.tolist() == [3, 2, 1, 0]
    table, none = torch.zeros(0, 5, dtype=I32, device="cuda"), torch.zeros(0, dtype=I32, device="cuda")
    starts, slots, positions = ops.grow_pages(pool, table, none, none, 3)
    assert starts.tolist() == [0] and slots.tolist() == [-1] * 3 and positions.tolist() == [0] * 3
    ops.release_pages(pool, table, none, none)
    narrow = torch.zeros(2, 0, dtype=I32, device="cuda")
    starts, slots, _ = ops.grow_pages(pool, narrow, i32([0, 0]), i32([1, 0]), 0)
    assert starts.tolist() == [0, 0, 0] and slots.numel() == 0 and pool.report() == (4, 0, 1)


# --- together, and what calls promise ------------------------------------------

def step(ops, s):
    """A step of a block's first half."""
    starts, slots, positions = ops.grow_pages(s["pool"], s["table"], s["lens"], s["more"], s["tokens"])
    rows, s["h"] = ops.add_rms_norm(s["x"], s["norm"], s["h"], int8=True, sum_out=s["h"])
    H, Hk, D = s["heads"], s["cache"].heads, s["cache"].dim
    qkv = ops.int8_linear(rows, *s["qkv"]).view(-1, H + 2 * Hk, D)
    q, k, v = qkv.split([H, Hk, Hk], 1)
    ops.rotary_cache_write(s["cache"], q, k, v, positions, slots, s["frequencies"], out=q)
    a = ops.paged_attention(q, s["cache"], s["table"], starts, s["lens"])
    s["x"].copy_(ops.int8_linear(a.view(s["tokens"], -1), *s["out"]))


def step_state(ops, seed=0):
    """Sequences of several lengths, one of them idle, a batch padded by one row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731

    def weight(n, k):
        w = normal(n, k) / math.sqrt(k)
        ws = w.abs().amax(-1) / 127
        return torch.round(w / ws[:, None]).to(I8), ws

    B, width, H, Hk, D, P, W = 4, 12, 4, 2, 64, 16, 256
    s = {"cache": ops.PagedCache.empty(40, Hk, P, D), "pool": ops.PagePool.full(40, P), "heads": H, "tokens": 4,
         "table": torch.full((B, width), -1, dtype=I32, device="cuda"), "lens": i32([0] * B), "more": i32([1, 1, 0, 1]),
         "norm": (1 + 0.1 * normal(W)).to(BF16), "qkv": weight((H + 2 * Hk) * D, W), "out": weight(W, H * D),
         "frequencies": ops.rotary_frequencies(D)}
    prompts = [30, 15, 9, 16]
    starts, slots, positions = ops.grow_pages(s["pool"], s["table"], s["lens"], i32(prompts), sum(prompts))
    k, v = (normal(sum(prompts), Hk, D).to(BF16) for _ in range(2))
    ops.rotary_cache_write(s["cache"], normal(sum(prompts), H, D).to(BF16), k, v, positions, slots, s["frequencies"])
    s["x"], s["h"] = normal(4, W).to(BF16), normal(4, W).to(BF16)
    return s


def values(s):
    return [s["x"][:3], s["h"][:3], s["table"], s["lens"], s["pool"].free, s["pool"].counts, s["cache"].k, s["cache"].v,
            s["cache"].k_scale, s["cache"].v_scale]


def test_a_step_together_in_a_graph(ops):
    """Decoding steps captured once and replayed, pages taken as they are needed, against the same steps by
    themselves, with other work between; two such graphs of states of their own beside each other."""
    eager, states, graphs = [step_state(ops, i) for i in range(2)], [step_state(ops, i) for i in range(2)], []
    for s in states:
        start = [t.clone() for t in values(s)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(ops, s)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(ops, s)
        graphs.append(graph)
        for t, v in zip(values(s), start):
            t.copy_(v)
    for i in range(20):
        for s, graph in zip(states, graphs):
            graph.replay()
        for e in eager:
            step(ops, e)
        torch.cuda.synchronize()
        for e, s in zip(eager, states):
            for a, b in zip(values(e), values(s)):
                assert torch.equal(a, b), i
    assert eager[0]["lens"].tolist() == [50, 35, 9, 36] and eager[0]["pool"].report()[0] == 40 - 4 - 3 - 1 - 3


def test_a_step_by_the_definitions(ops):
    """One step's pieces in 64 bits, from the values that each piece was given."""
    s = step_state(ops, 3)
    x, h0 = s["x"].cpu(), s["h"].cpu()
    old, free = s["lens"].tolist(), s["pool"].report()[0]
    page = S.Pages(s["pool"].free.tolist(), free, 16, s["table"].tolist(), old)
    want = page.grow([1, 1, 0, 1], 4)
    step(ops, s)
    assert s["table"].tolist() == page.table and s["lens"].tolist() == page.lens
    y, tol, h = S.norm(x, s["norm"].cpu(), h0, 1e-6)
    assert torch.equal(s["h"].cpu(), h)
    rows = ops.add_rms_norm(x.cuda(), s["norm"], h0.cuda(), int8=True)[0]
    S.check_codes(rows.codes, rows.scale, y, tol, "norm")
    qkv = ops.int8_linear(rows, *s["qkv"]).view(4, 8, 64).cpu()
    kr, kt = S.rotate(qkv[:3, 4:6], torch.tensor(want[2][:3]), s["frequencies"].cpu(), False, 1.0)
    at = torch.tensor(want[1][:3])
    S.check_codes(s["cache"].k.cpu()[at // 16, :, at % 16], s["cache"].k_scale.cpu()[at // 16, :, at % 16], kr, kt, "keys")


def test_side_stream_and_determinism(ops):
    x, w, r = (t.cuda() for t in norm_inputs(300, 4096, BF16, BF16, BF16, 1))
    q = torch.randn(300, 12, 128, generator=gen(2)).to(BF16).cuda()
    pos, slots, f = torch.arange(300, dtype=I32).cuda(), torch.arange(300, dtype=I32).cuda(), frequencies(64).cuda()

    def run():
        cache = ops.PagedCache.empty(20, 2, 16, 128)
        pool = ops.PagePool.full(2000, 16)
        table, lens = torch.full((300, 8), -1, dtype=I32, device="cuda"), torch.zeros(300, dtype=I32, device="cuda")
        rows, h = ops.add_rms_norm(x, w, r, int8=True)
        y, _ = ops.add_rms_norm(x, w, r)
        a = ops.rotary_cache_write(cache, q[:, :8], q[:, 8:10], q[:, 10:], pos, slots, f)
        return [rows.codes, rows.scale, h, y, a, cache.k, cache.v, cache.k_scale, *ops.grow_pages(pool, table, lens, pos % 40, 6000), table, lens]

    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(want, run()))


def test_refusals(ops):
    from conv_bn_silu_amd.binding import CbsError
    dev = dict(device="cuda")
    x, w, r = torch.zeros(4, 64, dtype=BF16, **dev), torch.zeros(64, dtype=BF16, **dev), torch.zeros(4, 64, dtype=BF16, **dev)
    for bad in (dict(x=x.double()), dict(weight=w.half()), dict(residual=r.half()), dict(weight=w.double()), dict(x=None),
                dict(out=torch.zeros(4, 64, **dev)), dict(sum_out=torch.zeros(4, 64, **dev))):
        with pytest.raises(TypeError):
            ops.add_rms_norm(**{**dict(x=x, weight=w, residual=r), **bad})
    for bad in (dict(weight=w[:63]), dict(residual=r[:3]), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
                dict(eps=1e-45), dict(out=r[:3]), dict(int8=True, out=torch.zeros_like(x)), dict(x=x.cpu()),
                dict(residual=None, sum_out=r), dict(weight=torch.zeros(128, dtype=BF16, **dev)[::2]),
                dict(x=torch.zeros(4, 64, dtype=BF16, requires_grad=True, **dev)), dict(x=x[0, 0]), dict(x=x[:, :0]),
                dict(sum_out=torch.zeros(4, 128, dtype=BF16, **dev)[:, ::2])):
        with pytest.raises(ValueError):
            ops.add_rms_norm(**{**dict(x=x, weight=w, residual=r), **bad})
    buf = torch.zeros(5 * 64, dtype=BF16, **dev)
    for bad in (dict(out=x), dict(out=r), dict(sum_out=x), dict(residual=buf[:256].view(4, 64), sum_out=buf[64:].view(4, 64)),
                dict(out=buf[:256].view(4, 64), sum_out=buf[64:].view(4, 64))):
        with pytest.raises(CbsError):  # outputs over inputs or each other
            ops.add_rms_norm(**{**dict(x=x, weight=w, residual=r), **bad})
    with pytest.raises(CbsError):
        ops.add_rms_norm(torch.zeros(1, 131080, **dev))

    rows = ops.add_rms_norm(x, w, int8=True)
    lw, ls = torch.zeros(8, 64, dtype=I8, **dev), torch.zeros(8, **dev)
    ops.int8_linear(rows, lw, ls)
    for bad in (dict(w=lw[:, :32]), dict(w_scale=ls[:7]), dict(bias=ls.cpu()), dict(activation="gelu"), dict(out=x),
                dict(x=ops.Rows8(rows.buffer[:-16], (4, 64), BF16)), dict(x=ops.Rows8(rows.buffer, (17, 64), BF16)),
                dict(x=ops.Rows8(rows.buffer.cpu(), (4, 64), BF16))):
        with pytest.raises(ValueError):
            ops.int8_linear(**{**dict(x=rows, w=lw, w_scale=ls), **bad})
    for bad in (dict(w=lw.float()), dict(x=ops.Rows8(rows.buffer, (4, 64), I8)), dict(x=ops.Rows8(rows.buffer.float(), (4, 64), BF16)),
                dict(out=torch.zeros(4, 8, **dev))):
        with pytest.raises(TypeError):
            ops.int8_linear(**{**dict(x=rows, w=lw, w_scale=ls), **bad})

    q, pos, f = torch.zeros(3, 4, 64, dtype=BF16, **dev), i32([0, 1, 2]), torch.zeros(32, dtype=F64, **dev)
    for bad in (dict(x=q.double()), dict(positions=pos.long()), dict(frequencies=f.float()), dict(out=q.float())):
        with pytest.raises(TypeError):
            ops.rotary(**{**dict(x=q, positions=pos, frequencies=f), **bad})
    for bad in (dict(x=q[0]), dict(x=q.transpose(1, 2)), dict(positions=pos[:2]), dict(frequencies=torch.zeros(33, dtype=F64, **dev)),
                dict(frequencies=f[:0]), dict(frequencies=f[::2]), dict(magnitude=math.nan), dict(out=q[:2]), dict(x=q[:, :0]),
                dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            ops.rotary(**{**dict(x=q, positions=pos, frequencies=f), **bad})
    long = torch.zeros(4, 4, 64, dtype=BF16, **dev)
    over = torch.zeros(3 * 64, dtype=BF16, **dev).as_strided((3, 4, 64), (64, 0, 1))
    for bad in (dict(x=long[:3], out=long[1:]), dict(x=torch.zeros(1, 1, 514, **dev), positions=pos[:1]), dict(out=over),
                dict(x=torch.zeros(3, 65537, 2, **dev), frequencies=f[:1]),
                dict(x=long[:3], out=long.view(-1)[8:8 + 768].view(3, 4, 64))):
        with pytest.raises(CbsError):
            ops.rotary(**{**dict(x=q, positions=pos, frequencies=f), **bad})

    cache = ops.PagedCache.empty(4, 2, 16, 64)
    fused = torch.zeros(3, 8, 64, dtype=BF16, **dev)
    good = dict(cache=cache, q=fused[:, :4], k=fused[:, 4:6], v=fused[:, 6:], positions=pos, slots=pos, frequencies=f)
    ops.rotary_cache_write(**good)
    for bad in (dict(k=fused[:, 4:6].half()), dict(slots=pos.long()), dict(q=fused[:, :4].double())):
        with pytest.raises(TypeError):
            ops.rotary_cache_write(**{**good, **bad})
    for bad in (dict(k=fused[:, 4:5]), dict(v=fused[:2, 6:]), dict(q=fused[:, :4, :32]), dict(slots=pos[:2]), dict(positions=pos[:2]),
                dict(out=fused[:, :3])):
        with pytest.raises(ValueError):
            ops.rotary_cache_write(**{**good, **bad})
    for bad in (dict(out=fused[:, 1:5]), dict(out=fused[:, 4:]), dict(out=fused[:, 3:7])):  # over q's, k's or v's rows
        with pytest.raises(CbsError):
            ops.rotary_cache_write(**{**good, **bad})

    pool = ops.PagePool.full(8, 16)
    table, lens = torch.zeros(2, 4, dtype=I32, **dev), i32([0, 0])
    grow = dict(pool=pool, table=table, lens=lens, more=i32([1, 1]), tokens=2)
    for bad in (dict(table=table.long()), dict(lens=lens.float()), dict(more=lens.long())):
        with pytest.raises(TypeError):
            ops.grow_pages(**{**grow, **bad})
    for bad in (dict(table=table[0]), dict(table=table.t().contiguous().t()), dict(lens=i32([0])), dict(more=i32([1])), dict(tokens=-1),
                dict(tokens=2 ** 31), dict(lens=lens.cpu()), dict(table=table[:1].expand(2, 4))):
        with pytest.raises(ValueError):
            ops.grow_pages(**{**grow, **bad})
    for bad in (dict(more=lens), dict(lens=pool.free[:2]), dict(table=pool.free.view(2, 4))):
        with pytest.raises(CbsError):
            ops.grow_pages(**{**grow, **bad})
    with pytest.raises(CbsError):
        ops.release_pages(pool, table, lens, lens)
    for bad in ((torch.zeros(0, dtype=I32, **dev), i32([0, 0, 0]), 16), (i32([1, 2]), i32([2, 0]), 16), (i32([1, 2]), i32([2, 0, 0]), 0),
                (i32([1, 2]), i32([2, 0, 0]), 2 ** 30 + 1), (i32([[1, 2]]), i32([2, 0, 0]), 16)):
        with pytest.raises(ValueError):
            ops.PagePool(*bad)
    with pytest.raises(TypeError):
        ops.PagePool(i32([1]).long(), i32([1, 0, 0]), 16)
    t = pool.counts
    t.data = torch.zeros_like(t)
    with pytest.raises(ValueError, match="other memory"):
        ops.grow_pages(**grow)

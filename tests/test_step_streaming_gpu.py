"""Tensors beyond what the memory-side cache holds, which pass by the caches: each such kernel against the definitions at some
rows, and bit for bit against smaller calls, which do not stream, at all of them."""
import pytest
import torch

import block8_oracle as O
import step_oracle as S

pytestmark = pytest.mark.gpu

BF16, F16, F32, F64, I8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int8, torch.int32
CACHED = 256 << 20  # bytes from which on tensors stream


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    import conv_bn_silu_amd
    yield conv_bn_silu_amd
    torch.cuda.empty_cache()


def say(*a):
    print(*a, flush=True)


def size(dtype):
    return torch.finfo(dtype).bits // 8


def normal(g, *shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


TYPES = [(BF16, BF16, BF16), (F16, F32, F16), (F32, F32, F32), (BF16, F32, F32), (BF16, None, F32), (F16, None, None), (F32, None, F32)]


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join("none" if x is None else str(x)[6:] for x in t))
@pytest.mark.parametrize("K", [104, 200, 400, 1000, 2056, 8192, 8200, 16384, 16392, 20480, 131072])
def test_norm_streams(ops, K, types):
    dtype, held, weight = types
    each = K * (size(dtype) + (2 * size(held) if held else 0))  # of a row, into 8 bits; 16 and 32 bits are more
    M = CACHED // each + 5
    g = torch.Generator(device="cuda").manual_seed(K)
    say("[norm streams]", M, K, types)
    x = normal(g, M, K, dtype=dtype)
    r = normal(g, M, K, dtype=held) if held else None
    w = (1 + 0.2 * normal(g, K, dtype=F32)).to(weight) if weight else None
    at = torch.tensor(sorted({0, 1, 63, 64, M // 2, M // 3, M - 65, M - 2, M - 1}), device="cuda").clamp(0, M - 1)
    take = lambda t: None if t is None else t[at].cpu()  # noqa: E731
    y, tol, h = S.norm(take(x), None if w is None else w.cpu(), take(r), 1e-6)
    part = M // 5 + 1  # far below the border
    small = [[ops.add_rms_norm(x[m:m + part], w, None if r is None else r[m:m + part], int8=int8) for m in range(0, M, part)]
             for int8 in (False, True)]

    rows = ops.add_rms_norm(x, w, r, int8=True)
    if held:
        rows, s = rows
        assert torch.equal(s[at].cpu(), h) and torch.equal(s, torch.cat([p[1] for p in small[1]]))
        small[1] = [p[0] for p in small[1]]
        del s
    codes = rows.codes
    S.check_codes(codes[at], rows.scale[at], y, tol, f"{K} {types}")
    assert torch.equal(codes, torch.cat([p.codes for p in small[1]])) and torch.equal(rows.scale, torch.cat([p.scale for p in small[1]]))
    del rows, codes
    got = ops.add_rms_norm(x, w, r, sum_out=r)  # in the residual's place
    if held:
        got, s = got
        assert s is r and torch.equal(r[at].cpu(), h) and torch.equal(r, torch.cat([p[1] for p in small[0]]))
        small[0] = [p[0] for p in small[0]]
    O.check(got[at], y, O.rounded(y, tol, dtype), f"{K} {types}")
    assert torch.equal(got, torch.cat(small[0]))


ROTARY = [
    # heads, kv heads (0: no cache), dim, pairs, type, cache's type
    (32, 8, 128, 64, BF16, I8), (32, 8, 128, 64, F32, I8), (16, 4, 256, 128, BF16, I8), (16, 4, 256, 32, F16, F16), (6, 3, 64, 32, F16, I8),
    (32, 8, 128, 64, F32, F32), (40, 8, 64, 16, BF16, F32), (24, 0, 64, 32, F32, None), (8, 0, 512, 256, BF16, None), (5, 0, 200, 40, F16, None),
    (12, 0, 256, 128, F32, None), (40, 0, 128, 32, BF16, None), (9, 1, 136, 64, BF16, BF16),
]


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("case", ROTARY, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_rotary_streams(ops, case, interleaved):
    """Parts of a wider tensor that begins off 16 bytes; queries into a new tensor and in their place."""
    H, Hk, D, n, dtype, held = case
    rows, P = H + 2 * Hk, 16
    T = CACHED // (rows * D * 2 * size(dtype)) + 9
    T = (T + P - 1) // P * P
    say("[rotary streams]", T, case, interleaved)
    g = torch.Generator(device="cuda").manual_seed(D)
    wide = torch.empty(T * rows * D + 1, dtype=dtype, device="cuda")[1:].view(T, rows, D)
    wide.normal_(generator=g)
    before = wide.clone()
    pos = torch.randint(0, 200000, (T,), generator=g, device="cuda", dtype=I32)
    slots = torch.randperm(T, generator=g, device="cuda").to(I32)
    f = 10000.0 ** (-torch.arange(n, dtype=F64, device="cuda") / n)
    at = torch.tensor([0, 1, T // 2, T // 3, T - 2, T - 1], device="cuda")
    ref, tol = S.rotate(wide[at].cpu(), pos[at].cpu(), f.cpu(), interleaved, 1.1)
    how = f, interleaved, 1.1
    part = T // 5 + 1
    parts = [slice(t, min(t + part, T)) for t in range(0, T, part)]
    if not Hk:
        y = ops.rotary(wide, pos, *how)
        O.check(y[at], ref, O.rounded(ref, tol, dtype), f"{case}")
        assert torch.equal(y, torch.cat([ops.rotary(wide[t], pos[t], *how) for t in parts]))
        ops.rotary(wide, pos, *how, out=wide)
        assert torch.equal(wide, y)
        return
    q, k, v = wide.split([H, Hk, Hk], 1)
    caches = [ops.PagedCache.empty(T // P, Hk, P, D, held) for _ in range(3)]
    y = ops.rotary_cache_write(caches[0], q, k, v, pos, slots, *how)
    O.check(y[at], ref[:, :H], O.rounded(ref, tol, dtype)[:, :H], f"{case}")
    assert torch.equal(y, torch.cat([ops.rotary_cache_write(caches[1], q[t], k[t], v[t], pos[t], slots[t], *how) for t in parts]))
    ops.rotary_cache_write(caches[2], q, k, v, pos, slots, *how, out=q)
    assert torch.equal(q, y) and torch.equal(wide[:, H:], before[:, H:])
    for c in caches[1:]:
        for a, b in zip((caches[0].k, caches[0].v, caches[0].k_scale, caches[0].v_scale), (c.k, c.v, c.k_scale, c.v_scale)):
            assert a is None or torch.equal(a, b)
    page, off = slots[at].long() // P, slots[at].long() % P
    values = before[at, H + Hk:].cpu().to(F64)
    for what, t, s, y, tl in (("keys", caches[0].k, caches[0].k_scale, ref[:, H:H + Hk], tol[:, H:H + Hk]),
                              ("values", caches[0].v, caches[0].v_scale, values, 0 * values)):
        if held == I8:
            S.check_codes(t[page, :, off], s[page, :, off], y, tl, f"{what} {case}")
        else:
            O.check(t[page, :, off], y, O.rounded(y, tl, held), f"{what} {case}")

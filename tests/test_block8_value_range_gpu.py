"""Attention over 8-bit caches whose value scales differ by many powers of two: a key that a token
does not see, or to which it gives next to no weight, takes nothing from the others, whatever its
scale.

The tolerance counts, beside the roundings that `block8_oracle.attention` counts, what the product of a
probability and a value's scale loses in fp16 where it is small: half of 2^-24 of a unit that
is at most twice the row's largest such product, for each key, times its code."""
import math

import pytest
import torch

import block8_oracle as O
from test_block8_gpu import BF16, F16, attention_case, run_case, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    from conv_bn_silu_amd import block8
    return block8


def expect(c):
    """Outputs in 64 bits and their tolerance."""
    codes, scales = c["tensors"][1].double(), c["tensors"][3].double().nan_to_num(0)
    c["kv64"] = (c["kv64"][0], codes * scales[..., None])
    # a share that is not quite fp16's, for which the oracle would allow for the largest value seen
    ref, _, mine = O.attention(c["q"], *c["kv64"], c["table"], c["starts"], c["lens"], c["window"], c["scale"], 0.0)
    assert bool(mine.all())
    _, tol, _ = O.attention(c["q"].double(), *c["kv64"], c["table"], c["starts"], c["lens"], c["window"], c["scale"],
                            O.half_step(F16) * (1 + 2.0 ** -30))
    return ref, O.rounded(ref, tol + small_products(c), c["q"].dtype)


def for_each_row(c, lost):
    """lost(p, pages, head, offsets) for the keys that a token sees, p their probabilities for each head of a group."""
    table, page = c["table"].long(), c["tensors"][0].shape[2]
    k = c["kv64"][0]
    heads, hk = c["q"].shape[1], k.shape[1]
    out = torch.zeros(c["q"].shape, dtype=O.F64)
    for b, n in enumerate(c["lens"]):
        j = torch.arange(n)
        pages, new = table[b][j // page], c["starts"][b + 1] - c["starts"][b]
        for i in range(new):
            pos, at = n - new + i, c["starts"][b] + i
            seen = (j <= pos) & (j > pos - (c["window"] or n))
            for h in range(hk):
                mine = slice(h * heads // hk, (h + 1) * heads // hk)
                z = c["q"][at, mine].double() @ k[pages, h, j % page][seen].t() * c["scale"]
                out[at, mine] = lost(torch.softmax(z, -1), pages[seen], h, (j % page)[seen])[:, None]
    return out


def small_products(c):
    s = c["tensors"][3].double().nan_to_num(0).abs()
    return for_each_row(c, lambda p, pages, h, off: 127 * p.shape[1] * 2.0 ** -24 * (p * s[pages, h, off]).amax(-1))


def check(ops, c, what):
    ref, tol = expect(c)
    say("[value range]", what)
    out = run_case(ops, c).cpu().double()
    most = torch.finfo(c["q"].dtype).max
    # what the type does not hold is infinite
    fits = ((ref - tol <= out) & (out <= ref + tol) & out.isfinite()) | ((out == math.inf) & (ref + tol >= most)) | (
        (out == -math.inf) & (ref - tol <= -most))
    worst = ((out - ref).abs() / tol)[~fits]
    assert bool(fits.all()), f"{what}: {int((~fits).sum())} of {fits.numel()} outside tolerance, worst {float(worst.max()):.3g} times it"


def at_key(c, b, j):
    page = c["tensors"][0].shape[2]
    return int(c["table"][b, j // page]), j % page


CALLS = {
    # new, lens, heads, kv heads, dim: single tokens, a few, one prompt, chunks with room for two waves to a row and without
    "decode": ([1, 1], [200, 70], 8, 2, 64),
    "few": ([4, 2], [40, 30], 8, 2, 128),
    "few256": ([3, 1], [140, 30], 4, 2, 256),
    "prompt": ([4], [4], 4, 1, 128),
    "chunk": ([70, 3], [200, 30], 4, 2, 64),
    "chunk128": ([90, 40], [150, 40], 8, 2, 128),
    "chunk256": ([90], [120], 4, 1, 256),
    "long": ([40], [3000], 4, 1, 96),
}
GAINS = [2.0 ** 10, 2.0 ** 20, 2.0 ** 30, 2.0 ** 100, 2.0 ** -100]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("gain", GAINS, ids=lambda g: f"2^{int(math.log2(g))}")
def test_later_tokens(ops, call, gain, dtype):
    """The last token's values (and the last but four's) are far from the others: those before do not see them."""
    new, lens, heads, hk, dim = CALLS[call]
    c = attention_case(new, lens, heads, hk, dim, 16, dtype, True, seed=51)
    for back in (1, 5):
        if lens[0] > back:
            page, off = at_key(c, 0, lens[0] - back)
            c["tensors"][3][page, :, off] *= gain
    check(ops, c, f"{call} {gain}")


@pytest.mark.parametrize("call", ["decode", "few", "chunk", "chunk128", "long"])
@pytest.mark.parametrize("gain", GAINS, ids=lambda g: f"2^{int(math.log2(g))}")
def test_out_of_the_window(ops, call, gain):
    """Keys that have left the window of all tokens, or of some, have other scales."""
    new, lens, heads, hk, dim = CALLS[call]
    c = attention_case(new, lens, heads, hk, dim, 16, BF16, True, window=20, seed=52)
    for b in range(len(lens)):
        for j in range(max(0, lens[b] - 19)):
            page, off = at_key(c, b, j)
            c["tensors"][3][page, :, off] *= gain
    check(ops, c, f"{call} {gain}")


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("gain", [2.0 ** 15, 2.0 ** 30, 2.0 ** 60], ids=lambda g: f"2^{int(math.log2(g))}")
@pytest.mark.parametrize("first", [True, False], ids=["first", "middle"])
def test_negligible_weight(ops, call, gain, first):
    """A key with a score some 75 below the others', and so a weight of about 2^-108, has large values."""
    new, lens, heads, hk, dim = CALLS[call]
    c = attention_case(new, lens, heads, hk, dim, 16, BF16, True, seed=53)
    c["q"] = c["q"].abs() + 0.5
    j = 0 if first else lens[0] // 2
    page, off = at_key(c, 0, j)
    c["tensors"][0][page, :, off] = -100
    s = 75 / (100 * dim ** 0.5 * float(c["q"].double().mean()))
    c["tensors"][2][page, :, off] = s
    c["kv64"][0][page, :, off] = -100 * c["tensors"][2][page, :, off].double()[..., None]
    c["tensors"][3][page, :, off] *= gain
    check(ops, c, f"{call} {gain}")


@pytest.mark.parametrize("call", CALLS)
def test_scales_of_every_size(ops, call):
    """Scales spread over 2^80, all keys but one in 16 without values, none at all, negative ones."""
    new, lens, heads, hk, dim = CALLS[call]
    c = attention_case(new, lens, heads, hk, dim, 16, BF16, True, seed=54)
    scales = c["tensors"][3]
    g = torch.Generator().manual_seed(54)
    plain = scales.clone()
    scales *= 2.0 ** (80 * torch.rand(scales.shape, generator=g) - 40)
    check(ops, c, f"{call} spread")
    for least in (2.0 ** -126, 0.0):
        scales.copy_(plain)
        hide = (torch.rand(scales.shape, generator=g) > 1 / 16) & ~scales.isnan()
        c["tensors"][1][hide] = 0
        scales[hide] = least
        check(ops, c, f"{call} zeros {least}")
    scales[~scales.isnan()] = 0
    c["tensors"][1][:] = 0
    check(ops, c, f"{call} nothing")
    c = attention_case(new, lens, heads, hk, dim, 16, BF16, True, seed=54)
    c["tensors"][3][:, :, ::3] *= -3
    check(ops, c, f"{call} negative")


@pytest.mark.parametrize("call", CALLS)
def test_small_weights_of_large_values(ops, call):
    """fp16 caches: keys of a weight of 2^-24 to 2^-28 with values of thousands, beside ones of thousandths.

    The largest probability is 2^6 or more in the unit in which they become fp16, which is off by up to 2^-25: for
    each key 2^-31 of the largest probability, times the largest value."""
    new, lens, heads, hk, dim = CALLS[call]
    c = attention_case(new, lens, heads, hk, dim, 16, F16, False, seed=55)
    g = torch.Generator().manual_seed(55)
    c["q"] = torch.ones_like(c["q"])
    k, v = c["tensors"]
    live = ~k[..., :1].isnan()
    far = (torch.rand(live.shape, generator=g) < 0.3) & live
    score = torch.where(far, -17 - 2.5 * torch.rand(live.shape, generator=g), 0.0)
    value = torch.randn(v.shape, generator=g)
    k.copy_(torch.where(live, (score * dim ** -0.5).expand_as(k), math.nan))
    v.copy_(torch.where(live, torch.where(far, 8000 * value.clamp(-4, 4), 1e-3 * value), math.nan))
    c["kv64"] = tuple(torch.where(live, t.double(), 0.0) for t in (k, v))
    ref, _, _ = O.attention(c["q"], *c["kv64"], c["table"], c["starts"], c["lens"], 0, c["scale"], 0.0)
    _, tol, _ = O.attention(c["q"].double(), *c["kv64"], c["table"], c["starts"], c["lens"], 0, c["scale"],
                            O.half_step(F16) * (1 + 2.0 ** -30))
    tol = tol + for_each_row(c, lambda p, pages, h, off: p.shape[1] * 2.0 ** -31 * p.amax(-1) * c["kv64"][1][pages, h, off].abs().amax())
    say("[value range]", call, "small weights")
    O.check(run_case(ops, c), ref, O.rounded(ref, tol, F16), call)

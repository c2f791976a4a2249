"""The measured cases of the 8-bit block operators: the linear layer in 8-bit
integers, the paged cache that quantises what it is given, and the attention
that reads it.

Each case is one call pattern of a served transformer block.  ``run`` computes
it either in elementary torch operations (``own`` false) or through this
package's operators (``own`` true), on the same inputs; ``exact`` computes it
from the definition in 64 bits.

Definitions:

* rows to 8 bits: s = max(amax / 127 rounded to fp32, 2^-126), code =
  round-half-even(x / s);
* linear: y = act(sum_k a[m,k] w[n,k] * sa[m] * sw[n] + bias[n]), with a and sa
  the rows of x in 8 bits;
* cache: [pages, heads, page size, head dim] codes with one scale per token
  and head; a token's slot is page * page size + offset; a slot outside the
  cache is skipped by the write and reads as zeros;
* attention: the new tokens of a sequence are its last ones; each sees the
  keys up to itself (and within the window, if one is set).
"""
import math

import torch

own = False

F32, BF16, F16 = "float32", "bfloat16", "float16"
_TINY = 2.0 ** -126  # the smallest scale


def _linear(name, m, n, k, dtype, bias, silu):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias, "silu": silu}


def _cache(name, tokens, heads, dim, page, dtype, skipped):
    return {"name": name, "op": "cache", "tokens": tokens, "heads": heads, "dim": dim, "page": page, "dtype": dtype,
            "skipped": skipped}


def _attention(name, batch, new_lo, new_hi, old_lo, old_hi, heads, kv_heads, dim, page, dtype, int8, window):
    return {"name": name, "op": "attention", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "old_lo": old_lo,
            "old_hi": old_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype,
            "int8": int8, "window": window}


def listed():
    return [
        # one request's next token through a square projection: latency
        _linear("linear: one token", 1, 4096, 4096, BF16, False, False),
        # the first half of a feed-forward layer for a batch of decoding requests
        _linear("linear: 40 tokens, SiLU", 40, 16384, 4096, BF16, True, True),
        # a classifier-like head with sizes off every tile, fp32 in and out
        _linear("linear: ragged fp32", 333, 1001, 1999, F32, True, False),
        # a long prompt through a wide projection: matrix-bound
        _linear("linear: prompt", 8192, 8192, 8192, BF16, False, False),
        # one decoding step of 64 requests enters the cache and is read back
        _cache("cache: one step", 64, 8, 128, 16, BF16, False),
        # odd head count, head size and page size, padding tokens without a slot
        _cache("cache: ragged", 5001, 5, 80, 24, F16, True),
        # a batch of prompts
        _cache("cache: prompts", 32768, 8, 128, 64, BF16, False),
        # a few short conversations, one new token each: latency
        _attention("attention: short decode", 4, 1, 1, 90, 600, 8, 2, 64, 16, BF16, False, 0),
        # a full batch of long conversations, one new token each, 8-bit cache
        _attention("attention: long decode", 64, 1, 1, 2000, 16000, 32, 8, 128, 16, BF16, True, 0),
        # prompt chunks and decoding requests in one batch
        _attention("attention: mixed chunks", 16, 1, 640, 0, 8000, 32, 8, 128, 16, BF16, False, 0),
        # sliding window, sizes off every tile, 8-bit cache
        _attention("attention: window, ragged", 5, 33, 801, 0, 3000, 15, 3, 80, 24, F16, True, 512),
        # two long prompts from an empty cache: matrix-bound
        _attention("attention: prompts", 2, 8192, 8192, 0, 0, 32, 8, 128, 64, BF16, True, 0),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(("linear", "linear", "cache", "attention", "attention", "attention"))
    dtype = rng.choice((BF16, BF16, F16, F32)) if op != "attention" else rng.choice((BF16, BF16, F16))
    if op == "linear":
        m, n, k = _log_between(rng, 1, 8192), _log_between(rng, 64, 16384), _log_between(rng, 64, 8192)
        if rng.random() < 0.6:
            n, k = (n + 63) // 64 * 64, (k + 63) // 64 * 64
        return _linear("", m, n, k, dtype, rng.random() < 0.5, rng.random() < 0.5)
    dim = rng.choice((64, 80, 96, 128, 128, 256))
    page = rng.choice((16, 16, 32, 64, 24, 17, 128))
    kv_heads = rng.choice((1, 2, 3, 4, 5, 8, 8))
    if op == "cache":
        return _cache("", _log_between(rng, 1, 32768), kv_heads, dim, page, dtype, rng.random() < 0.3)
    heads = kv_heads * rng.choice((1, 2, 4, 4, 5, 8))
    batch = _log_between(rng, 1, 64)
    new_hi = 1 if rng.random() < 0.4 else _log_between(rng, 2, 4096)
    new_lo = 1 if new_hi == 1 or rng.random() < 0.5 else rng.randint(1, new_hi)
    old_hi = _log_between(rng, 1, 16000)
    old_lo = rng.randint(0, old_hi)
    window = _log_between(rng, 64, 4096) if rng.random() < 0.2 else 0
    return _attention("", batch, new_lo, new_hi, old_lo, old_hi, heads, kv_heads, dim, page, dtype,
                      rng.random() < 0.6, window)


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        b, f = top.get(c["op"], (0, 0))
        top[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] > top[c["op"]][0] or w["flops"] > top[c["op"]][1]:
            continue
        if c["op"] == "attention":
            new, old = _lengths(c)
            kv = max(a + b for a, b in zip(new, old))
            # the plain form pads every sequence to the longest
            if c["batch"] * c["heads"] * max(new) * kv > 2 ** 32 or c["batch"] * c["kv_heads"] * c["dim"] * kv > 2 ** 31:
                continue
        del c["name"]
        return c


def _lengths(c):
    """New and earlier tokens of each sequence, spread over the case's ranges."""
    n = c["batch"]
    new = [c["new_lo"] + (c["new_hi"] - c["new_lo"]) * ((5 * i + 2) % n) // max(1, n - 1) for i in range(n)]
    old = [c["old_lo"] + (c["old_hi"] - c["old_lo"]) * ((3 * i + 1) % n) // max(1, n - 1) for i in range(n)]
    return new, old


def _seen(c):
    """(query, key) pairs, and keys that some query sees, over all sequences (per head)."""
    pairs = keys = 0
    for n, o in zip(*_lengths(c)):
        w = c["window"] or n + o
        keys += n + o - max(0, o + 1 - w)
        # query i sees min(o + i + 1, w) keys
        full = min(n, max(0, w - o))  # queries whose window reaches the first key
        pairs += full * (o + 1) + full * (full - 1) // 2 + (n - full) * w
    return pairs, keys


def _element(dtype):
    return 4 if dtype == F32 else 2


def work(case):
    c = case
    if c["op"] == "linear":
        e = _element(c["dtype"])
        return {"bytes": c["m"] * c["k"] * e + c["n"] * c["k"] + c["n"] * (8 if c["bias"] else 4) + c["m"] * c["n"] * e,
                "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["op"] == "cache":
        values = 2 * c["tokens"] * c["heads"] * c["dim"]
        scales = 2 * c["tokens"] * c["heads"] * 4
        # the write reads the values and stores codes; the read does the reverse
        return {"bytes": 2 * (values * (_element(c["dtype"]) + 1) + scales) + 8 * c["tokens"], "flops": 6 * values}
    pairs, keys = _seen(c)
    queries = sum(_lengths(c)[0]) * c["heads"] * c["dim"]
    row = c["dim"] + 4 if c["int8"] else 2 * c["dim"]
    return {"bytes": 2 * 2 * queries + 2 * keys * c["kv_heads"] * row + 4 * (keys // c["page"] + 2 * c["batch"] + 1),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# Inputs


def _quantize64(x):
    """Codes and scale of the rows of x, by the definition, in 64 bits."""
    x = x.double()
    s = (x.abs().amax(-1) / 127).float().clamp_min(_TINY)
    return torch.round(x / s.double()[..., None]).to(torch.int8), s


def prepare(case, seed):
    c, dev = case, torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype = getattr(torch, c["dtype"])

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if c["op"] == "linear":
        # activations with a few large channels, as they come out of a norm;
        # weights quantised once, row by row, as a model loader does
        x = normal(c["m"], c["k"]) * (1 + 5 * (torch.rand(c["k"], generator=g, device=dev) > 0.99))
        w, ws = _quantize_weight(normal(c["n"], c["k"]) / math.sqrt(c["k"]))
        return {"case": c, "x": x.to(dtype), "w": w, "ws": ws, "bias": 0.3 * normal(c["n"]) if c["bias"] else None}
    if c["op"] == "cache":
        t, h, d, p = c["tokens"], c["heads"], c["dim"], c["page"]
        pages = (t + p - 1) // p + 8
        # keys carry a per-channel offset; the tokens' slots are scattered over
        # the cache's pages, page by page as an allocator hands them out
        k = normal(t, h, d) + 2 * normal(h, d)
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        slots = order[at // p] * p + at % p
        if c["skipped"]:
            slots = torch.where(torch.rand(t, generator=g, device=dev) < 0.1, -1, slots)
        cache = _empty_cache(pages, h, p, d, torch.int8)
        return {"case": c, "k": k.to(dtype), "v": normal(t, h, d).to(dtype), "slots": slots.to(torch.int32),
                "cache": cache}
    new, old = _lengths(c)
    p, hk, d = c["page"], c["kv_heads"], c["dim"]
    lens = torch.tensor([a + b for a, b in zip(new, old)], device=dev)
    starts = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    width = (int(max(a + b for a, b in zip(new, old))) + p - 1) // p
    used = (lens + p - 1) // p
    pages = int(sum((a + b + p - 1) // p for a, b in zip(new, old))) + 4
    # each sequence's pages lie anywhere in the cache; the table's unused
    # entries hold -1
    order = torch.randperm(pages, generator=g, device=dev)
    first = used.cumsum(0) - used
    col = torch.arange(width, device=dev)
    table = torch.where(col < used[:, None], order[(first[:, None] + col).clamp_max(pages - 1)], -1).to(torch.int32)
    cache = _empty_cache(pages, hk, p, d, torch.int8 if c["int8"] else dtype)
    for name in ("k", "v"):
        values = normal(pages, hk, p, d)
        if name == "k":
            values += normal(hk, 1, d)
        if c["int8"]:
            scale = (values.abs().amax(-1) / 127).clamp_min(_TINY)
            cache[name].copy_(torch.round(values / scale[..., None]))
            cache[name + "_scale"].copy_(scale)
        else:
            cache[name].copy_(values)
        del values
    # what lies past a sequence's end in its last page was never written
    tail = (torch.arange(p, device=dev) >= ((lens - 1) % p + 1)[:, None]).nonzero()
    last = table.gather(1, (used - 1)[:, None].long())[:, 0].long()
    for name in ("k_scale", "v_scale") if c["int8"] else ("k", "v"):
        cache[name][last[tail[:, 0]], :, tail[:, 1]] = math.nan
    q = normal(sum(new), c["heads"], d).to(dtype)
    return {"case": c, "q": q, "cache": cache, "table": table, "starts": starts, "lens": lens.to(torch.int32),
            "longest": max(a + b for a, b in zip(new, old)), "most_new": max(new)}


def _quantize_weight(w):
    s = (w.abs().amax(-1) / 127).clamp_min(_TINY)
    return torch.round(w / s[:, None]).to(torch.int8), s


def _empty_cache(pages, heads, page, dim, dtype):
    dev = torch.device("cuda", 0)
    cache = {n: torch.zeros(pages, heads, page, dim, dtype=dtype, device=dev) for n in ("k", "v")}
    for n in ("k_scale", "v_scale"):
        cache[n] = torch.zeros(pages, heads, page, device=dev) if dtype == torch.int8 else None
    return cache


# One pass


def run(state):
    return {"linear": _run_linear, "cache": _run_cache, "attention": _run_attention}[state["case"]["op"]](state)


def _run_linear(s):
    if own:
        from conv_bn_silu_amd import int8_linear
        return int8_linear(s["x"], s["w"], s["ws"], bias=s["bias"], activation="silu" if s["case"]["silu"] else None)
    codes, scale = _plain_quantize(s["x"])
    # sums of up to 16129 * K: fp32 products, summed by the library in fp32
    y = (codes @ s["w"].float().t()) * scale[:, None] * s["ws"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["case"]["silu"]:
        y = y / (1 + torch.exp(-y))
    return y.to(s["x"].dtype)


def _plain_quantize(x):
    """Rows of x to 8 bits; the quotient in 64 bits, so that values next to a
    border between two codes fall on the right side."""
    x = x.float()
    scale = (x.abs().amax(-1) / 127).clamp_min(_TINY)
    return torch.round(x.double() / scale.double()[..., None]).float(), scale


def _run_cache(s):
    c, cache, slots = s["case"], s["cache"], s["slots"]
    if own:
        from conv_bn_silu_amd import PagedCache, cache_read, cache_write
        paged = PagedCache(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"])
        cache_write(paged, s["k"], s["v"], slots)
        return cache_read(paged, slots, dtype=s["k"].dtype)
    there = slots >= 0
    at = slots[there].long() if c["skipped"] else slots.long()
    page, off = at // c["page"], at % c["page"]
    out = []
    for name in ("k", "v"):
        codes, scale = _plain_quantize(s[name][there] if c["skipped"] else s[name])
        cache[name][page, :, off] = codes.to(torch.int8)
        cache[name + "_scale"][page, :, off] = scale
        values = cache[name][page, :, off].float() * cache[name + "_scale"][page, :, off][..., None]
        if c["skipped"]:
            back = torch.zeros_like(s[name])
            back[there] = values.to(back.dtype)
        else:
            back = values.to(s[name].dtype)
        out.append(back)
    return tuple(out)


def _run_attention(s):
    c = s["case"]
    if own:
        from conv_bn_silu_amd import PagedCache, paged_attention
        cache = s["cache"]
        paged = PagedCache(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"])
        return paged_attention(s["q"], paged, s["table"], s["starts"], s["lens"], window=c["window"])
    p, hk, dim, group = c["page"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    table, lens, starts = s["table"], s["lens"].long(), s["starts"].long()
    batch = lens.numel()
    new = starts[1:] - starts[:-1]
    # keys and values of every sequence, padded to the longest
    j = torch.arange(s["longest"], device=lens.device)
    live = j < lens[:, None]
    page = table[:, j // p].clamp_min(0).long()
    kv = []
    for name in ("k", "v"):
        x = s["cache"][name][page, :, j % p].float()
        if c["int8"]:
            x = x * s["cache"][name + "_scale"][page, :, j % p][..., None]
        kv.append(torch.where(live[..., None, None], x, 0.0).permute(0, 2, 1, 3).contiguous())
        del x
    # queries, padded to the most new tokens
    i = torch.arange(s["most_new"], device=lens.device)
    token = (starts[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][token].float().view(batch, i.numel(), hk, group, dim).permute(0, 2, 3, 1, 4)
    q = q.reshape(batch, hk, group * i.numel(), dim)
    scores = torch.matmul(q, kv[0].transpose(-1, -2).contiguous()).view(batch, hk, group, i.numel(), -1)
    pos = (lens - new)[:, None] + i
    seen = live[:, None, :] & (j <= pos[..., None])
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    scores.mul_(dim ** -0.5).masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    probs = scores.sub_(top).exp_()
    total = probs.sum(-1, keepdim=True)
    out = torch.matmul(probs.view(batch, hk, group * i.numel(), -1), kv[1]).view(batch, hk, group, i.numel(), dim)
    out = torch.where(total > 0, out / total, 0.0)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, i.numel(), c["heads"], dim)
    return out[i < new[:, None]].to(s["q"].dtype)


# The definition, in 64 bits


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "linear":
        codes, scale = _quantize64(s["x"])
        y = torch.mm(codes.double(), s["w"].double().t().contiguous())
        y = y * (scale.double()[:, None] * s["ws"].double()[None, :])
        if s["bias"] is not None:
            y = y + s["bias"].double()
        return y * torch.sigmoid(y) if c["silu"] else y
    if c["op"] == "cache":
        out = []
        for name in ("k", "v"):
            codes, scale = _quantize64(s[name])
            back = codes.double() * scale.double()[..., None]
            back[s["slots"] < 0] = 0
            out.append(back)
        return tuple(out)
    p, group = c["page"], c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (n, old) in enumerate(zip(*_lengths(c))):
        total = n + old
        j = torch.arange(total, device=out.device)
        pages = s["table"][b].long()[j // p]
        pos = torch.arange(old, total, device=out.device)[:, None]
        hidden = j[None, :] > pos
        if c["window"]:
            hidden |= j[None, :] + c["window"] <= pos
        for h in range(c["kv_heads"]):
            k, v = (s["cache"][x][pages, h, j % p].double() for x in ("k", "v"))
            if c["int8"]:
                k = k * s["cache"]["k_scale"][pages, h, j % p].double()[:, None]
                v = v * s["cache"]["v_scale"][pages, h, j % p].double()[:, None]
            for head in range(h * group, (h + 1) * group):
                z = torch.mm(s["q"][at:at + n, head].double(), k.t().contiguous()) / math.sqrt(c["dim"])
                z.masked_fill_(hidden, -math.inf)
                out[at:at + n, head] = torch.mm(torch.softmax(z, -1), v)
        at += n
    return out

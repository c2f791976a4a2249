"""The measured cases of what a served block's step does between its layers, its
cache and its attention: the residual's addition with the root-mean-square norm
(whose output can be rows in 8 bits, for the linear layer), rotary positions (of
a tensor, or of queries and keys on their way into the paged cache), and the
pages of the cache, handed out and taken back by the sequences' lengths.

Each case is one call pattern of such a step.  ``run`` computes it either in
elementary torch operations (``own`` false) or through this package's operators
(``own`` true), on the same inputs; ``exact`` computes it from the definition in
64 bits.

Definitions:

* norm: h = x + residual, rounded to the residual's type; y = h w / sqrt(mean(h^2)
  + eps), rounded to x's type, or to 8 bits as the linear layer does with its rows
  (s = max(amax / 127 rounded to fp32, 2^-126), code = round-half-even(y / s));
* rotary: the pair (a, b) of a head becomes m (a cos t - b sin t, b cos t + a sin t)
  with t = position * frequency; pair i is (i, i + n) or (2i, 2i + 1), i below the
  number n of frequencies; what lies past the first 2n dims stays;
* pages: sequences grow in order, each by pages from the top of the pool's stack,
  as long as there are enough; one that would pass its row of the table, or whose
  tokens pass the batch, stays as it is.  Pages come back so that what is taken and
  given back leaves the stack as it was.
"""
import math

import torch

own = False

F32, BF16, F16 = "float32", "bfloat16", "float16"
_TINY = 2.0 ** -126  # the smallest scale
_EPS = 1e-6


def _norm(name, m, k, n, dtype, residual, weight):
    """n: outputs of the 8-bit layer that follows; 0 for the norm alone.  residual: its type, or ""."""
    return {"name": name, "op": "norm", "m": m, "k": k, "n": n, "dtype": dtype, "residual": residual, "weight": weight}


def _rotary(name, tokens, heads, kv_heads, dim, turned, interleaved, dtype, held, page, far, skipped, magnitude):
    """turned: dims that are rotated.  held: the cache's type, or "" for a tensor by itself, which has
    heads + kv_heads heads and lies in a wider one."""
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "turned": turned, "interleaved": interleaved, "dtype": dtype, "held": held, "page": page, "far": far,
            "skipped": skipped, "magnitude": magnitude}


def _pages(name, batch, new_lo, new_hi, old_lo, old_hi, page, padding, short):
    """padding: rows of the batch behind the last sequence.  short: the pool has pages for most sequences only."""
    return {"name": name, "op": "pages", "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "old_lo": old_lo,
            "old_hi": old_hi, "page": page, "padding": padding, "short": short}


def listed():
    return [
        # one request's next token before a projection: latency
        _norm("norm: one token", 1, 4096, 0, BF16, BF16, BF16),
        # a batch of decoding requests through the norm and the first half of a feed-forward layer
        _norm("norm: 40 tokens, into a layer", 40, 4096, 16384, BF16, BF16, BF16),
        # a model kept in fp32, sizes off every tile, no residual (the first norm)
        _norm("norm: ragged fp32", 333, 1999, 0, F32, "", F32),
        # a batch of prompts, residual stream in 16 bits: HBM
        _norm("norm: prompts", 16384, 8192, 0, BF16, BF16, BF16),
        # a prompt into the projection of shared keys, residual stream in fp32
        _norm("norm: prompt, into a layer", 8192, 8192, 1024, BF16, F32, F32),
        # one decoding step of 64 requests
        _rotary("rotary: one step", 64, 32, 8, 128, 128, False, BF16, "int8", 16, 16000, False, 1.0),
        # odd head counts and sizes, part of the head, neighbouring pairs, padding tokens without a slot
        _rotary("rotary: ragged", 5001, 15, 5, 80, 32, True, F16, F16, 24, 3000, True, 1.0),
        # a prompt's queries and keys as they lie in the projection's output, for an attention without cache
        _rotary("rotary: without a cache", 8192, 32, 8, 128, 64, False, BF16, "", 0, 8192, False, 1.0),
        # a batch of prompts far into long contexts, scaled
        _rotary("rotary: prompts", 32768, 32, 8, 128, 128, False, BF16, "int8", 64, 131072, False, 1.2),
        # one decoding step of 64 requests: latency
        _pages("pages: one step", 64, 1, 1, 90, 16000, 16, 0, False),
        # prompt chunks, decoding requests and idle ones in a padded batch
        _pages("pages: ragged", 300, 0, 700, 0, 5000, 24, 1000, False),
        # prompts enter an empty cache
        _pages("pages: prompts", 1024, 100, 4000, 0, 0, 16, 0, False),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(("norm", "rotary", "rotary", "pages"))
    dtype = rng.choice((BF16, BF16, F16, F32))
    if op == "norm":
        m, k = _log_between(rng, 1, 16384), _log_between(rng, 64, 16384)
        if rng.random() < 0.6:
            k = (k + 63) // 64 * 64
        n = _log_between(rng, 64, 16384) if rng.random() < 0.4 else 0
        return _norm("", m, k, n, dtype, rng.choice(("", dtype, dtype, F32)), rng.choice((dtype, F32)))
    if op == "rotary":
        held = rng.choice(("", "int8", "int8", dtype))
        dim = rng.choice((64, 80, 96, 128, 128, 256) if held else (64, 72, 80, 100, 128, 128, 256))
        turned = dim if rng.random() < 0.6 else rng.choice((dim // 2, dim // 4 * 2, 20, 32, 64))
        kv_heads = rng.choice((1, 2, 3, 4, 5, 8, 8))
        heads = kv_heads * rng.choice((1, 2, 4, 4, 5, 8))
        return _rotary("", _log_between(rng, 1, 32768), heads, kv_heads, dim, turned, rng.random() < 0.4, dtype, held,
                       rng.choice((16, 16, 32, 64, 24, 17, 128)) if held else 0, _log_between(rng, 100, 1 << 20),
                       rng.random() < 0.3 and held != "", rng.choice((1.0, 1.0, 1.2)))
    batch = _log_between(rng, 1, 2048)
    new_hi = 1 if rng.random() < 0.4 else _log_between(rng, 2, 4096)
    new_lo = 1 if new_hi == 1 or rng.random() < 0.5 else rng.randint(0, new_hi)
    old_hi = _log_between(rng, 1, 16000)
    return _pages("", batch, new_lo, new_hi, rng.randint(0, old_hi), old_hi, rng.choice((16, 16, 32, 64, 24, 17, 128)),
                  rng.choice((0, 0, 100, 1000)), rng.random() < 0.2)


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
        # the plain form looks at every entry of the table
        if c["op"] == "pages" and c["batch"] * _width(c) > 2 ** 22:
            continue
        del c["name"]
        return c


def _lengths(c):
    """New and earlier tokens of each sequence, spread over the case's ranges."""
    n = c["batch"]
    new = [c["new_lo"] + (c["new_hi"] - c["new_lo"]) * ((5 * i + 2) % n) // max(1, n - 1) for i in range(n)]
    old = [c["old_lo"] + (c["old_hi"] - c["old_lo"]) * ((3 * i + 1) % n) // max(1, n - 1) for i in range(n)]
    return new, old


def _width(c):
    new, old = _lengths(c)
    return (max(a + b for a, b in zip(new, old)) + c["page"] - 1) // c["page"]


def _taken(c):
    """Pages that the sequences have, and that they take for their new tokens."""
    p = c["page"]
    new, old = _lengths(c)
    had = sum((b + p - 1) // p for b in old)
    return had, sum((a + b + p - 1) // p for a, b in zip(new, old)) - had


def _element(dtype):
    return 4 if dtype == F32 else 2


def work(case):
    c = case
    if c["op"] == "norm":
        values, e = c["m"] * c["k"], _element(c["dtype"])
        moved = values * (e + (2 * _element(c["residual"]) if c["residual"] else 0)) + c["k"] * _element(c["weight"])
        if not c["n"]:
            return {"bytes": moved + values * e, "flops": 6 * values}
        return {"bytes": moved + c["n"] * (c["k"] + 4) + c["m"] * c["n"] * e, "flops": 2 * values * c["n"]}
    if c["op"] == "rotary":
        e = _element(c["dtype"])
        q, kv = (c["tokens"] * h * c["dim"] for h in (c["heads"], c["kv_heads"]))
        turned = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["turned"]
        if not c["held"]:
            return {"bytes": 2 * (q + kv) * e + 4 * c["tokens"], "flops": 3 * turned}
        moved = 2 * q * e + 2 * kv * e + 8 * c["tokens"]
        if c["held"] == "int8":  # and what was written is read back
            scales = 2 * c["tokens"] * c["kv_heads"] * 4
            moved += 2 * (2 * kv + scales) + 2 * kv * 2 + 4 * c["tokens"]
        else:
            moved += 2 * kv * _element(c["held"])
        return {"bytes": moved, "flops": 3 * turned + 6 * kv}
    tokens, taken = sum(_lengths(c)[0]) + c["padding"], _taken(c)[1]
    # slots and positions; each page taken from the stack into the table, and back; the sequences' numbers
    return {"bytes": 8 * tokens + 20 * taken + 28 * c["batch"], "flops": 8 * tokens}


# Inputs


def _frequencies(n, dev):
    """Of each pair, in radians per position."""
    return 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)


def prepare(case, seed):
    c, dev = case, torch.device("cuda", 0)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    if c["op"] == "norm":
        # a residual stream with a few large channels, and a block's output to add to it
        dtype, k = getattr(torch, c["dtype"]), c["k"]
        large = 1 + 8 * (torch.rand(k, generator=g, device=dev) > 0.99)
        s = {"case": c, "x": normal(c["m"], k), "residual": None,
             "weight": (1 + 0.2 * normal(k)).to(getattr(torch, c["weight"]))}
        if c["residual"]:
            s["residual"] = (2 * normal(c["m"], k) * large).to(getattr(torch, c["residual"]))
        else:
            s["x"] *= large
        s["x"] = s["x"].to(dtype)
        if c["n"]:
            # weights quantised once, row by row, as a model loader does
            w = normal(c["n"], k) / math.sqrt(k)
            s["ws"] = (w.abs().amax(-1) / 127).clamp_min(_TINY)
            s["w"] = torch.round(w / s["ws"][:, None]).to(torch.int8)
        return s
    if c["op"] == "rotary":
        t, h, hk, d, p = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        dtype = getattr(torch, c["dtype"])
        positions = torch.randint(0, c["far"], (t,), generator=g, device=dev)
        # queries, keys and values are parts of one projection's output; keys carry a per-channel offset
        fused = normal(t, h + 2 * hk, d)
        fused[:, h:h + hk] += 2 * normal(hk, d)
        fused = fused.to(dtype)
        s = {"case": c, "q": fused[:, :h], "k": fused[:, h:h + hk], "v": fused[:, h + hk:], "both": fused[:, :h + hk],
             "positions": positions.to(torch.int32), "frequencies": _frequencies(c["turned"] // 2, dev)}
        if c["held"]:
            pages = (t + p - 1) // p + 8
            order = torch.randperm(pages, generator=g, device=dev)
            at = torch.arange(t, device=dev)
            slots = order[at // p] * p + at % p
            if c["skipped"]:
                slots = torch.where(torch.rand(t, generator=g, device=dev) < 0.1, -1, slots)
            s["slots"] = slots.to(torch.int32)
            held = getattr(torch, c["held"])
            for name in ("ck", "cv"):
                s[name] = torch.zeros(pages, hk, p, d, dtype=held, device=dev)
                s[name + "_scale"] = torch.zeros(pages, hk, p, device=dev) if c["held"] == "int8" else None
        return s
    # the sequences' pages lie anywhere in the cache; the table's unused entries hold -1
    new, old = _lengths(c)
    p, width = c["page"], _width(c)
    had, takes = _taken(c)
    pages = had + (takes * 7 // 8 if c["short"] else takes + 50)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    lens = torch.tensor(old, device=dev)
    used = (lens + p - 1) // p
    first, col = used.cumsum(0) - used, torch.arange(width, device=dev)
    table = torch.where(col < used[:, None], order[(first[:, None] + col).clamp_max(pages - 1)], -1)
    free = torch.zeros(pages, dtype=torch.int32, device=dev)
    free[:pages - had] = order[had:]
    counts = torch.tensor([pages - had, 0, 0], dtype=torch.int32, device=dev)
    lens = lens.to(torch.int32)
    # the new tokens turn out to be drafts that are all rejected: each sequence keeps what it had
    return {"case": c, "free": free, "counts": counts, "table": table.to(torch.int32), "lens": lens, "keep": lens.clone(),
            "new": torch.tensor(new, dtype=torch.int32, device=dev), "tokens": sum(new) + c["padding"]}


# One pass


def run(state):
    return {"norm": _run_norm, "rotary": _run_rotary, "pages": _run_pages}[state["case"]["op"]](state)


def _plain_quantize(x):
    """Rows of x to 8 bits; the quotient in 64 bits, so that values next to a
    border between two codes fall on the right side."""
    scale = (x.abs().amax(-1) / 127).clamp_min(_TINY)
    return torch.round(x.double() / scale.double()[..., None]).float(), scale


def _run_norm(s):
    c = s["case"]
    if own:
        from conv_bn_silu_amd import add_rms_norm, int8_linear
        y = add_rms_norm(s["x"], s["weight"], s["residual"], eps=_EPS, int8=bool(c["n"]))
        y, h = y if c["residual"] else (y, None)
        return (int8_linear(y, s["w"], s["ws"]) if c["n"] else y), h
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    y = h.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * s["weight"].float()
    if c["n"]:
        codes, scale = _plain_quantize(y)
        y = (codes @ s["w"].float().t()) * scale[:, None] * s["ws"]
    return y.to(s["x"].dtype), None if s["residual"] is None else h


def _plain_rotate(x, s):
    """x in fp32; the angles in 64 bits, where fp32 loses those of far positions."""
    c, n = s["case"], s["frequencies"].numel()
    angle = (s["positions"].double()[:, None] * s["frequencies"])[:, None]
    cos, sin = (c["magnitude"] * torch.cos(angle)).float(), (c["magnitude"] * torch.sin(angle)).float()
    y = x.float()
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if c["interleaved"] else (y[..., :n], y[..., n:2 * n])
    pair = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(pair, -1).flatten(-2) if c["interleaved"] else torch.cat(pair, -1)
    return torch.cat((turned, y[..., 2 * n:]), -1)


def _read_type(c):
    """In which the codes' values are read back: the attention's."""
    return torch.bfloat16 if c["dtype"] == F32 else getattr(torch, c["dtype"])


def _run_rotary(s):
    c = s["case"]
    if own:
        from conv_bn_silu_amd import PagedCache, cache_read, rotary, rotary_cache_write
        how = {"interleaved": c["interleaved"], "magnitude": c["magnitude"]}
        if not c["held"]:
            return rotary(s["both"], s["positions"], s["frequencies"], **how)
        cache = PagedCache(s["ck"], s["cv"], s["ck_scale"], s["cv_scale"])
        q = rotary_cache_write(cache, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["frequencies"], **how)
        if c["held"] == "int8":
            return (q, *cache_read(cache, s["slots"], dtype=_read_type(c)))
        return q, s["ck"], s["cv"]
    if not c["held"]:
        return _plain_rotate(s["both"], s).to(s["both"].dtype)
    q = _plain_rotate(s["q"], s).to(s["q"].dtype)
    there = s["slots"] >= 0
    at = s["slots"][there].long() if c["skipped"] else s["slots"].long()
    page, off = at // c["page"], at % c["page"]
    out = [q]
    for name, x in (("ck", _plain_rotate(s["k"], s)), ("cv", s["v"].float())):
        x = x[there] if c["skipped"] else x
        if c["held"] != "int8":
            s[name][page, :, off] = x.to(s[name].dtype)
            out.append(s[name])
            continue
        codes, scale = _plain_quantize(x)
        s[name][page, :, off] = codes.to(torch.int8)
        s[name + "_scale"][page, :, off] = scale
        values = s[name][page, :, off].float() * s[name + "_scale"][page, :, off][..., None]
        if c["skipped"]:
            back = torch.zeros(s["k"].shape, dtype=_read_type(c), device=values.device)
            back[there] = values.to(back.dtype)
        else:
            back = values.to(_read_type(c))
        out.append(back)
    return tuple(out)


def _run_pages(s):
    c = s["case"]
    if own:
        from conv_bn_silu_amd import PagePool, grow_pages, release_pages
        pool = PagePool(s["free"], s["counts"], c["page"])
        starts, slots, positions = grow_pages(pool, s["table"], s["lens"], s["new"], s["tokens"])
        release_pages(pool, s["table"], s["lens"], s["keep"])
    else:
        starts, slots, positions = _plain_grow(s)
        _plain_release(s)
    return {"starts": starts, "slots": slots, "positions": positions, "table": s["table"], "lens": s["lens"],
            "free": s["free"], "counts": s["counts"]}


def _plain_grow(s):
    p, table, free, counts = s["case"]["page"], s["table"], s["free"], s["counts"]
    batch, width = table.shape
    n, l = s["new"].clamp_min(0).long(), s["lens"].clamp_min(0).long()
    end = n.cumsum(0)
    start = end - n
    old, want = (l + p - 1) // p, (l + n + p - 1) // p
    fits = (want <= width) & (end <= s["tokens"])
    need = torch.where(fits, want - old, 0)
    cum = need.cumsum(0)
    grows = fits & (cum <= counts[0])
    top = counts[0].long() - 1 - (cum - need)  # of the stack, for each sequence
    starts = torch.cat((start[:1], end)).clamp_max(s["tokens"])
    # the tokens' sequences: how many end at a token or before it
    t = torch.arange(s["tokens"], device=table.device)
    b = torch.zeros(s["tokens"] + 1, dtype=torch.long, device=table.device).index_add_(0, starts[1:], torch.ones_like(end))
    b = b.cumsum(0)[:-1]
    there = b < batch
    b = b.clamp_max(batch - 1)
    there = there & grows[b]
    pos = torch.where(there, l[b] + t - start[b], 0)
    i = pos // p
    fresh = i - old[b]
    page = torch.where(fresh >= 0, free[(top[b] - fresh).clamp(0, free.numel() - 1)], table[b, i.clamp_max(width - 1)])
    slots = torch.where(there & (page >= 0) & (page < free.numel()), page * p + pos % p, -1)
    # the state
    col = torch.arange(width, device=table.device)
    fresh = col - old[:, None]
    taken = grows[:, None] & (fresh >= 0) & (col < want[:, None])
    table.copy_(torch.where(taken, free[(top[:, None] - fresh).clamp(0, free.numel() - 1)], table))
    s["lens"].copy_(torch.where(grows & (n > 0), l + n, s["lens"]))
    counts.copy_(torch.stack((counts[0] - torch.where(grows, need, 0).sum(), (cum[-1] - counts[0]).clamp_min(0),
                              ((n > 0) & ~grows).sum())))
    return starts.to(torch.int32), slots.to(torch.int32), pos.to(torch.int32)


def _plain_release(s):
    p, table, free, counts = s["case"]["page"], s["table"], s["free"], s["counts"]
    l = s["lens"].clamp_min(0)
    kept = torch.minimum(l, s["keep"].clamp_min(0))
    col = torch.arange(table.shape[1], device=table.device)
    given = (col >= ((kept + p - 1) // p)[:, None]) & (col < ((l + p - 1) // p)[:, None])
    good = (given & (table >= 0) & (table < free.numel())).flatten()
    rank = good.long().cumsum(0)
    back = counts[0] + rank[-1]
    to = torch.where(good & (back - rank < free.numel()), back - rank, free.numel())
    free.copy_(torch.cat((free, free[:1])).scatter(0, to, table.flatten())[:-1])
    table.copy_(torch.where(given, -1, table))
    s["lens"].copy_(torch.where(kept < l, kept, s["lens"]))
    counts[0] = back.clamp_max(free.numel())


# The definition, in 64 bits


def _codes64(y):
    """Codes and scales of the rows of y."""
    scale = (y.abs().amax(-1) / 127).float().clamp_min(_TINY).double()
    return torch.round(y / scale[..., None]), scale


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "pages": _exact_pages}[case["op"]](case, s)


def _exact_norm(c, s):
    h = s["x"].double()
    if c["residual"]:
        # the sum of two such numbers is exact in 64 bits, but for far apart ones, which round alike
        h = (h + s["residual"].double()).to(s["residual"].dtype).double()
    length = torch.linalg.vector_norm(h, dim=-1, keepdim=True)
    y = h * s["weight"].double() / torch.sqrt(length.square() / c["k"] + _EPS)
    if c["n"]:
        codes, scale = _codes64(y)
        y = torch.mm(codes, s["w"].double().t().contiguous()) * (scale[:, None] * s["ws"].double()[None, :])
    return y, h if c["residual"] else None


def _rotate64(x, positions, frequencies, interleaved, magnitude):
    """Pairs as complex numbers."""
    n = frequencies.numel()
    y = x.double().clone()
    by = torch.polar(torch.full_like(frequencies, magnitude).expand(x.shape[0], n),
                     positions.double()[:, None] * frequencies[None, :])[:, None, :]
    if interleaved:
        z = torch.complex(y[..., 0:2 * n:2], y[..., 1:2 * n:2]) * by
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :n], y[..., n:2 * n]) * by
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def _exact_rotary(c, s):
    how = s["positions"], s["frequencies"], c["interleaved"], c["magnitude"]
    if not c["held"]:
        return _rotate64(s["both"], *how)
    out = [_rotate64(s["q"], *how)]
    nowhere = s["slots"] < 0
    for x in (_rotate64(s["k"], *how), s["v"].double()):
        if c["held"] == "int8":
            codes, scale = _codes64(x)
            x = codes * scale[..., None]
            x[nowhere] = 0
            out.append(x)
            continue
        held = torch.zeros(s["ck"].shape, dtype=torch.float64, device=x.device).transpose(1, 2)
        at = s["slots"][~nowhere].long()
        held[at // c["page"], at % c["page"]] = x[~nowhere]
        out.append(held.transpose(1, 2).contiguous())
    return tuple(out)


def _exact_pages(c, s):
    """Sequence by sequence, with a list for a stack."""
    p, tokens = c["page"], s["tokens"]
    count = int(s["counts"][0])
    below = s["free"].tolist()
    stack = below[:count]
    rows, lens, news, keeps = (s[n].tolist() for n in ("table", "lens", "new", "keep"))
    starts, slots, positions = [0], [-1] * tokens, [0] * tokens
    lacking, left, at = 0, 0, 0
    for b, n in enumerate(news):
        first, at = at, at + n
        starts.append(min(at, tokens))
        if not n:
            continue
        had, want = -(-lens[b] // p), -(-(lens[b] + n) // p)
        if want > len(rows[b]) or at > tokens:
            left += 1
            continue
        if lacking or want - had > len(stack):
            lacking += want - had - (0 if lacking else len(stack))
            left += 1
            continue
        for i in range(had, want):
            rows[b][i] = stack.pop()
        for j in range(n):
            pos = lens[b] + j
            slots[first + j], positions[first + j] = rows[b][pos // p] * p + pos % p, pos
        lens[b] += n
    back = []
    for b, keep in enumerate(keeps):
        to = min(lens[b], keep)
        for i in range(-(-to // p), -(-lens[b] // p)):
            back.append(rows[b][i])
            rows[b][i] = -1
        lens[b] = to
    stack += back[::-1]
    new = lambda x: torch.tensor(x, dtype=torch.int32, device=s["free"].device)  # noqa: E731
    return {"starts": new(starts), "slots": new(slots), "positions": new(positions), "table": new(rows), "lens": new(lens),
            "free": new(stack + below[len(stack):]), "counts": new([len(stack), lacking, left])}

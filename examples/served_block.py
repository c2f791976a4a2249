"""A transformer block served in 8 bits: its projections as int8 linear layers,
its keys and values in a quantising paged cache, attention over that cache, and
what lies between: norms whose outputs are rows in 8 bits, rotary positions on the
way into the cache, pages handed out on the device.

Prompts of several lengths enter in chunks, then every sequence grows token by
token, as a server's scheduler would have it: each step is one batch that mixes
whatever the sequences bring.  The block's outputs are compared with the same
block computed in float32 from the dequantised weights (no cache, no 8 bits), and
the steps are timed.  A step reads nothing back to the host.

    python examples/served_block.py [--width 1024] [--heads 8] [--kv-heads 2]
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from conv_bn_silu_amd import (PagedCache, PagePool, add_rms_norm, grow_pages, int8_linear, paged_attention,  # noqa: E402
                              release_pages, rotary_cache_write, rotary_frequencies)


def quantize_weight(w):
    """Rows of a weight to codes and scales, once, as a loader does."""
    scale = (w.abs().amax(-1) / 127).clamp_min(2.0 ** -126)
    return torch.round(w / scale[:, None]).to(torch.int8), scale


class Block:
    """x + out(attention(qkv(norm x))), queries and keys turned by their positions, then that + down(silu(up(norm of it)))."""

    def __init__(self, width, heads, kv_heads, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, width // heads

        def weight(n, k):
            return quantize_weight(torch.randn(n, k, generator=g, device=device) / math.sqrt(k))

        def gain():
            return (1 + 0.1 * torch.randn(width, generator=g, device=device)).to(torch.bfloat16)

        self.norms = gain(), gain()
        self.frequencies = rotary_frequencies(self.dim, device=device)
        self.qkv = weight((heads + 2 * kv_heads) * self.dim, width)
        self.out = weight(width, heads * self.dim)
        self.up = weight(4 * width, width)
        self.up_bias = 0.1 * torch.randn(4 * width, generator=g, device=device)
        self.down = weight(width, 4 * width)

    def split(self, qkv):
        h, kv, d = self.heads, self.kv_heads, self.dim
        return (qkv[:, :h * d].view(-1, h, d), qkv[:, h * d:(h + kv) * d].view(-1, kv, d),
                qkv[:, (h + kv) * d:].view(-1, kv, d))

    def step(self, x, cache, table, lens, starts, slots, positions):
        """One batch of new tokens, whose places ``grow_pages`` has given."""
        q, k, v = self.split(int8_linear(add_rms_norm(x, self.norms[0], int8=True), *self.qkv))
        rotary_cache_write(cache, q, k, v, positions, slots, self.frequencies, out=q)
        a = paged_attention(q, cache, table, starts, lens)
        rows, x = add_rms_norm(int8_linear(a.view(x.shape[0], -1), *self.out), self.norms[1], x, int8=True)
        return x + int8_linear(int8_linear(rows, *self.up, bias=self.up_bias, activation="silu"), *self.down)

    def plain(self, x):
        """One whole sequence in float32, without cache or 8-bit activations."""
        w = {n: c.float() * s[:, None] for n, (c, s) in
             {"qkv": self.qkv, "out": self.out, "up": self.up, "down": self.down}.items()}
        x = x.float()

        def norm(x, i):
            return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * self.norms[i].float()

        angle = torch.arange(x.shape[0], device=x.device).double()[:, None] * self.frequencies
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def turned(x):
            a, b = x.chunk(2, -1)
            return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

        q, k, v = self.split(norm(x, 0) @ w["qkv"].t())
        q, k = turned(q), turned(k)
        group, n = self.heads // self.kv_heads, x.shape[0]
        hidden = torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1)
        a = []
        for h in range(self.heads):
            z = (q[:, h] @ k[:, h // group].t().contiguous()) / math.sqrt(self.dim)
            a.append(torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[:, h // group])
        x = x + torch.cat(a, -1) @ w["out"].t()
        up = norm(x, 1) @ w["up"].t() + self.up_bias
        return x + (up * torch.sigmoid(up)) @ w["down"].t()


class Pages:
    """Which pages each sequence has and how long it is, on the device."""

    def __init__(self, batch, pages, page_size, width, device="cuda"):
        self.pool = PagePool.full(pages, page_size, device)
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)

    def grow(self, new):
        """Room for new[b] tokens of each sequence; the step's starts, slots and positions."""
        more = torch.tensor(new, dtype=torch.int32).to(self.lens.device)
        return grow_pages(self.pool, self.table, self.lens, more, sum(new))

    def end(self):
        """All sequences have ended."""
        release_pages(self.pool, self.table, self.lens, torch.zeros_like(self.lens))


def serve(block, prompts, chunk, decode, page_size=16):
    """The prompts' sequences through the block, `chunk` tokens at most of each at a
    time and `decode` more one by one (their inputs are given too); outputs of
    each, and the seconds of each step."""
    batch, width = len(prompts), prompts[0].shape[1]
    longest = max(p.shape[0] for p in prompts)
    per = (longest + page_size - 1) // page_size
    pages = Pages(batch, batch * per, page_size, per)
    cache = PagedCache.empty(batch * per, block.kv_heads, page_size, block.dim)
    outputs, times, old = [[] for _ in prompts], [], [0] * batch
    while any(n < p.shape[0] for n, p in zip(old, prompts)):
        new = []
        for n, p in zip(old, prompts):
            left = p.shape[0] - n
            new.append(min(chunk, left - decode) if left > decode else min(1, left))
        x = torch.cat([p[n:n + m] for p, n, m in zip(prompts, old, new)])
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = block.step(x, cache, pages.table, pages.lens, *pages.grow(new))
        torch.cuda.synchronize()
        times.append(time.perf_counter() - t)
        old = [n + m for n, m in zip(old, new)]
        for o, part in zip(outputs, y.split(new)):
            o.append(part)
    assert all(y.shape[1] == width for o in outputs for y in o)
    assert pages.pool.report()[1:] == (0, 0) and pages.lens.tolist() == old
    pages.end()
    assert pages.pool.report()[0] == batch * per
    return [torch.cat(o) for o in outputs], times


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--prompts", type=int, nargs="+", default=[500, 37, 1, 210])
    ap.add_argument("--chunk", type=int, default=128)
    ap.add_argument("--decode", type=int, default=16)
    a = ap.parse_args(argv)
    block = Block(a.width, a.heads, a.kv_heads)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randn(n + a.decode, a.width, generator=g, device="cuda").to(torch.bfloat16) for n in a.prompts]
    got, times = serve(block, prompts, a.chunk, a.decode)
    worst = 0.0
    for y, p in zip(got, prompts):
        want = block.plain(p)
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    print(f"{len(times)} steps, first {times[0] * 1e3:.2f} ms, median of the last {a.decode // 2} "
          f"{sorted(times[-(a.decode // 2):])[a.decode // 4] * 1e6:.0f} us; against float32 without 8 bits: "
          f"relative error {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()

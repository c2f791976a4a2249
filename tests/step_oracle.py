"""The definitions of a step's other operators (norm, rotary positions, pages) in 64 bits on
the CPU, and the tolerances that the roundings of their 32-bit steps allow."""
import torch

from block8_oracle import F64, U32, half_step, rounded


def norm(x, weight, residual, eps):
    """y with its tolerance before y's own rounding, and h.  h r is rounded to fp32 once, its product with the
    weight again; r is good to 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(residual.dtype)
    z = h.to(F64)
    y = z / (z.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.to(F64)
    return y, 2 * U32 * y.abs() + 2.0 ** -149, h


def check_codes(codes, scale, y, tol, what):
    """Rows in 8 bits of values known within tol: the scale is theirs within the largest tolerance and its own
    two roundings, and each code the nearest whole number to a quotient known within tol / s and the scale's
    share of 127."""
    top = y.abs().amax(-1)
    s = (top / 127).clamp_min(2.0 ** -126)
    most = tol.amax(-1)
    ds = most / 127 + 2 * U32 * s
    scale, codes = scale.cpu().to(F64), codes.cpu().to(F64)
    assert bool(((scale - s).abs() <= ds).all()), f"{what}: a scale is off"
    slack = tol / s[..., None] + 128 * (ds / s)[..., None] + 128 * 4 * U32
    off = (codes - y / s[..., None]).abs()
    assert bool((off <= 0.5 + slack).all()), f"{what}: a code is {float(off.max())} off"
    assert bool((codes.abs() <= 127).all())


def rotate(x, positions, frequencies, interleaved, magnitude):
    """x turned, and the tolerance before its own rounding.  The angle is good to 2^-51 of itself; less whole
    quarters it goes through fp32 three times (rounded, times 2 pi, whose own rounding is the third: 2.4 half
    steps at pi / 4), the series' last additions round by 2 more at most and leave out less than 1, the magnitude makes 2
    more and, as fp32 number, 1; the products and their sum round 3 times."""
    n = frequencies.numel()
    y, t = x.to(F64).clone(), positions.to(F64)[:, None] * frequencies.to(F64)[None]
    m = float(torch.tensor(magnitude, dtype=torch.float32))
    cos, sin = (m * t.cos())[:, None], (m * t.sin())[:, None]
    if interleaved:
        a, b = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
    else:
        a, b = slice(0, n), slice(n, 2 * n)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * cos - v * sin, v * cos + u * sin
    tol = torch.zeros_like(y)
    each = (u.abs() + v.abs()) * abs(m) * (11 * U32 + (t.abs() * 2.0 ** -51)[:, None])
    tol[..., a], tol[..., b] = each, each
    return y, tol


class Pages:
    """Tables, lengths and the pool as lists, sequence by sequence."""

    def __init__(self, free, count, page, table, lens):
        self.below, self.count, self.page = list(free), count, page
        self.table, self.lens = [list(r) for r in table], list(lens)
        self.lacking = self.left = 0

    def grow(self, more, tokens):
        p, pages = self.page, len(self.below)
        starts, slots, positions = [0], [-1] * tokens, [0] * tokens
        at = wanted = 0
        count, self.left = self.count, 0
        for b, n in enumerate(more):
            n, l = max(n, 0), max(self.lens[b], 0)
            first, at = at, at + n
            starts.append(min(at, tokens))
            if n == 0:
                continue
            had, want = -(-l // p), -(-(l + n) // p)
            if want > len(self.table[b]) or at > tokens or l + n >= 2 ** 31:
                self.left += 1
                continue
            wanted += want - had
            if wanted > count:
                self.left += 1
                continue
            for i in range(had, want):
                self.count -= 1
                self.table[b][i] = self.below[self.count]
            for j in range(n):
                page, off = self.table[b][(l + j) // p], (l + j) % p
                slots[first + j] = page * p + off if 0 <= page < pages else -1
                positions[first + j] = l + j
            self.lens[b] = l + n
        self.lacking = max(0, wanted - count)
        return starts, slots, positions

    def release(self, keep):
        p, back = self.page, []
        for b, k in enumerate(keep):
            l = max(self.lens[b], 0)
            k = min(l, max(k, 0))
            for i in range(-(-k // p), min(-(-l // p), len(self.table[b]))):
                back.append(self.table[b][i])
                self.table[b][i] = -1
            self.lens[b] = k
        back = [page for page in back if 0 <= page < len(self.below)]
        for r, page in enumerate(back):
            to = self.count + len(back) - 1 - r
            if to < len(self.below):
                self.below[to] = page
        self.count = min(self.count + len(back), len(self.below))

    def counts(self):
        return [self.count, self.lacking, self.left]

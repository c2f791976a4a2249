"""The definitions of the 8-bit block operators in 64 bits on the CPU, and the
tolerances that the roundings of their 32- and 16-bit steps allow."""
import math

import torch

F64 = torch.float64
U32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def quantize(x):
    """Rows of x (last axis) to codes and scales, as float64 and float32."""
    x = x.to(F64)
    s = (x.abs().amax(-1) / 127).float().clamp_min(2.0 ** -126)
    return torch.round(x / s.to(F64)[..., None]), s


def rounded(ref, tol, dtype):
    """Tolerance of a value known within tol that is then rounded to dtype."""
    return tol + half_step(dtype) * (ref.abs() + tol) + torch.finfo(dtype).smallest_normal * half_step(dtype)


def linear(x, w, ws, bias, silu):
    """y and its tolerance: the sum is exact; as fp32 it is rounded (1), times sa
    (2), times sw plus bias (3, 4); SiLU has a slope below 1.1 and its exponential,
    sum, reciprocal and product are good to 8 half steps and |v| of them (the
    exponent's rounding; without it for fp32, where it is compensated)."""
    codes, s = quantize(x)
    p = codes @ w.to(F64).t() * (s.to(F64)[:, None] * ws.to(F64))
    b = torch.zeros(w.shape[0], dtype=F64) if bias is None else bias.to(F64)
    v = p + b
    tol = 4 * U32 * (p.abs() + b.abs())
    if silu:
        y = v * torch.sigmoid(v)
        tol = 1.1 * tol + y.abs() * U32 * (8 + (0 if x.dtype == torch.float32 else 2 * v.abs()))
    else:
        y = v
    return y, rounded(y, tol, x.dtype)


def attention(q, k, v, table, starts, lens, window, scale, u_p):
    """out [tokens, heads, dim] and its tolerance; k, v: [pages, heads, page, dim]
    as float64 (what the cache stands for).

    u_p is half a step of the type in which the probabilities meet the values:
    each probability times its value's scale is off by that share, or, for fp16,
    by 2^-25 of the largest.  The scores are sums of dim products in fp32
    (their error turns into the probabilities' relative error, twice: once in the
    weights, once in the sum), exp2 and the scalings are good to 8 half steps, and the
    weighted sum runs over n keys in fp32, tile after tile, rescaled."""
    heads, dim = q.shape[1], q.shape[2]
    hk, page = k.shape[1], k.shape[2]
    group = heads // hk
    out = torch.zeros(q.shape, dtype=F64)
    tol = torch.zeros(q.shape, dtype=F64)
    mine = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(len(lens)):
        first, new = starts[b], starts[b + 1] - starts[b]
        n = min(lens[b], table.shape[1] * page)
        j = torch.arange(max(n, 0))
        pages = table[b].long()[j // page] if n > 0 else j
        there = (pages >= 0) & (pages < k.shape[0])
        pages = pages.clamp(0, k.shape[0] - 1)
        for i in range(new):
            mine[first + i] = True
            pos = lens[b] - new + i
            seen = there & (j <= pos)
            if window:
                seen &= j > pos - window
            if not bool(seen.any()):
                continue
            js, ps = j[seen], pages[seen]
            for h in range(hk):
                kk, vv = k[ps, h, js % page], v[ps, h, js % page]
                qq = q[first + i, h * group:(h + 1) * group].to(F64)
                z = qq @ kk.t() * scale
                p = torch.softmax(z, -1)
                o = p @ vv
                a = p @ vv.abs()
                dz = (dim + 8) * U32 * (qq.abs() @ kk.abs().t() * abs(scale)).amax(-1, keepdim=True)
                t = a * (u_p + 2 * dz + (8 + dim / 16 + len(js) / 16) * U32)
                if u_p == half_step(torch.float16):
                    t = t + len(js) * 2.0 ** -25 * (p.amax(-1, keepdim=True) * vv.abs().amax())
                out[first + i, h * group:(h + 1) * group] = o
                tol[first + i, h * group:(h + 1) * group] = t
    return out, rounded(out, tol, q.dtype), mine


def check(got, ref, tol, what):
    err = (got.cpu().to(F64) - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside tolerance, worst "
                                 f"{float((err / tol.clamp_min(1e-300)).nan_to_num(math.inf).max()):.3g} times it")

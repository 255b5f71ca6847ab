"""64-bit references of the operators around the layer, and inputs whose products are exact.

Everything here is written from the formulas in include/moe.h with elementary torch operations in float64.
"""
from __future__ import annotations

import torch

TINY = 2.0 ** -100
FLOOR = float(torch.tensor(TINY, dtype=torch.float32) / 127)  # the fp32 scale of a row of zeros
U24 = 2.0 ** -24  # half a step of fp32, relative
U8 = 2.0 ** -8    # half a step of bf16, relative


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm(v, w, w_add, eps):
    return v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * (w.double() + w_add)


def block_norm(r, y, w_post, gate, w_pre, r_scale, y_scale, w_add, eps):
    """(r', u, error bound of r', error bound of u) without the outputs' own rounding.  The bounds count fp32
    roundings: a norm's factor carries those of a sum of at most 64 + 8 terms in a row, its division, square root and
    two products, below 128 half steps in all; r' adds four products or sums."""
    k = 128 * U24
    r = r.double() * r_scale
    br = torch.zeros_like(r)
    if y is not None:
        z = y.double()
        if w_post is not None:
            z = norm(z, w_post, w_add, eps)
        if gate is not None:
            z = z * gate.double()
        z = z * y_scale
        br = k * (z.abs() + r.abs())
        r = r + z
    else:
        br = k * r.abs()
    if w_pre is None:
        return r, None, br, None
    rms = (r.square().mean(-1, keepdim=True) + eps).sqrt()
    u = norm(r, w_pre, w_add, eps)
    f = (w_pre.double() + w_add).abs() / rms
    # the factor's own error: the mean square moves with br, at most max(br) / rms relatively
    bu = f * br + u.abs() * (br.amax(-1, keepdim=True) / rms + k)
    return r, u, br, bu


def row_scales(v):
    """(scale, step) of the rows of v: max magnitude over 127, floored."""
    return v.abs().amax(-1).clamp_min(TINY) / 127


def swiglu(gu):
    g, u = gu.double().chunk(2, dim=-1)
    return g * torch.sigmoid(g) * u


def ints(g, shape, lo, hi, dtype):
    return torch.randint(lo, hi + 1, shape, generator=g, device=g.device).to(dtype)


def powers(g, shape):
    """Scales that are powers of two: products with them are exact."""
    return torch.exp2(torch.randint(-3, 4, shape, generator=g, device=g.device).float())


def grouped_positions(off, counts, rows, P, R):
    """[(expert, output row)] of every position that an expert owns, by the rule of the header (host lists)."""
    out = []
    E = len(off) - 1
    for e in range(E):
        first = min(max(off[e], 0), P)
        n = counts[e] if counts is not None else off[e + 1] - first
        for p in range(first, first + min(max(n, 0), P - first)):
            i = rows[p] if rows is not None else p
            if 0 <= i < R:
                out.append((e, i))
    return out

"""64-bit references of the operators around attention, from the formulas in include/moe.h, and their error bounds.

Bounds count roundings: U24 is half a step of fp32, U8 of bf16, relative to the value.
"""
from __future__ import annotations

import math

import torch

from tests.block_ref import TINY, U8, U24

TOP = {"i8": 127.0, "e4m3": 448.0}
TYPES = {"bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}


def rope(x, w, w_add, eps, pos, freq, mscale, rot, interleaved):
    """(values, bound of the fp32 computation) of x [T, heads, D].  The norm's factor carries fewer than 64 half steps
    (a sum of at most 8 + 5 terms in a row, a division, a square root, three products); an angle is off by one rounding
    of a value below pi, its sine and cosine by 4 ulp and mscale's product; the rotation adds two products and a sum."""
    v = x.double()
    if w is not None:
        v = v / (v.square().mean(-1, keepdim=True) + eps).sqrt() * (w.double() + w_add)
    bound = (64 * U24 * v.abs()) if w is not None else torch.zeros_like(v)
    if rot == 0:
        return v, bound
    turns = pos.double()[:, None] * freq
    a = 2 * math.pi * (turns - torch.round(turns))
    c, s = (a.cos() * mscale)[:, None], (a.sin() * mscale)[:, None]
    i = torch.arange(rot // 2, device=x.device)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out = v.clone()
    out[..., p] = v[..., p] * c - v[..., q] * s
    out[..., q] = v[..., q] * c + v[..., p] * s
    mag = (v[..., p].abs() + v[..., q].abs()) * abs(mscale)
    bound = bound.clone()
    bound[..., p] = bound[..., q] = (80 if w is not None else 16) * U24 * mag
    return out, bound


def scales(v, kind):
    return v.abs().amax(-1).clamp_min(TINY) / TOP[kind]


def code_bound(v, kind):
    """How far the value of a code may be from v, in units of the scale: half a step."""
    if kind == "i8":
        return torch.full_like(v, 0.5)
    return torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))


def gather(cache, scale, pages, n, P):
    """[Hkv, n, D] float64 keys of one sequence."""
    j = torch.arange(n, device=cache.device)
    page = pages.long()[j // P]
    x = cache[page, :, j % P].double()
    if scale is not None:
        x = x * scale[page, :, j % P].double()[..., None]
    return x.transpose(0, 1)


def attention(q, k_cache, v_cache, k_scale, v_scale, pages, q_start, kv_len, Hq, Hkv, D, P, scale, window, terms):
    """(out [T, Hq, D], lse [T, Hq], bound of out, bound of lse); rows outside all sequences are NaN.  `terms`: bf16
    terms of the softmax weights.

    A score is a sum of D exact products in fp32 (below D half steps of the sum of magnitudes), times the scale (one or
    two products) and, less the maximum, in base 2 (three more on its magnitude): ds.  A weight then is off by
    relative ds, the exponential's ulp (two half steps), and its rounding to bf16; the sums over n keys add n half
    steps, rescaling two per tile of 32 keys, joining parts a few."""
    T, G = q.shape[0], Hq // Hkv
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64, device=q.device)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    starts, lens = q_start.tolist(), kv_len.tolist()
    for s, L in enumerate(lens):
        a, n = starts[s], starts[s + 1] - starts[s]
        if n <= 0:
            continue
        L = max(0, min(L, pages.shape[1] * P))
        k, v = gather(k_cache, k_scale, pages[s], L, P), gather(v_cache, v_scale, pages[s], L, P)
        i = torch.arange(n, device=q.device)[:, None] + (L - n)
        j = torch.arange(L, device=q.device)[None]
        seen = (j <= i) & (j > i - window if window else True)
        for h in range(Hq):
            x = q[a:a + n, h * D:(h + 1) * D].double()
            kh, vh = k[h // G], v[h // G]
            sc = (x @ kh.t().contiguous()) * scale
            mag = (x.abs() @ kh.abs().t().contiguous()) * scale
            sc = torch.where(seen, sc, -math.inf)
            ds = (((D + 8) * U24) * torch.where(seen, mag, 0.0)).amax(-1, keepdim=True) if L else torch.zeros(n, 1, device=q.device, dtype=torch.float64)
            most = sc.amax(-1, keepdim=True) if L else torch.full((n, 1), -math.inf, device=q.device, dtype=torch.float64)
            e = torch.exp(sc - torch.where(most == -math.inf, 0.0, most)) * seen
            total = e.sum(-1, keepdim=True)
            none = ~seen.any(-1, keepdim=True) if L else torch.ones(n, 1, dtype=torch.bool, device=q.device)
            w = e / torch.where(none, 1.0, total)
            # a value that a row does not see leaves it alone, also if it is no number
            poison = (seen[..., None] & ~vh.isfinite()).any(1) if L and not bool(vh.isfinite().all()) else None
            o = w @ vh.nan_to_num(0.0, 0.0, 0.0)
            if poison is not None:
                o = torch.where(poison, float("nan"), o)
            rel = 2 * ds + (L + 2 * (L // 32) + 64) * U24 + U8 ** terms
            out[a:a + n, h] = torch.where(none, 0.0, o)
            lse[a:a + n, h] = torch.where(none, -math.inf, most + total.log())[:, 0]
            b_out[a:a + n, h] = rel * (w @ vh.abs().nan_to_num(0.0, 0.0, 0.0)) + U8 * o.abs()
            b_lse[a:a + n, h] = (ds + (L + 2 * (L // 32) + 64) * U24 + 8 * U24 * most.abs().nan_to_num(0, 0, 0))[:, 0]
    return out, lse, b_out, b_lse

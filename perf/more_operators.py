"""Cases for measuring the operators of the attention half of a block: rotary positions, the paged cache, attention
over it, and the bf16 products around it.

``run`` computes a case in plain torch operations (``own`` false) or through the library's entry points (``own``
true).  Kinds of cases:

  rope       heads of the query rows, normed or not, rotated by their positions
  cache      a step's q, k and v rows: q and k normed and rotated, k and v written to the paged cache, then read back
  attention  new tokens of ragged sequences over the paged cache
  gemm       c = act(a b^T + bias) + add in bf16
"""
import math
import random

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100  # rows quantise against at least this magnitude
DEV = "cuda"
TOP = {"i8": 127.0, "e4m3": 448.0}  # largest code of a type
CACHE = {"bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the query heads of one token in a decode step: launch latency
        dict(name="rope one token", kind="rope", T=1, heads=32, D=128, rot=128, pairs="half", norm=True, start=1000,
             stretch=1.0),
        # a long prefill far into a stretched context, part of each head rotated
        dict(name="rope prefill", kind="rope", T=8192, heads=32, D=128, rot=64, pairs="interleaved", norm=False,
             start=250000, stretch=8.0),
        # a decode step of several requests: one new token of each into an 8-bit float cache
        dict(name="cache decode e4m3", kind="cache", T=32, Hq=32, Hkv=4, D=128, rot=128, pairs="half", norm=True,
             start=5000, stretch=1.0, type="e4m3", P=64),
        # a prefill's tokens into an 8-bit integer cache
        dict(name="cache prefill i8", kind="cache", T=8192, Hq=16, Hkv=8, D=128, rot=128, pairs="half", norm=True,
             start=0, stretch=1.0, type="i8", P=64),
        # one token of one short request: launch latency
        dict(name="attention one token", kind="attention", S=1, new=1, past=128, ragged=False, Hq=32, Hkv=4, D=128,
             P=64, type="bf16", window=0, lse=False),
        # a decode step of requests of all lengths: the cache is read once
        dict(name="attention decode", kind="attention", S=64, new=1, past=8192, ragged=True, Hq=32, Hkv=4, D=128, P=64,
             type="bf16", window=0, lse=False),
        # two very long contexts: few rows, a long axis
        dict(name="attention decode long", kind="attention", S=2, new=1, past=131071, ragged=False, Hq=16, Hkv=2,
             D=256, P=128, type="e4m3", window=0, lse=False),
        # drafts of odd length verified over a cache of small pages
        dict(name="attention verify", kind="attention", S=16, new=7, past=4999, ragged=True, Hq=40, Hkv=8, D=128, P=16,
             type="i8", window=0, lse=False),
        # ragged chunks with a sliding window
        dict(name="attention window", kind="attention", S=13, new=1021, past=3000, ragged=True, Hq=24, Hkv=8, D=64,
             P=32, type="bf16", window=1024, lse=True),
        # a whole prompt
        dict(name="attention prefill", kind="attention", S=1, new=8192, past=0, ragged=False, Hq=32, Hkv=4, D=128,
             P=64, type="bf16", window=0, lse=False),
        # the output projection of one token, added to the residual stream
        dict(name="gemm one token", kind="gemm", M=1, K=4096, N=2048, bias=False, add=True, act="none", out="bf16"),
        # a biased and activated projection of a prefill
        dict(name="gemm prefill", kind="gemm", M=8192, K=2048, N=5120, bias=True, add=True, act="silu", out="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def _draw_rows(rng):
    D = rng.choice([64, 128, 256])
    return dict(D=D, rot=rng.choice([D, D // 2, D // 4]), pairs=rng.choice(["half", "interleaved"]),
                norm=rng.random() < 0.5, start=_log(rng, 1, 1000000), stretch=rng.choice([1.0, 4.0, 32.0]))


def draw(rng):
    kind = rng.choice(["rope", "cache", "attention", "attention", "attention", "gemm"])
    if kind == "rope":
        return dict(kind=kind, T=_log(rng, 1, 8192), heads=rng.randrange(1, 33), **_draw_rows(rng))
    if kind == "cache":
        Hkv = rng.choice([1, 2, 4, 8])
        return dict(kind=kind, T=_log(rng, 1, 8192), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, **_draw_rows(rng),
                    type=rng.choice(["bf16", "i8", "e4m3"]), P=rng.choice([16, 32, 64, 128, 256]))
    if kind == "gemm":
        return dict(kind=kind, M=_log(rng, 1, 8192), K=_log(rng, 64, 4096, 8), N=_log(rng, 64, 4096, 8),
                    bias=rng.random() < 0.5, add=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu"]),
                    out=rng.choice(["bf16", "fp32"]))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 128, 256])
    S = _log(rng, 1, 64)
    new = rng.choice([1, _log(rng, 2, 16), _log(rng, 17, 8192)])
    past = rng.choice([0, _log(rng, 1, 131072)])
    # no more than the prompt of the listed cases: scores of the padded batch, cached elements, arithmetic
    while S > 1 and S * new * (new + past) * Hkv * G > 2 ** 31 or S * (new + past) * Hkv * D > 2 ** 28:
        S = S // 2 if S > 1 else S
        past = past // 2 if S == 1 else past
    case = dict(kind=kind, S=S, new=new, past=past, ragged=rng.random() < 0.7, Hq=Hkv * G, Hkv=Hkv, D=D,
                P=rng.choice([16, 32, 64, 128, 256]), type=rng.choice(["bf16", "i8", "e4m3"]),
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), lse=rng.random() < 0.5)
    while case["S"] * case["Hq"] * case["new"] * (case["new"] + past) > 2 ** 31 or work(case)["flops"] > 5e11:
        case["new"] //= 2
    return case


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6007 + 29)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)


def _lengths(case):
    """(new tokens, keys) of each sequence: all alike, or spread over the range, single tokens and short contexts among
    them.  The seed only permutes them, so that every seed has the same work."""
    S, new, past = case["S"], case["new"], case["past"]
    if not case["ragged"]:
        return [(new, new + past)] * S
    n = [max(1, round(new * (s + 1) / S)) for s in range(S)]
    return [(n[s], n[s] + round(past * ((s * 0.6180339887 + 0.5) % 1.0))) for s in range(S)]


def _frequencies(rot, stretch):
    """Turns per token of each pair; stretched contexts slow the pairs that turn less than once in the original
    context of 4096 tokens, keep those that turn more than 32 times, and blend between (the rule of YaRN)."""
    f = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot) / (2 * math.pi)
    if stretch == 1.0:
        return f, 1.0
    keep = ((f * 4096 - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / stretch), 0.1 * math.log(stretch) + 1.0


def _quantised(g, kind, *shape):
    """(cache contents, scales) as a model leaves them: bell-shaped rows."""
    if kind == "bf16":
        return _randn(g, *shape), None
    top = TOP[kind]
    x = torch.randn(*shape, generator=g, device=DEV).mul_(top / 3.5).clamp_(-top, top)
    scale = torch.rand(*shape[:-1], generator=g, device=DEV).mul_(0.5).add_(0.75).mul_(3.5 / top)
    return (x.round_().to(torch.int8) if kind == "i8" else x.to(torch.float8_e4m3fn)), scale


def prepare(case, seed):
    g = _gen(seed)
    rng = random.Random(seed)
    s = dict(case)
    kind = case["kind"]
    bf = dict(dtype=torch.bfloat16, device=DEV)
    if kind in ("rope", "cache"):
        T, D = case["T"], case["D"]
        s["freq"], s["mscale"] = _frequencies(case["rot"], case["stretch"])
        s["pos"] = torch.arange(T, dtype=torch.int32, device=DEV) + (case["start"] + rng.randrange(1000))
        H = case["heads"] if kind == "rope" else case["Hq"]
        s["wq"] = _randn(g, D, scale=0.1).add_(1.0) if case["norm"] else None
        if kind == "rope":
            s["x"] = _randn(g, T, H * D)
            s["out"] = torch.empty(T, H * D, **bf)
            return s
        Hkv, P = case["Hkv"], case["P"]
        s["wk"] = _randn(g, D, scale=0.1).add_(1.0) if case["norm"] else None
        qkv = _randn(g, T, (H + 2 * Hkv) * D)  # one product's rows
        s["q"], s["k"], s["v"] = qkv[:, :H * D], qkv[:, H * D:(H + Hkv) * D], qkv[:, (H + Hkv) * D:]
        s["q_out"] = torch.empty(T, H * D, **bf)
        s["n_pages"] = n = T // P + 3
        # pages in no order, the first one filled from its middle
        page = torch.randperm(n, generator=g, device=DEV)
        at = torch.arange(T, device=DEV) + P // 2
        s["slots"] = (page[at // P] * P + at % P).to(torch.int32)
        s["k_cache"] = torch.zeros(n, Hkv, P, D, dtype=CACHE[case["type"]], device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["k_scale"] = None if case["type"] == "bf16" else torch.zeros(n, Hkv, P, dtype=torch.float32, device=DEV)
        s["v_scale"] = None if case["type"] == "bf16" else torch.zeros_like(s["k_scale"])
        s["k_back"], s["v_back"] = torch.empty(T, Hkv, D, **bf), torch.empty(T, Hkv, D, **bf)
        return s
    if kind == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["b"] = _randn(g, M, K), _randn(g, N, K, scale=K ** -0.5)
        s["bias_t"] = _randn(g, N, dtype=torch.float32) if case["bias"] else None
        s["add_t"] = _randn(g, M, N) if case["add"] else None
        s["c"] = torch.empty(M, N, dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16, device=DEV)
        return s
    lengths = _lengths(case)
    rng.shuffle(lengths)
    S, Hq, Hkv, D, P = case["S"], case["Hq"], case["Hkv"], case["D"], case["P"]
    new, keys = zip(*lengths)
    s["T"] = T = sum(new)
    s["most_new"], s["most_keys"] = max(new), max(keys)
    need = [-(-n // P) for n in keys]
    s["n_pages"], s["max_pages"] = n, m = sum(need) + 2, max(need) + 1
    # each sequence's pages lie anywhere in the pool; entries behind its last page name none
    s["q_start"] = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(keys, dtype=torch.int32, device=DEV)
    page = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(need[:i]) for i in range(S)], device=DEV)[:, None]
    col = torch.arange(m, device=DEV)[None]
    used = col < torch.tensor(need, device=DEV)[:, None]
    s["pages"] = torch.where(used, page[(first + col).clamp(max=n - 1)], -1).to(torch.int32).contiguous()
    s["k_cache"], s["k_scale"] = _quantised(g, case["type"], n, Hkv, P, D)
    s["v_cache"], s["v_scale"] = _quantised(g, case["type"], n, Hkv, P, D)
    s["q"] = _randn(g, T, Hq * D)
    s["scale"] = D ** -0.5
    s["out"] = torch.empty(T, Hq * D, **bf)
    s["lse_t"] = torch.empty(T, Hq, dtype=torch.float32, device=DEV) if case["lse"] else None
    # partial results of split sequences: what a program keeps for all layers
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_rope(s, x, w):
    """[T, heads, D] rows as rotated fp32 heads."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    turns = s["pos"].double()[:, None] * s["freq"]
    a = (turns - turns.floor()) * (2 * math.pi)
    c, n = (a.cos() * s["mscale"]).float()[:, None], (a.sin() * s["mscale"]).float()[:, None]
    r = s["rot"]
    x1, x2 = (x[..., :r // 2], x[..., r // 2:r]) if s["pairs"] == "half" else (x[..., 0:r:2], x[..., 1:r:2])
    y1, y2 = x1 * c - x2 * n, x2 * c + x1 * n
    y = torch.cat([y1, y2], -1) if s["pairs"] == "half" else torch.stack([y1, y2], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _plain_stored(x, kind):
    """fp32 rows as the cache holds them."""
    if kind == "bf16":
        return x.to(torch.bfloat16)
    a = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
    q = x * (TOP[kind] / a)
    q = q.round() if kind == "i8" else q.to(torch.float8_e4m3fn).float()
    return (q * (a / TOP[kind])).to(torch.bfloat16)


def _plain_keys(s, cache, scale):
    """[S * Hkv, keys, D] fp32 of a padded batch, zeros behind a sequence's last key."""
    P = s["P"]
    j = torch.arange(s["most_keys"], device=DEV)
    page = s["pages"].long()[:, j // P].clamp_min(0)
    at = (j % P).expand_as(page)
    x = cache[page, :, at].float()
    if scale is not None:
        x = x * scale[page, :, at][..., None]
    x = x * (j < s["kv_len"][:, None])[..., None, None]
    return x.transpose(1, 2).reshape(-1, s["most_keys"], s["D"])


def _plain_attention(s):
    S, Hq, Hkv, D, n = s["S"], s["Hq"], s["Hkv"], s["D"], s["most_new"]
    G = Hq // Hkv
    start = s["q_start"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(n, device=DEV)
    live = i < count[:, None]
    row = (start[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].view(s["T"], Hkv, G, D)[row].permute(0, 2, 1, 3, 4).reshape(S * Hkv, n * G, D).float()
    k, v = _plain_keys(s, s["k_cache"], s["k_scale"]), _plain_keys(s, s["v_cache"], s["v_scale"])
    score = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(s["scale"])
    j = torch.arange(s["most_keys"], device=DEV)
    at = (s["kv_len"].long() - count)[:, None] + i
    seen = j <= at[..., None]
    if s["window"]:
        seen = seen & (j > at[..., None] - s["window"])
    score.view(S, Hkv, n, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    most = score.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, 0.0, most)
    p = score.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p, v) / total.clamp_min(1e-38)
    o = o.view(S, Hkv, n, G, D).transpose(1, 2).reshape(S, n, Hq * D)
    lse = (most + total.log()).view(S, Hkv, n, G).transpose(1, 2).reshape(S, n, Hq)
    out = {"o": o[live].to(torch.bfloat16)}
    return {**out, "lse": lse[live]} if s["lse"] else out


def _run_plain(s):
    kind = s["kind"]
    if kind == "rope":
        x = _plain_rope(s, s["x"].view(s["T"], s["heads"], s["D"]), s["wq"])
        return {"x": x.to(torch.bfloat16).flatten(1)}
    if kind == "cache":
        q = _plain_rope(s, s["q"].unflatten(1, (s["Hq"], s["D"])), s["wq"])
        k = _plain_rope(s, s["k"].unflatten(1, (s["Hkv"], s["D"])), s["wk"])
        v = s["v"].unflatten(1, (s["Hkv"], s["D"])).float()
        return {"q": q.to(torch.bfloat16).flatten(1), "k": _plain_stored(k, s["type"]),
                "v": _plain_stored(v, s["type"])}
    if kind == "attention":
        return _plain_attention(s)
    c = s["a"].float() @ s["b"].float().t()
    if s["bias_t"] is not None:
        c = c + s["bias_t"]
    if s["act"] == "silu":
        c = c / (1.0 + torch.exp(-c))
    elif s["act"] == "gelu":
        c = 0.5 * c * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (c + 0.044715 * c * c * c)))
    if s["add_t"] is not None:
        c = c + s["add_t"].float()
    return {"c": c.to(s["c"].dtype)}


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    from sparse_moe_layer_03_amd import moe
    kind = s["kind"]
    pairs = moe.ROPE_INTERLEAVED if s.get("pairs") == "interleaved" else moe.ROPE_HALF
    if kind == "rope":
        moe.moe_rope(s["x"], s["wq"], s["pos"], s["freq"], s["T"], s["heads"], s["D"], s["rot"], pairs, s["out"],
                     mscale=s["mscale"], eps=EPS)
        return {"x": s["out"]}
    if kind == "cache":
        moe.moe_cache_write(s["q"], s["wq"], s["q_out"], s["k"], s["wk"], s["v"], s["pos"], s["freq"], s["slots"],
                            s["T"], s["Hq"], s["Hkv"], s["D"], s["rot"], pairs, s["k_cache"], s["v_cache"],
                            s["k_scale"], s["v_scale"], s["n_pages"], s["P"], mscale=s["mscale"], eps=EPS)
        moe.moe_cache_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"], s["T"], s["Hkv"],
                           s["D"], s["n_pages"], s["P"], s["k_back"], s["v_back"])
        return {"q": s["q_out"], "k": s["k_back"], "v": s["v_back"]}
    if kind == "attention":
        moe.moe_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["pages"], s["q_start"],
                          s["kv_len"], s["T"], s["S"], s["Hq"], s["Hkv"], s["D"], s["n_pages"], s["P"],
                          s["max_pages"], s["out"], s["workspace"], scale=s["scale"], window=s["window"],
                          lse=s["lse_t"])
        return {"o": s["out"], "lse": s["lse_t"]} if s["lse"] else {"o": s["out"]}
    act = {"none": moe.ACT_NONE, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}[s["act"]]
    moe.moe_gemm(s["a"], s["b"], s["bias_t"], s["add_t"], s["M"], s["N"], s["K"], s["c"], act=act)
    return {"c": s["c"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ work and exact values
def _seen(first, last, window):
    """Keys that the positions first .. last see together, with a window (0: none)."""
    full = lambda p: p * (p + 1) // 2  # positions 0 .. p - 1 see 1 .. p keys
    if not window:
        return full(last + 1) - full(first)
    short = lambda p: full(min(p, window)) + max(0, p - window) * window
    return short(last + 1) - short(first)


def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["T"] * case["heads"] * case["D"]
        return {"bytes": 4 * n + 4 * case["T"] + 4 * case["rot"], "flops": n * (7 if case["norm"] else 3)}
    if kind == "cache":
        T, D, Hq, Hkv = case["T"], case["D"], case["Hq"], case["Hkv"]
        held = 2 if case["type"] == "bf16" else 1
        scale = 0 if held == 2 else 4
        # q in and out, k and v in, into the cache, out of it and back
        n = T * (4 * Hq * D + 2 * Hkv * (2 * D + 2 * (held * D + scale) + 2 * D) + 12)
        return {"bytes": n, "flops": T * (Hq + 2 * Hkv) * D * (7 if case["norm"] else 3)}
    if kind == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        out = 4 if case["out"] == "fp32" else 2
        extra = (4 * N if case["bias"] else 0) + (2 * M * N if case["add"] else 0)
        return {"bytes": 2 * K * (M + N) + out * M * N + extra, "flops": 2.0 * M * N * K}
    D, Hq, Hkv, w = case["D"], case["Hq"], case["Hkv"], case["window"]
    row = D * (2 if case["type"] == "bf16" else 1) + (0 if case["type"] == "bf16" else 4)
    lengths = _lengths(case)
    T = sum(n for n, _ in lengths)
    read = sum(min(L, w + n - 1) if w else L for n, L in lengths)
    seen = sum(_seen(L - n, L - 1, w) for n, L in lengths)
    return {"bytes": 4 * T * Hq * D + 2 * read * Hkv * row + (4 * T * Hq if case["lse"] else 0) + 4 * read // case["P"],
            "flops": 4.0 * D * Hq * seen}


def _d(t):
    return None if t is None else t.to(torch.float64)


def _exact_rope(s, x, w):
    x = _d(x).clone()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * _d(w)
    r = s["rot"]
    # the angles' whole turns are taken out before the trigonometric functions see them
    turns = torch.remainder(torch.outer(_d(s["pos"]), s["freq"]), 1.0)
    z = torch.polar(torch.full_like(turns, s["mscale"]), 2 * math.pi * turns).unsqueeze(1)
    a = torch.arange(r // 2, device=x.device)
    first, second = (a, a + r // 2) if s["pairs"] == "half" else (2 * a, 2 * a + 1)
    z = torch.complex(x[..., first], x[..., second]) * z
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_stored(x, kind):
    """Rows after quantisation, as the values the codes stand for."""
    if kind == "bf16":
        return x
    largest = torch.maximum(x.max(dim=-1, keepdim=True).values, -x.min(dim=-1, keepdim=True).values)
    step = torch.clamp(largest, min=TINY) / TOP[kind]
    x = x / step
    if kind == "i8":
        return torch.round(x) * step
    # three bits behind the leading one, down to 2^-9
    ulp = torch.exp2(torch.clamp(torch.frexp(x).exponent - 1, min=-6).double() - 3)
    return torch.round(x / ulp) * ulp * step


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return {"x": _exact_rope(s, s["x"].view(s["T"], s["heads"], s["D"]), s["wq"]).flatten(1)}
    if kind == "cache":
        T, D = s["T"], s["D"]
        q = _exact_rope(s, s["q"].reshape(T, s["Hq"], D), s["wq"])
        k = _exact_rope(s, s["k"].reshape(T, s["Hkv"], D), s["wk"])
        v = _d(s["v"].reshape(T, s["Hkv"], D))
        return {"q": q.flatten(1), "k": _exact_stored(k, s["type"]), "v": _exact_stored(v, s["type"])}
    if kind == "gemm":
        c = torch.matmul(_d(s["a"]), _d(s["b"]).T.contiguous())
        if s["bias_t"] is not None:
            c += _d(s["bias_t"])
        if case["act"] == "silu":
            c = c * torch.sigmoid(c)
        elif case["act"] == "gelu":
            # (1 + tanh z) / 2 = sigmoid(2 z)
            c = c * torch.sigmoid(math.sqrt(8.0 / math.pi) * (c + 0.044715 * c.pow(3)))
        if s["add_t"] is not None:
            c += _d(s["add_t"])
        return {"c": c}
    D, P, G = s["D"], s["P"], s["Hq"] // s["Hkv"]
    out = torch.zeros(s["T"], s["Hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], s["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    start, keys = s["q_start"].tolist(), s["kv_len"].tolist()
    for b in range(s["S"]):
        n, L = start[b + 1] - start[b], keys[b]
        if n == 0 or L == 0:
            continue
        used = s["pages"][b, :-(-L // P)].long()
        i = torch.arange(n, device=DEV)[:, None] + (L - n)
        j = torch.arange(L, device=DEV)[None]
        hidden = (j > i) | (j <= i - s["window"]) if s["window"] else j > i
        for h in range(s["Hkv"]):
            k, v = _d(s["k_cache"][used, h].reshape(-1, D)[:L]), _d(s["v_cache"][used, h].reshape(-1, D)[:L])
            if s["k_scale"] is not None:
                k = k * _d(s["k_scale"][used, h].reshape(-1, 1)[:L])
                v = v * _d(s["v_scale"][used, h].reshape(-1, 1)[:L])
            kt = k.T.contiguous()
            for a in range(h * G, (h + 1) * G):
                x = torch.matmul(_d(s["q"][start[b]:start[b + 1], a * D:(a + 1) * D]), kt) * s["scale"]
                x[hidden] = -math.inf
                lse[start[b]:start[b + 1], a] = torch.logsumexp(x, -1)
                out[start[b]:start[b + 1], a] = torch.matmul(torch.softmax(x, -1), v)
    return {"o": out.flatten(1), "lse": lse} if s["lse"] else {"o": out.flatten(1)}

"""Rotary positions, the paged cache and attention over it against 64-bit references."""
import math

import pytest

from sparse_moe_layer_03_amd import moe
from tests import attend_ref as A
from tests import block_ref as B
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


def within(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, what
    odd = ~ref.isfinite()
    assert bool((got.isnan() == ref.isnan()).all()), f"{what}: NaN in other places"
    assert bool((got[odd & ~ref.isnan()] == ref[odd & ~ref.isnan()]).all()), f"{what}: infinities"
    d = torch_where(odd, got, ref)
    assert bool((d <= tol).all()), f"{what}: off by up to {float((d / tol.clamp_min(1e-300)).max()):.3g} of the bound"


def torch_where(odd, got, ref):
    import torch
    return torch.where(odd, 0.0, (got - ref).abs())


def rnd(torch, g, *shape, scale=1.0, dtype=None):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype or torch.bfloat16)


def columns(torch, g, T, width, extra):
    """[T, width] bf16 as the columns of wider rows (extra > 0), and the whole matrix."""
    whole = rnd(torch, g, T, width + extra)
    return (whole[:, extra // 2 // 8 * 8:][:, :width], whole) if extra else (whole, whole)


# ------------------------------------------------------------------ rotary positions
ROPE = [
    # T, heads, D, rot, interleaved, norm, extra columns, first position
    (1, 1, 8, 8, False, False, 0, 0), (1, 32, 128, 128, False, True, 0, 77), (3, 5, 64, 64, True, True, 16, 1000000),
    (7, 3, 96, 24, False, False, 0, 5), (5, 2, 80, 20, False, True, 8, 123), (4, 9, 256, 256, False, True, 0, 131071),
    (2, 130, 128, 64, True, False, 0, 9), (33, 1, 16, 2, False, False, 0, 2 ** 31 - 40), (9, 4, 64, 0, False, True, 24, 0),
    (5000, 2, 64, 32, False, False, 0, 0), (2049, 8, 128, 126, True, True, 64, 7), (3, 1, 256, 254, False, False, 0, 3),
    (6, 40, 72, 72, True, True, 0, -3),
]


@pytest.mark.parametrize("T,heads,D,rot,interleaved,norm,extra,first", ROPE)
def test_rope(torch, T, heads, D, rot, interleaved, norm, extra, first):
    G.say(f"[rope] T={T} heads={heads} D={D} rot={rot} interleaved={interleaved} norm={norm}")
    g = B.gen(T + heads + D + rot)
    x, _ = columns(torch, g, T, heads * D, extra)
    out, whole = columns(torch, g, T, heads * D, 2 * extra)
    before = whole.clone()
    w = rnd(torch, g, D, scale=0.3) if norm else None
    pos = torch.arange(first, first + T, device="cuda").int() if rot else None
    freq, ms = moe.moe_rope_frequencies(rot, 1e4, moe.ROPE_YARN, 4.0, 2048, "cuda") if rot else (None, 1.0)
    kw = dict(mscale=ms, w_add=1.0, eps=1e-5)
    moe.moe_rope(x, w, pos, freq, T, heads, D, rot, int(interleaved), out, **kw)
    ref, bound = A.rope(x.reshape(T, heads, D), w, 1.0, 1e-5, pos, freq, ms, rot, interleaved)
    within(out.reshape(T, heads, D), ref, bound + B.U8 * ref.abs() + 2.0 ** -133, "out")
    # columns beside the output keep their bits
    lo = 2 * extra // 2 // 8 * 8 if extra else 0
    for part in (slice(0, lo), slice(lo + heads * D, None)):
        assert torch.equal(whole[:, part], before[:, part])
    again = x.clone() if extra == 0 else torch.cat([x, x], dim=1)[:, :heads * D]
    moe.moe_rope(again, w, pos, freq, T, heads, D, rot, int(interleaved), again, **kw)
    assert torch.equal(again, out)


def test_rope_far_positions(torch):
    """The fastest pair turns by one radian a token: at position 2^31 - 1 the angle is right to fp32."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 999983], dtype=torch.int32, device="cuda")
    freq = torch.tensor([1 / (2 * math.pi)], dtype=torch.float64, device="cuda")
    x = torch.tensor([[1.0, 0.0]] * 3, dtype=torch.bfloat16, device="cuda")
    x = torch.nn.functional.pad(x, (0, 6))
    out = torch.empty_like(x)
    moe.moe_rope(x, None, pos, freq, 3, 1, 8, 2, moe.ROPE_INTERLEAVED, out)
    for t in range(3):
        for got, want in ((out[t, 0], math.cos(int(pos[t]))), (out[t, 1], math.sin(int(pos[t])))):
            # 2^31 turns of a radian: the frequency's own rounding moves the angle by 2^31 2^-53 2 pi
            assert abs(float(got) - want) <= B.U8 * abs(want) + 2.0 ** -18


def test_rope_not_finite(torch):
    """An infinity or a NaN reaches its pair, with a norm its head, and nothing else."""
    T, heads, D = 3, 4, 64
    g = B.gen(5)
    x = rnd(torch, g, T, heads * D)
    freq, _ = moe.moe_rope_frequencies(D, 1e4, device="cuda")
    pos = torch.arange(T, device="cuda").int()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    clean, out = torch.empty_like(x), torch.empty_like(x)
    for norm in (None, w):
        moe.moe_rope(x, norm, pos, freq, T, heads, D, D, moe.ROPE_HALF, clean)
        bad = x.clone()
        bad[1, 2 * D + 5] = float("nan")
        moe.moe_rope(bad, norm, pos, freq, T, heads, D, D, moe.ROPE_HALF, out)
        same = (out == clean)
        hit = [5, 37] if norm is None else list(range(D))
        assert bool(out[1, 2 * D:3 * D][hit].isnan().all())
        same[1, [2 * D + i for i in hit]] = True
        assert bool(same.all())


# ------------------------------------------------------------------ the cache
def new_cache(torch, kind, n_pages, Hkv, P, D, fill=None):
    t = torch.zeros(n_pages, Hkv, P, D, device="cuda")
    if fill is not None:
        t += fill
    k = t.to(A.TYPES[kind])
    s = None if kind == "bf16" else torch.full((n_pages, Hkv, P), -5.0, device="cuda")
    return k, k.clone(), s, None if s is None else s.clone()


CACHE = [
    # T, Hq, Hkv, D, rot, interleaved, norm, P, extra
    (1, 0, 1, 64, 64, False, False, 16, 0), (1, 8, 2, 128, 128, False, True, 64, 0), (37, 4, 4, 64, 32, True, True, 32, 8),
    (130, 6, 2, 256, 256, False, True, 128, 0), (65, 0, 3, 96, 96, False, False, 16, 40), (3000, 2, 1, 128, 64, True, False, 256, 0),
    (9, 40, 8, 128, 0, False, False, 1024, 0), (20, 3, 1, 8, 8, False, True, 16, 0),
]


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,norm,P,extra", CACHE)
def test_cache_write_and_read(torch, kind, T, Hq, Hkv, D, rot, interleaved, norm, P, extra):
    G.say(f"[cache] {kind} T={T} Hq={Hq} Hkv={Hkv} D={D} rot={rot} P={P}")
    g = B.gen(T + D + Hkv)
    width = (Hq + 2 * Hkv) * D
    qkv, _ = columns(torch, g, T, width, extra)
    qkv[:, ::29] *= 9
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
    wq, wk = (rnd(torch, g, D, scale=0.3), rnd(torch, g, D, scale=0.3)) if norm else (None, None)
    pos = (torch.arange(T, device="cuda") * 3 + 11).int() if rot else None
    freq = moe.moe_rope_frequencies(rot, 5e5, device="cuda")[0] if rot else None
    n_pages = T // P + 3
    kc, vc, ks, vs = new_cache(torch, kind, n_pages, Hkv, P, D, fill=1.5)
    slots = torch.randperm(n_pages * P, generator=g, device="cuda")[:T].int()
    slots[1::7] = -1
    slots[3::11] = n_pages * P + 3
    ok = (slots >= 0) & (slots < n_pages * P)
    old = [t.clone() if t is not None else None for t in (kc, vc, ks, vs)]
    q_out = torch.full((T, Hq * D), float("nan"), dtype=torch.bfloat16, device="cuda") if Hq else None
    kw = dict(w_add=1.0, eps=1e-5)
    moe.moe_cache_write(q if Hq else None, wq if Hq else None, q_out, k, wk, v, pos, freq, slots, T, Hq, Hkv, D, rot,
                        int(interleaved), kc, vc, ks, vs, n_pages, P, **kw)
    if Hq:
        alone = torch.empty_like(q_out)
        moe.moe_rope(q, wq, pos, freq, T, Hq, D, rot, int(interleaved), alone, **kw)
        assert torch.equal(q_out, alone)
    rk, bk = A.rope(k.reshape(T, Hkv, D), wk, 1.0, 1e-5, pos, freq, 1.0, rot, interleaved)
    rv = v.reshape(T, Hkv, D).double()
    at = slots[ok].long()
    page, place = at // P, at % P
    for name, cache, scale, ref, b, was, s_was in (("k", kc, ks, rk, bk, old[0], old[2]),
                                                   ("v", vc, vs, rv, 0 * rv, old[1], old[3])):
        got, ref, b = cache[page, :, place], ref[ok], b[ok]
        if kind == "bf16":
            within(got, ref, b + B.U8 * ref.abs() + 2.0 ** -133, name)
        else:
            s = A.scales(ref, kind)
            ds = b.amax(-1) / A.TOP[kind] + 4 * B.U24 * s
            within(scale[page, :, place], s, ds, name + " scale")
            u = ref / s[..., None]
            near = b / s[..., None] + u.abs() * ((ds / s)[..., None] + 4 * B.U24)
            within(got, u, A.code_bound(u.abs() + near, kind) + near, name + " codes")
        # every other slot as it was
        rest = torch.ones(n_pages, P, dtype=torch.bool, device="cuda")
        rest[page, place] = False
        same = cache.view(torch.uint8).reshape(n_pages, Hkv, P, -1) == was.view(torch.uint8).reshape(n_pages, Hkv, P, -1)
        assert bool(same.all(-1).transpose(1, 2)[rest].all())
        if scale is not None:
            assert bool((scale == s_was).transpose(1, 2)[rest].all())
    # read back: code times scale, rounded once; rows of other slots keep their bits
    for dt in (torch.bfloat16, torch.float32):
        k2, v2 = (torch.full((T, Hkv, D), -3.25, dtype=dt, device="cuda") for _ in range(2))
        moe.moe_cache_read(kc, vc, ks, vs, slots, T, Hkv, D, n_pages, P, k2, v2)
        for got, cache, scale in ((k2, kc, ks), (v2, vc, vs)):
            want = torch.full((T, Hkv, D), -3.25, device="cuda")
            x = cache[page, :, place].float()
            want[ok] = x if scale is None else x * scale[page, :, place][..., None]
            assert torch.equal(got, want.to(dt))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_cache_extremes(torch, kind):
    """Zeros, values below the floor, the largest bf16, infinities and NaN; a bad head leaves the others alone."""
    T, D, P = 6, 64, 16
    x = torch.zeros(T, 2 * D)
    x[1, :D] = 2.0 ** -120
    x[2, :D] = torch.finfo(torch.bfloat16).max
    x[3, 3] = float("inf")
    x[4, D - 1] = float("nan")
    x[5, :D] = torch.linspace(-3, 3, D)
    x[:, D:] = 1.0
    x = x.to(torch.bfloat16).cuda()
    kc, vc, ks, vs = new_cache(torch, kind, 1, 2, P, D)
    slots = torch.arange(T, device="cuda").int()
    moe.moe_cache_write(None, None, None, x, None, x, None, None, slots, T, 0, 2, D, 0, 0, kc, vc, ks, vs, 1, P)
    top = A.TOP[kind]
    floor = torch.tensor(B.TINY, dtype=torch.float32) / top
    for c, s in ((kc, ks), (vc, vs)):
        c = c.float()
        assert float(s[0, 0, 0]) == float(s[0, 0, 1]) == float(floor)
        assert bool(s[0, 0, 3].isnan()) and bool(s[0, 0, 4].isnan())
        for row in (0, 1, 3, 4):
            assert bool((c[0, 0, row] == 0).all())
        assert bool((c[0, 0, 2] == top).all()) and bool(s[0, 0, 2].isfinite())
        assert float(c[0, 0, 5].max()) == top and float(c[0, 0, 5].min()) == -top
        assert bool((c[0, 1, :T] == top).all()) and bool((s[0, 1, :T] == torch.tensor(1.0) / top).all())


@pytest.mark.parametrize("kind,j", [("i8", 1), ("e4m3", 1), ("e4m3", 3), ("e4m3", 5)])
def test_cache_halves(torch, kind, j):
    """Quotients halfway between two codes go to the even one.  Rows of bf16 values with a maximum of top * j: the code
    of j * v is v rounded.  The factor top / (top * j) rounded to fp32 is off by 0, 1/3 and 2/5 of a unit at most for 1 /
    1, 1 / 3 and 1 / 5, and v at most 31 / 16 of its power of two, so that a product is off by less than half a unit
    and rounds to v itself."""
    D, P = 64, 16
    top = A.TOP[kind]
    # i8: c + 1/2; e4m3: five significant bits, the last one set
    v = torch.arange(31 if kind == "i8" else 15, dtype=torch.float32)
    v = v + 0.5 if kind == "i8" else torch.cat([(17 + 2 * (v % 8)) * 2.0 ** e for e in (-5, 0, 3)])[:31]
    rows = torch.zeros(4, D)
    for i, e in enumerate((-9, 0, 1, 40)):
        rows[i, :31], rows[i, 31:62] = v * j * 2.0 ** e, -v * j * 2.0 ** e
        rows[i, 63] = top * j * 2.0 ** e
    x = rows.to(torch.bfloat16)
    assert torch.equal(x.float(), rows)
    x = x.cuda()
    kc, vc, ks, vs = new_cache(torch, kind, 1, 1, P, D)
    slots = torch.arange(4, device="cuda").int()
    moe.moe_cache_write(None, None, None, x, None, x, None, None, slots, 4, 0, 1, D, 0, 0, kc, vc, ks, vs, 1, P)
    want = v.round() if kind == "i8" else v.to(torch.float8_e4m3fn).float()
    for c in (kc, vc):
        for i in range(4):
            got = c[0, 0, i].float().cpu()
            assert torch.equal(got[:31], want) and torch.equal(got[31:62], -want) and float(got[63]) == top


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("D", [8, 64, 200])
def test_cache_codes_of_bf16_rows(torch, kind, D):
    """Codes of bf16 rows are x * top / max rounded to nearest, halves to even, all of them.  With x = X 2^p and max = M
    2^q in integers below 2^8, a boundary between codes is an odd B below 2^8 times a power of two, and X top and M B, up
    to a power of two, are integers below 2^17: they are equal, where the quotient is the boundary itself and fp32 holds
    it, or differ by more than 2^-17 of either, a hundred times what a quotient in fp32 is off by."""
    T, Hkv, P = 512, 4, 64
    n = T // P
    top = A.TOP[kind]
    x = torch.randn(T, Hkv * D, generator=B.gen(D), device="cuda").to(torch.bfloat16)
    kc, vc, ks, vs = new_cache(torch, kind, n, Hkv, P, D)
    slots = torch.arange(T, device="cuda").int()
    moe.moe_cache_write(None, None, None, x, None, x, None, None, slots, T, 0, Hkv, D, 0, 0, kc, vc, ks, vs, n, P)
    x = x.view(T, Hkv, D).double()
    want = x * top / x.abs().amax(-1, keepdim=True)
    want = want.round() if kind == "i8" else want.float().to(torch.float8_e4m3fn).double()
    for c in (kc, vc):
        got = c.float().permute(0, 2, 1, 3).reshape(T, Hkv, D).double()
        assert torch.equal(got, want)


# ------------------------------------------------------------------ attention
class Case:
    """Sequences (new tokens, keys) over a cache of random pages; slots and table entries that no row sees hold
    garbage."""

    def __init__(self, torch, lengths, Hq, Hkv, D, P, kind, window=0, seed=0, spare_rows=3, poison=True, q_scale=1.0):
        g = B.gen(seed * 7 + len(lengths) + D)
        self.torch, self.g = torch, g
        self.S, self.Hq, self.Hkv, self.D, self.P, self.kind, self.window = len(lengths), Hq, Hkv, D, P, kind, window
        new = [n for n, _ in lengths]
        keys = [L for _, L in lengths]
        self.T = sum(new) + spare_rows
        need = [-(-L // P) for L in keys]
        self.n_pages, self.max_pages = sum(need) + 2, max(need + [0]) + 2
        order = torch.randperm(self.n_pages, generator=g, device="cuda").int()
        self.pages = torch.full((self.S, self.max_pages), -1, dtype=torch.int32, device="cuda")
        self.pages[:, 1::2] = 2 ** 31 - 1
        at = 0
        for s, n in enumerate(need):
            self.pages[s, :n] = order[at:at + n]
            at += n
        self.q_start = torch.tensor([sum(new[:i]) for i in range(self.S + 1)], dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(keys, dtype=torch.int32, device="cuda")
        shape = (self.n_pages, Hkv, P, D)
        self.k, self.ks = self.fill(shape)
        self.v, self.vs = self.fill(shape)
        self.q = rnd(torch, g, self.T, Hq * D, scale=q_scale)
        if poison:
            self.poison(keys, new)

    def fill(self, shape):
        torch = self.torch
        if self.kind == "bf16":
            return rnd(torch, self.g, *shape), None
        top = A.TOP[self.kind]
        x = (torch.randn(*shape, generator=self.g, device="cuda") * top / 3).clamp(-top, top)
        s = (torch.rand(*shape[:-1], generator=self.g, device="cuda") + 0.5) * 3 / top
        return (x.round() if self.kind == "i8" else x).to(A.TYPES[self.kind]), s

    def poison(self, keys, new):
        """NaN in every slot that no row sees: behind the sequences' ends, before their windows, in unused pages."""
        torch, P = self.torch, self.P
        seen = torch.zeros(self.n_pages, P, dtype=torch.bool, device="cuda")
        for s, L in enumerate(keys):
            lo = max(0, L - new[s] - self.window + 1) if self.window else 0
            j = torch.arange(lo, max(lo, L), device="cuda")
            seen[self.pages[s].long()[j // P], j % P] = True
            if self.window and new[s]:
                self.pages[s, :lo // P] = -7  # pages that the window has left behind
        off = ~seen[:, None, :].expand(-1, self.Hkv, -1)
        for c, sc in ((self.k, self.ks), (self.v, self.vs)):
            if self.kind == "i8":
                c[off] = 77
            else:
                c.view(torch.int16 if self.kind == "bf16" else torch.uint8)[off] = 0x7fc0 if self.kind == "bf16" else 0x7f
            if sc is not None:
                sc[off] = float("nan")

    def args(self):
        return (self.T, self.S, self.Hq, self.Hkv, self.D, self.n_pages, self.P, self.max_pages)

    def workspace(self):
        torch = self.torch
        n = moe.moe_attention_workspace_size(self.T, self.S, self.Hq, self.Hkv, self.D, self.max_pages * self.P)
        return torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") if n else None

    def run(self, q=None, out=None, lse=True, workspace=None, **kw):
        torch = self.torch
        q = self.q if q is None else q
        if out is None:
            out = torch.full((self.T, self.Hq * self.D), -9.5, dtype=torch.bfloat16, device="cuda")
        l = torch.full((self.T, self.Hq), -9.5, device="cuda") if lse else None
        moe.moe_attention(q, self.k, self.v, self.ks, self.vs, self.pages, self.q_start, self.kv_len, *self.args(),
                          out, self.workspace() if workspace is None else workspace, window=self.window, lse=l, **kw)
        return out, l

    def check(self, out, lse, scale=None):
        torch = self.torch
        few = self.T * (self.Hq // self.Hkv) <= 32 * self.S
        pages = self.pages.clamp(0, self.n_pages - 1)
        ref, rl, bo, bl = A.attention(self.q, self.k, self.v, self.ks, self.vs, pages, self.q_start, self.kv_len,
                                      self.Hq, self.Hkv, self.D, self.P, scale or self.D ** -0.5, self.window,
                                      2 if few else 1)
        end = int(self.q_start[-1])
        assert bool((out[end:] == -9.5).all()), "rows behind the last sequence"
        within(out[:end].view(end, self.Hq, self.D), ref[:end], bo[:end], "out")
        if lse is not None:
            assert bool((lse[end:] == -9.5).all())
            within(lse[:end], rl[:end], bl[:end], "lse")


LENGTHS = {
    "one": [(1, 1)],
    "one long": [(1, 4097)],
    "decode": [(1, 700), (1, 1), (1, 64), (1, 65), (1, 127), (1, 128), (1, 2049), (1, 33)],
    "many decode": [(1, 3 + 41 * i % 900) for i in range(150)],
    "drafts": [(5, 500), (1, 1), (0, 40), (7, 7), (4, 1029), (3, 31), (2, 0), (6, 3)],
    "prompt": [(300, 300)],
    "chunk": [(129, 1500)],
    "ragged": [(70, 200), (0, 0), (1, 900), (257, 257), (33, 100), (0, 5), (128, 640), (9, 4)],
    "long chunk": [(64, 9000), (31, 6001)],
}
HEADS = [(1, 1, 64, 16, "bf16", 0), (8, 1, 128, 64, "bf16", 0), (6, 2, 256, 32, "bf16", 0), (32, 4, 128, 16, "i8", 0),
         (3, 3, 64, 128, "e4m3", 0), (16, 2, 256, 256, "e4m3", 0), (5, 1, 64, 32, "i8", 100), (4, 2, 128, 64, "bf16", 37),
         (12, 4, 64, 16, "bf16", 1), (4, 1, 256, 64, "i8", 300), (2, 2, 128, 1024, "e4m3", 700)]


@pytest.mark.parametrize("Hq,Hkv,D,P,kind,window", HEADS)
@pytest.mark.parametrize("lengths", list(LENGTHS))
def test_attention(torch, lengths, Hq, Hkv, D, P, kind, window):
    G.say(f"[attention] {lengths} Hq={Hq} Hkv={Hkv} D={D} P={P} {kind} window={window}")
    c = Case(torch, LENGTHS[lengths], Hq, Hkv, D, P, kind, window)
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", ["one long", "drafts", "chunk", "long chunk"])
def test_attention_types(torch, lengths, D, kind):
    """Every head size with every type, large scores among them: sharp rows, maxima that rise from tile to tile."""
    G.say(f"[attention types] {lengths} D={D} {kind}")
    c = Case(torch, LENGTHS[lengths], 4, 2, D, 32, kind, q_scale=6.0, seed=3)
    c.k.view(torch.uint8)  # the caches keep their types
    out, lse = c.run()
    c.check(out, lse)
    again, l2 = c.run()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, l2)


def test_attention_rows_in_place_of_columns(torch):
    """q as columns of a wider product's rows, out as columns of a wider buffer; a scale of its own; no lse."""
    c = Case(torch, LENGTHS["ragged"], 4, 2, 128, 16, "bf16", seed=5)
    wide = torch.full((c.T, c.Hq * c.D + 256), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:64 + c.Hq * c.D] = c.q
    to = torch.full((c.T, c.Hq * c.D + 40), -9.5, dtype=torch.bfloat16, device="cuda")
    out, _ = c.run(q=wide[:, 64:64 + c.Hq * c.D], out=to[:, 8:8 + c.Hq * c.D], lse=False, scale=0.25)
    c.check(out, None, scale=0.25)
    assert bool((to[:, :8] == -9.5).all()) and bool((to[:, 8 + c.Hq * c.D:] == -9.5).all())


@pytest.mark.parametrize("lengths,D,kind", [([(1, 900), (0, 5), (3, 3)], 128, "bf16"),
                                            ([(1, 5000)], 256, "bf16"),
                                            ([(7, 40), (2, 0)], 64, "i8"),
                                            ([(150, 400), (33, 20)], 128, "e4m3"),
                                            ([(200, 4500)], 64, "bf16"),
                                            ([(17000, 17000)], 128, "bf16")])
def test_attention_in_place(torch, lengths, D, kind):
    """out may be q: single tokens, shared-out keys, all row tiles; one sequence's row with an infinity in its q takes
    the second pass over its keys."""
    c = Case(torch, lengths, 8, 2, D, 16, kind, seed=11)
    if c.S == 1 and c.T < 9000:
        c.q[0, 3] = float("inf")
    want, wl = c.run()
    x = c.q.clone()
    out, lse = c.run(q=x, out=x)
    end = int(c.q_start[-1])
    assert torch.equal(x[:end].view(torch.int16), want[:end].view(torch.int16))
    assert torch.equal(lse.view(torch.int32), wl.view(torch.int32))
    assert torch.equal(x[end:], c.q[end:])


@pytest.mark.parametrize("lengths,Hq,Hkv,D,kind,window", [
    ([(431, 4000), (100, 2500)], 5, 1, 256, "bf16", 129),   # far windows, row tiles: not shared out
    ([(8, 3000), (1, 900), (5, 12)], 8, 2, 128, "i8", 1),   # the like for few rows
    ([(40, 5000), (3, 5000)], 4, 2, 64, "e4m3", 2500),      # a long window, shared out
    ([(300, 1500)], 4, 1, 128, "bf16", 0), ([(130, 1000), (64, 900)], 2, 2, 256, "i8", 0),  # few row tiles: small shares
    ([(900, 900)], 2, 1, 64, "e4m3", 0)])
def test_attention_shares(torch, lengths, Hq, Hkv, D, kind, window):
    """Both sides of the rule by which keys are shared out, over long tables of pages."""
    c = Case(torch, lengths, Hq, Hkv, D, 16, kind, window, seed=4)
    c.check(*c.run())


@pytest.mark.parametrize("lengths,where", [([(40, 40)], 20), ([(1, 300), (2, 300)], 299), ([(200, 700)], 650),
                                           ([(3, 9000)], 8998)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("in_v", [False, True])
def test_attention_not_finite(torch, lengths, where, bad, in_v):
    """A token whose key or value holds an infinity or a NaN: rows before it are those of a clean cache, bit for bit;
    rows that see it are NaN (key), or not finite in its channel alone (value)."""
    D, P = 64, 16
    c = Case(torch, lengths, 4, 2, D, P, "bf16", seed=9, poison=False)
    clean, _ = c.run()
    s = len(lengths) - 1
    page = int(c.pages[s, where // P])
    (c.v if in_v else c.k)[page, 1, where % P, 7] = bad
    out, lse = c.run()
    n, L = lengths[s]
    end = int(c.q_start[-1])
    first = end - n + max(0, where - (L - n))  # the first row that sees the token
    a, b = out.view(c.T, 4, D), clean.view(c.T, 4, D)
    ref, rl, bo, bl = A.attention(c.q, c.k, c.v, None, None, c.pages.clamp(0, c.n_pages - 1), c.q_start, c.kv_len, 4, 2,
                                  D, P, D ** -0.5, 0, 1)
    assert torch.equal(a[:, :2], b[:, :2])  # heads of the other key head
    if in_v:
        assert bool((~a[first:end, 2:, 7].isfinite()).all())
        keep = [d for d in range(D) if d != 7]
        within(a[:end, 2:][..., keep], ref[:end, 2:][..., keep], bo[:end, 2:][..., keep], "other channels")
        within(a[:first, 2:], ref[:first, 2:], bo[:first, 2:], "rows before")
    else:
        # a score of -infinity is a weight of 0, one of infinity or NaN makes the row NaN
        for r in range(first, end):
            for h in (2, 3):
                x = float(c.q[r, h * D + 7]) * bad
                if x == -float("inf"):
                    assert bool(a[r, h].isfinite().all())
                elif x != 0:
                    assert bool(a[r, h].isnan().all())
        assert torch.equal(a[:first], b[:first])


def test_attention_pages_that_are_none(torch):
    """A visible key whose page number is none: the rows that see it are NaN, nothing outside the cache is read."""
    for kind in ("bf16", "i8", "e4m3"):
        c = Case(torch, [(40, 100), (1, 70)], 2, 1, 64, 16, kind, poison=False)
        clean, _ = c.run()
        c.pages[0, 5] = c.n_pages  # keys 80 .. 95
        c.pages[1, 0] = -1
        out, _ = c.run()
        assert torch.equal(out[:20], clean[:20])  # positions 60 .. 79
        assert bool(out[20:41].isnan().all())


def test_attention_bounds_of_device_values(torch):
    """Lengths beyond the table and negative ones, starts outside [0, T] and falling: cut, never followed."""
    c = Case(torch, [(4, 40), (6, 50), (5, 60)], 2, 2, 64, 16, "bf16", poison=False)
    c.pages = c.pages[:, :4].contiguous()
    c.max_pages = 4
    c.pages.clamp_(0, c.n_pages - 1)
    c.kv_len[0], c.kv_len[1], c.kv_len[2] = 2 ** 31 - 1, -2 ** 31, 64
    c.q_start[0], c.q_start[3] = -5, 2 ** 30
    out, lse = c.run()
    start = c.q_start.clamp(0, c.T)
    kv = c.kv_len.clamp(0, 64)
    ref, rl, bo, bl = A.attention(c.q, c.k, c.v, None, None, c.pages, start, kv, 2, 2, 64, 16, 0.125, 0, 2)
    within(out.view(c.T, 2, 64), ref, bo, "out")
    within(lse, rl, bl, "lse")
    c.q_start[1], c.q_start[2] = 12, 3  # the middle sequence has no rows, the last begins before it
    out, _ = c.run()
    assert bool(out.isfinite().all())


def test_attention_long_cache(torch):
    """A cache of more than 2^32 elements: pages at its end, and one sequence of more than 2^17 keys."""
    Hkv, P, D = 2, 1024, 128
    n_pages = (2 ** 32 + 2 ** 28) // (Hkv * P * D)
    g = B.gen(1)
    k = torch.empty(n_pages, Hkv, P, D, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks = torch.empty(n_pages, Hkv, P, device="cuda")
    vs = torch.empty_like(ks)
    lengths = [140000, 1500]
    need = [-(-L // P) for L in lengths]
    used = torch.cat([torch.arange(n_pages - need[0], n_pages, device="cuda"), torch.arange(0, need[1], device="cuda")])
    k[used] = B.ints(g, (len(used), Hkv, P, D), -127, 127, torch.int8)
    v[used] = B.ints(g, (len(used), Hkv, P, D), -127, 127, torch.int8)
    ks[used] = torch.rand(len(used), Hkv, P, generator=g, device="cuda") * 0.02
    vs[used] = torch.rand(len(used), Hkv, P, generator=g, device="cuda") * 0.02
    pages = torch.full((2, need[0]), -1, dtype=torch.int32, device="cuda")
    pages[0], pages[1, :need[1]] = used[:need[0]].flip(0), used[need[0]:]
    for new in (1, 40):
        T, Hq = 2 * new, 4
        q = rnd(torch, g, T, Hq * D)
        q_start = torch.tensor([0, new, T], dtype=torch.int32, device="cuda")
        kv = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out = torch.empty(T, Hq * D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, Hq, device="cuda")
        ws = torch.empty(moe.moe_attention_workspace_size(T, 2, Hq, Hkv, D, need[0] * P), dtype=torch.uint8, device="cuda")
        moe.moe_attention(q, k, v, ks, vs, pages, q_start, kv, T, 2, Hq, Hkv, D, n_pages, P, need[0], out, ws, lse=lse)
        ref, rl, bo, bl = A.attention(q, k, v, ks, vs, pages.clamp_min(0), q_start, kv, Hq, Hkv, D, P, D ** -0.5, 0,
                                      2 if new * 2 <= 32 else 1)
        within(out.view(T, Hq, D), ref, bo, "out")
        within(lse, rl, bl, "lse")
    # the write and the read at the same places
    x = rnd(torch, g, 2, Hkv * D)
    slots = torch.tensor([n_pages * P - 1, 5], dtype=torch.int32, device="cuda")
    moe.moe_cache_write(None, None, None, x, None, x, None, None, slots, 2, 0, Hkv, D, 0, 0, k, v, ks, vs, n_pages, P)
    kb, vb = torch.empty(2, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, Hkv, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_cache_read(k, v, ks, vs, slots, 2, Hkv, D, n_pages, P, kb, vb)
    top = x.view(2, Hkv, D).float().abs().amax(-1, keepdim=True)
    for got in (kb, vb):
        assert bool(((got.float() - x.view(2, Hkv, D).float()).abs() <= top * (0.51 / 127 + B.U8)).all())


def test_attention_joined_halves(torch):
    """Two halves of the keys joined by their lse are the whole."""
    c = Case(torch, [(1, 256), (1, 512)], 4, 2, 128, 64, "bf16", seed=2, spare_rows=0)
    whole, lw = c.run()
    parts = []
    for lo in (True, False):
        h = Case(torch, [(1, 256), (1, 512)], 4, 2, 128, 64, "bf16", seed=2, spare_rows=0)
        half = h.kv_len // 2
        if not lo:
            h.pages = torch.stack([torch.roll(h.pages[s], -int(half[s]) // 64) for s in range(2)]).contiguous()
        h.kv_len = half.int()
        parts.append(h.run())
    (o1, l1), (o2, l2) = parts
    top = torch.maximum(l1, l2)
    w1, w2 = (l1 - top).exp()[..., None], (l2 - top).exp()[..., None]
    o = (o1.float().view(2, 4, 128) * w1 + o2.float().view(2, 4, 128) * w2) / (w1 + w2)
    # each half and the whole are rounded once
    mag = (o1.float().abs().view(2, 4, 128) * w1 + o2.float().abs().view(2, 4, 128) * w2) / (w1 + w2)
    assert bool(((o - whole.float().view(2, 4, 128)).abs() <= 2.1 * B.U8 * mag + 2.0 ** -14).all())
    assert bool((torch.logaddexp(l1, l2) - lw).abs().max() < 1e-5)


# ------------------------------------------------------------------ how they are called
@pytest.mark.parametrize("lengths", ["many decode", "long chunk", "ragged"])
def test_attention_streams_and_graphs(torch, lengths):
    """Two calls at once on two streams with a workspace each; captured, replayed several times with eager work and new
    lengths in place between the replays."""
    c = Case(torch, LENGTHS[lengths], 8, 2, 128, 32, "bf16", seed=11, poison=False)
    want, wl = c.run()
    ws = [c.workspace() for _ in range(2)]
    outs = [torch.full_like(want, -9.5) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, w, o in zip(streams, ws, outs):
            c.run(out=o, workspace=w, lse=False, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    lse = torch.empty(c.T, c.Hq, device="cuda")
    with torch.cuda.graph(g):
        moe.moe_attention(c.q, c.k, c.v, c.ks, c.vs, c.pages, c.q_start, c.kv_len, *c.args(), outs[0], ws[0], lse=lse)
    for step in range(4):
        outs[0].fill_(-9.5), lse.fill_(-9.5)
        g.replay()
        eager, el = c.run()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(lse, el)
        c.kv_len.sub_(1).clamp_min_(0)  # shorter contexts for the next replay
        c.q.mul_(-1)


def test_a_step_captured(torch):
    """The write, attention and the read of a decode step in one graph, replayed over growing lengths."""
    S, Hq, Hkv, D, P = 5, 4, 2, 64, 16
    g = B.gen(4)
    n_pages, max_pages = 40, 8
    kc, vc, ks, vs = new_cache(torch, "e4m3", n_pages, Hkv, P, D)
    pages = torch.randperm(n_pages, generator=g, device="cuda")[:S * max_pages].view(S, max_pages).int().contiguous()
    qkv = torch.empty(S, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:]
    pos, kv = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.zeros(S, dtype=torch.int32, device="cuda")
    slots, q_start = torch.zeros(S, dtype=torch.int32, device="cuda"), torch.arange(S + 1, device="cuda").int()
    freq, _ = moe.moe_rope_frequencies(D, 1e4, device="cuda")
    out, kb, vb = torch.empty(S, Hq * D, dtype=torch.bfloat16, device="cuda"), *(torch.empty(S, Hkv, D, device="cuda") for _ in range(2))
    n = moe.moe_attention_workspace_size(S, S, Hq, Hkv, D, max_pages * P)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")

    def step(out, kb, vb):
        moe.moe_cache_write(q, None, q, k, None, v, pos, freq, slots, S, Hq, Hkv, D, D, moe.ROPE_HALF, kc, vc, ks, vs,
                            n_pages, P)
        moe.moe_attention(q, kc, vc, ks, vs, pages, q_start, kv, S, S, Hq, Hkv, D, n_pages, P, max_pages, out, ws)
        moe.moe_cache_read(kc, vc, ks, vs, slots, S, Hkv, D, n_pages, P, kb, vb)
    x = rnd(torch, g, 12, S, (Hq + 2 * Hkv) * D)

    def set_step(t):
        qkv.copy_(x[t])
        pos.fill_(t), kv.fill_(t + 1)
        slots.copy_(pages[:, t // P] * P + t % P)
    set_step(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out, kb, vb)
    for t in range(12):
        set_step(t)
        graph.replay()
        torch.cuda.synchronize()
        got = [z.clone() for z in (out, kb, vb)]
        set_step(t)
        step(out, kb, vb)
        torch.cuda.synchronize()
        for a, b in zip(got, (out, kb, vb)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ products
def dense(torch, M, N, K, out, seed, lim=8):
    g = B.gen(seed + M + N + K)
    a, b = B.ints(g, (M, K), -lim, lim, torch.bfloat16), B.ints(g, (N, K), -lim, lim, torch.bfloat16)
    c = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    return g, a, b, c


GEMM = [(1, 8, 8), (1, 4096, 2048), (2, 24, 40), (3, 1000, 56), (15, 72, 64), (16, 64, 72), (17, 136, 128), (31, 512, 1024),
        (33, 1024, 520), (48, 40, 2048), (63, 2048, 256), (64, 256, 24), (65, 264, 2056), (100, 8, 4096), (129, 1032, 192),
        (200, 2048, 1024), (257, 768, 320), (300, 1544, 392), (511, 24, 8), (1000, 1000, 504), (1024, 2048, 1024),
        (2049, 520, 264), (70, 40, 65536), (2001, 3000, 200), (3900, 4104, 136), (4096, 4096, 128), (64, 4096, 1024),
        (40, 4096, 512)]


@pytest.mark.parametrize("M,N,K", GEMM)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_gemm_exact(torch, M, N, K, out):
    """Small integers: sums exact in fp32, every element bit for bit, with bias and addend too."""
    G.say(f"[gemm] {M} x {N} x {K} {out}")
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    g, a, b, c = dense(torch, M, N, K, dt, 0, lim=8 if K <= 4096 else 4)
    ref = a.double() @ b.double().t().contiguous()
    moe.moe_gemm(a, b, None, None, M, N, K, c)
    assert torch.equal(c, ref.float().to(dt))
    bias, add = B.ints(g, (N,), -64, 64, torch.float32), B.ints(g, (M, N), -64, 64, torch.bfloat16)
    for bt, at in ((bias, None), (None, add), (bias, add)):
        want = ref + (0 if bt is None else bt.double()) + (0 if at is None else at.double())
        c.fill_(float("nan"))
        moe.moe_gemm(a, b, bt, at, M, N, K, c)
        assert torch.equal(c, want.float().to(dt)), (bt is not None, at is not None)
    if out == "bf16":
        c2 = add.clone()
        moe.moe_gemm(a, b, bias, c2, M, N, K, c2)
        assert torch.equal(c2, c)


@pytest.mark.parametrize("M,N,K", [(1, 264, 512), (20, 72, 1032), (50, 1024, 128), (130, 520, 512), (600, 776, 264),
                                   (2000, 3000, 200), (3900, 4104, 136)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gemm_activations(torch, M, N, K, out, act):
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    g = B.gen(M + N + K)
    a, b = rnd(torch, g, M, K), rnd(torch, g, N, K, scale=2 * K ** -0.5)
    bias, add = rnd(torch, g, N, dtype=torch.float32), rnd(torch, g, M, N)
    c = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    for bt, at in ((None, None), (bias, add)):
        moe.moe_gemm(a, b, bt, at, M, N, K, c, act={"none": 0, "silu": 1, "gelu": 2}[act])
        v = a.double() @ b.double().t().contiguous()
        dv = (K + 2) * B.U24 * ((a.double().abs() @ b.double().abs().t().contiguous()) + (0 if bt is None else bt.double().abs()))
        if bt is not None:
            v = v + bt.double()
        f = v
        if act == "silu":
            f = v * torch.sigmoid(v)
        elif act == "gelu":
            f = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
        # the activations' slopes stay below 1.2; the exponent's argument z (below |v| or 1.6 |v| + 0.08 |v|^3) carries a
        # few half steps, and e^-z weighs them by z e^-z / (1 + e^-z)^2 < 0.3 of v
        tol = dv if act == "none" else 1.2 * dv + 16 * B.U24 * v.abs()
        if at is not None:
            f = f + at.double()
            tol = tol + 2 * B.U24 * (f.abs() + at.double().abs())
        within(c, f, tol + B.half_step(dt) * f.abs() + 1e-30, act)


def test_gemm_not_finite(torch):
    """A NaN in a row of a reaches its row of c alone, one in a row of b its column."""
    for M in (4, 40, 300):
        a, b = torch.ones(M, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(72, 64, dtype=torch.bfloat16, device="cuda")
        a[1, 63], b[9, 0] = float("nan"), float("inf")
        c = torch.empty(M, 72, dtype=torch.bfloat16, device="cuda")
        moe.moe_gemm(a, b, None, None, M, 72, 64, c)
        assert bool(c[1].isnan().all()) and bool((c[[0] + list(range(2, M)), 9] == float("inf")).all())
        c[1], c[:, 9] = 64, 64
        assert bool((c == 64).all())

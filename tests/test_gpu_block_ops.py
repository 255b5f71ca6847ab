"""The operators around the layer against 64-bit references: norms, 8-bit rows, dense and grouped products.

Products are tested on inputs whose sums and scales are exact in fp32 (small integers, powers of two), so that
every output element has to equal the correctly rounded one bit for bit, whatever the order of the sums; a second
set with general values is held to counted roundings.
"""
import pytest

from sparse_moe_layer_03_amd import moe
from tests import block_ref as B
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


def dt(torch, name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def same_bits(torch, a, b, what):
    it = {2: torch.int16, 4: torch.int32, 1: torch.int8}[a.element_size()]
    bad = (a.view(it) != b.view(it)).nonzero()
    assert bad.numel() == 0, f"{what}: {bad.shape[0]} elements differ, first at {bad[0].tolist()}"


def within(got, ref, tol, what):
    d = (got.double() - ref).abs()
    assert bool((d <= tol).all()), f"{what}: off by up to {float((d / tol.clamp_min(1e-300)).max()):.3g} of the bound"


# ------------------------------------------------------------------ norms
NORM_CASES = [
    # T, H, stream, y, post, gate rows (0 none, 1, 2 = T), x, q
    (1, 16, "bf16", True, True, 1, True, True), (3, 48, "fp32", True, False, 2, True, False),
    (5, 512, "bf16", True, True, 2, False, True), (7, 528, "fp32", False, False, 0, True, True),
    (4, 1024, "bf16", True, False, 0, True, False), (9, 1040, "bf16", True, True, 1, True, True),
    (1, 2048, "bf16", True, False, 0, True, True), (130, 2048, "fp32", True, True, 1, True, True),
    (6, 2064, "bf16", True, True, 2, True, True), (2, 4096, "fp32", True, True, 0, False, True),
    (3, 4112, "bf16", False, False, 0, True, False), (3, 8192, "fp32", True, True, 2, True, True),
    (2, 8208, "bf16", True, False, 1, True, True), (2, 16384, "fp32", True, True, 1, True, True),
    (5, 256, "bf16", True, True, 1, False, False), (5, 256, "fp32", False, False, 0, False, False),
    (4097, 64, "bf16", True, True, 1, True, True),
]


@pytest.mark.parametrize("T,H,stream,has_y,post,gate,has_x,has_q", NORM_CASES)
def test_block_norm(torch, T, H, stream, has_y, post, gate, has_x, has_q):
    G.say(f"[norm] T={T} H={H} {stream} y={has_y} post={post} gate={gate}")
    g = B.gen(T * 7 + H)
    bf = torch.bfloat16
    rt = dt(torch, stream)

    def rnd(*shape, scale=1.0, dtype=bf):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    r = rnd(T, H, scale=3.0, dtype=rt)
    y = rnd(T, H) if has_y else None
    w_post = rnd(H, scale=0.3) if post else None
    gt = None if gate == 0 else rnd(H) if gate == 1 else rnd(T, H)
    normed = has_x or has_q
    w_pre = rnd(H, scale=0.3) if normed else None
    r_out = torch.full((T, H), float("nan"), dtype=rt, device="cuda")
    x = torch.full((T, H), float("nan"), dtype=bf, device="cuda") if has_x else None
    q = torch.full((T, H), 99, dtype=torch.int8, device="cuda") if has_q else None
    qs = torch.full((T,), float("nan"), device="cuda") if has_q else None
    kw = dict(r_scale=0.75, y_scale=1.5, w_add=1.0, eps=1e-5)
    moe.moe_block_norm(r, y, w_post, gt, w_pre, T, H, r_out, x, q, qs, **kw)
    ref_r, ref_u, br, bu = B.block_norm(r, y, w_post, gt, w_pre, 0.75, 1.5, 1.0, 1e-5)
    within(r_out, ref_r, br + B.half_step(rt) * ref_r.abs(), "r'")
    if has_x:
        within(x, ref_u, bu + B.half_step(bf) * ref_u.abs(), "x")
    if has_q:
        s = B.row_scales(ref_u)
        ds = bu.amax(-1) / 127 + 4 * B.U24 * s
        within(qs, s, ds, "scale")
        # a code is within half a step of the value it stands for, its roundings and the scale's error added
        v = ref_u / s[:, None]
        within(q, v, 0.5 + bu / s[:, None] + v.abs() * (ds / s)[:, None] + 127 * 4 * B.U24, "codes")
    # in place: r' over r and x over y give the same bits
    if has_y and has_x:
        r2, y2 = r.clone(), y.clone()
        moe.moe_block_norm(r2, y2, w_post, gt, w_pre, T, H, r2, y2, None, None, **kw)
        same_bits(torch, r2, r_out, "r' in place")
        same_bits(torch, y2, x, "x in place")


def test_block_norm_extremes(torch):
    """Rows of zeros, of tiny and of large values, and one row with an infinity or a NaN beside clean ones."""
    H = 256
    r = torch.zeros(6, H, device="cuda")
    r[1] = 1e-30
    r[2, 5] = float("inf")
    r[3, 7] = float("nan")
    r[4] = torch.linspace(-1e15, 1e15, H, device="cuda")
    r[5] = torch.linspace(-1, 1, H, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(r)
    x = torch.empty(6, H, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(6, H, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    moe.moe_block_norm(r, None, None, None, w, 6, H, out, x, q, s, eps=1e-6)
    assert torch.equal(out.isnan(), r.isnan()) and torch.equal(out.nan_to_num(), r.nan_to_num())
    assert bool((x[0] == 0).all()) and bool((q[0] == 0).all()) and float(s[0]) == B.FLOOR
    for bad in (2, 3):
        assert bool(s[bad].isnan()) and bool((q[bad] == 0).all()) and bool(x[bad].isnan().any())
    for row in (4, 5):
        assert bool(s[row].isfinite()) and int(q[row].abs().max()) == 127 and bool(x[row].isfinite().all())
    # eps = 0 on a row of zeros is 0 * infinity, by the formula a NaN; the codes say so too
    moe.moe_block_norm(r, None, None, None, w, 1, H, None, x, q, s, eps=0.0)
    assert bool(x[0].isnan().all()) and bool(s[0].isnan())


# ------------------------------------------------------------------ 8-bit rows
@pytest.mark.parametrize("R,K", [(1, 16), (5, 48), (3, 512), (66, 528), (2, 1024), (9, 2048), (4, 2064), (3, 4096),
                                 (2, 8192), (2, 8208), (3, 16384), (2, 16400), (2, 32768), (5000, 32)])
def test_quantize_and_swiglu(torch, R, K):
    G.say(f"[quantize] R={R} K={K}")
    g = B.gen(R + K)
    x = torch.randn(R, 2 * K, generator=g, device="cuda")
    x[:, ::37] *= 20
    x = x.to(torch.bfloat16)
    q = torch.full((R, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((R,), float("nan"), device="cuda")
    plain = x[:, :K].contiguous()
    moe.moe_quantize_i8(plain, R, K, q, s)
    sr = B.row_scales(plain.double())
    within(s, sr, 2 * B.U24 * sr, "scale")
    v = plain.double() / sr[:, None]
    within(q, v, 0.5 + 127 * 4 * B.U24 + 0 * v, "codes")
    gate = torch.rand(R, generator=g, device="cuda")
    for rg in (None, gate):
        moe.moe_swiglu_i8(x, rg, R, K, q, s)
        h = B.swiglu(x)
        # silu: the exponent's argument carries |g| half steps, the rest of the chain below 8 more, twice each
        rel = (x[:, :K].double().abs().clamp_max(128).amax() + 8) * 2 * B.U24
        hr = B.row_scales(h)
        f = 1.0 if rg is None else rg.double()
        within(s, hr * f, (rel + 4 * B.U24) * hr * f + 1e-45, "swiglu scale")
        v = h / hr[:, None]
        within(q, v, 0.5 + 127 * (2 * rel + 4 * B.U24) + 0 * v, "swiglu codes")


def test_quantize_extremes(torch):
    """Zeros, values below the floor, the largest bf16, infinities and NaN; a bad row leaves the others alone."""
    K = 64
    x = torch.zeros(7, K)
    x[1] = 2.0 ** -120
    x[2] = torch.finfo(torch.bfloat16).max
    x[3, 0] = float("inf")
    x[4, 63] = float("nan")
    x[5] = torch.linspace(-3, 3, K)
    x[6, 3] = -float("inf")
    x = x.to(torch.bfloat16).cuda()
    q, s = torch.full((7, K), 99, dtype=torch.int8, device="cuda"), torch.zeros(7, device="cuda")
    moe.moe_quantize_i8(x, 7, K, q, s)
    for row in (0, 1, 3, 4, 6):
        assert bool((q[row] == 0).all())
    assert float(s[0]) == float(s[1]) == B.FLOOR
    assert bool(s[3].isnan()) and bool(s[4].isnan()) and bool(s[6].isnan())
    assert bool((q[2] == 127).all()) and bool(s[2].isfinite())
    assert int(q[5].max()) == 127 and int(q[5].min()) == -127
    # silu of far negative gates is 0, of far positive ones the gate itself
    gu = torch.tensor([[-1e30] * 16 + [2.0] * 16, [1e4] * 16 + [0.5] * 16], dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(2, 16, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    moe.moe_swiglu_i8(gu, None, 2, 16, q, s)
    assert bool((q[0] == 0).all()) and bool((q[1] == 127).all())
    assert float(s[0]) == B.FLOOR and abs(float(s[1]) * 127 - float(gu[1, 0]) * 0.5) < 1e-3


# ------------------------------------------------------------------ dense products
DENSE = [(1, 8, 16), (1, 4096, 2048), (2, 24, 48), (3, 1000, 112), (15, 72, 128), (16, 64, 144), (17, 136, 256),
         (31, 512, 2048), (33, 1024, 1040), (48, 40, 4096), (63, 2048, 512), (64, 256, 64), (65, 264, 4112),
         (100, 8, 8192), (127, 520, 272), (128, 128, 2048), (129, 1032, 384), (200, 2048, 2048), (255, 256, 128),
         (256, 512, 1024), (257, 768, 640), (300, 1544, 784), (511, 24, 16), (1000, 1000, 1008), (1024, 2048, 2048),
         (2049, 520, 528), (70, 40, 65536), (2000, 3000, 400), (2001, 3000, 384), (3900, 4104, 272), (4096, 4096, 256),
         (64, 4096, 2048), (65, 4104, 2064), (40, 4096, 1024), (17, 8200, 512)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_gemm_i8_exact(torch, M, N, K, out):
    """All codes, scales that are powers of two: the fp32 value is exact where the sum stays below 2^24, else one
    rounding of the sum, which float(int) makes."""
    G.say(f"[gemm_i8] {M} x {N} x {K} {out}")
    g = B.gen(M + N + K)
    a, b = B.ints(g, (M, K), -128, 127, torch.int8), B.ints(g, (N, K), -128, 127, torch.int8)
    sa, sb = B.powers(g, (M,)), B.powers(g, (N,))
    c = torch.full((M, N), float("nan"), dtype=dt(torch, out), device="cuda")
    moe.moe_gemm_i8(a, sa, b, sb, None, None, M, N, K, c)
    acc = (a.double() @ b.double().t()).float()
    same_bits(torch, c, (acc * sa[:, None] * sb).to(c.dtype), "c")


def test_gemm_i8_largest_sum(torch):
    """-128 * -128 over the longest row: 2^30, the largest sum there is."""
    K = 65536
    a = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(8, device="cuda")
    c = torch.empty(3, 8, device="cuda")
    moe.moe_gemm_i8(a, one, torch.full((8, K), -128, dtype=torch.int8, device="cuda"), one, None, None, 3, 8, K, c)
    assert bool((c == 2.0 ** 30).all())
    moe.moe_gemm_i8(a, one, torch.full((8, K), 127, dtype=torch.int8, device="cuda"), one, None, None, 3, 8, K, c)
    assert bool((c == -128.0 * 127 * K).all())


@pytest.mark.parametrize("M,N,K", [(1, 264, 512), (20, 72, 2064), (50, 1024, 256), (130, 520, 1024), (600, 776, 528),
                                   (2000, 3000, 400), (3900, 4104, 272)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("bias,add", [(False, False), (True, False), (False, True), (True, True)])
def test_gemm_i8_epilogue(torch, M, N, K, out, bias, add):
    g = B.gen(M * N + K)
    a, b = B.ints(g, (M, K), -127, 127, torch.int8), B.ints(g, (N, K), -127, 127, torch.int8)
    sa, sb = torch.rand(M, generator=g, device="cuda") * 1e-2, torch.rand(N, generator=g, device="cuda") * 1e-2
    sa[0] = float("nan")  # a token whose quantisation met an infinity: its row alone is NaN
    bt = torch.randn(N, generator=g, device="cuda") if bias else None
    at = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16) if add else None
    c = torch.full((M, N), 7.0, dtype=dt(torch, out), device="cuda")
    moe.moe_gemm_i8(a, sa, b, sb, bt, at, M, N, K, c)
    p = a.double() @ b.double().t() * sa.double()[:, None] * sb.double()
    ref, mag = p.clone(), p.abs()
    for t in (bt, at):
        if t is not None:
            ref, mag = ref + t.double(), mag + t.double().abs()
    assert bool(c[0].isnan().all())
    # roundings: the sum to fp32, two scales, two additions, of magnitudes at most `mag`
    within(c[1:], ref[1:], 5.01 * B.U24 * mag[1:] + B.half_step(c.dtype) * ref[1:].abs(), "c")
    if add and out == "bf16":  # the addend may be the output itself
        c2 = at.clone()
        moe.moe_gemm_i8(a, sa, b, sb, bt, c2, M, N, K, c2)
        assert torch.equal(c2[1:], c[1:])


# ------------------------------------------------------------------ grouped products
def layout(torch, g, kind, E, T, k):
    """(off, counts, rows, P) as device tensors, for R = T * k output rows: how a caller may lay out positions."""
    R = T * k
    if kind == "one expert":  # every row on the last expert, the others empty
        ids = torch.full((R,), E - 1, device="cuda")
    elif kind == "few":  # a third of the experts hold rows
        ids = torch.randint(0, max(1, E // 3), (R,), generator=g, device="cuda") * 3 % E
    else:
        w = torch.rand(E, generator=g, device="cuda") ** 3 + 1e-3
        ids = torch.multinomial(w, R, replacement=True, generator=g)
    order = torch.argsort(ids, stable=True).int()
    n = torch.bincount(ids, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    if kind == "padded":  # each expert's run padded to whole 32s with -1, counts given, garbage behind the last
        pad = (n + 31) // 32 * 32
        off[1:] = pad.cumsum(0).int()
        P = int(pad.sum()) + 40
        rows = torch.full((P,), -1, dtype=torch.int32, device="cuda")
        at = 0
        for e in range(E):
            c = int(n[e])
            rows[int(off[e]):int(off[e]) + c] = order[at:at + c]
            at += c
        rows[int(pad.sum()):] = 12345678
        return off, n.int(), rows, P
    off[1:] = n.cumsum(0).int()
    if kind == "contiguous":
        return off, None, None, R
    return off, None, order, R


GROUPED = [("random", 1, 3, 1, 16, 32), ("random", 4, 50, 2, 72, 112), ("contiguous", 8, 77, 3, 264, 144),
           ("padded", 16, 60, 4, 128, 528), ("one expert", 5, 300, 1, 520, 256), ("few", 60, 37, 8, 1416, 1008),
           ("random", 256, 4, 8, 1024, 2048), ("random", 256, 32, 8, 136, 2048), ("padded", 64, 500, 6, 512, 512),
           ("random", 128, 640, 8, 256, 272), ("contiguous", 3, 1000, 2, 328, 784),
           ("one expert", 256, 700, 2, 264, 128),
           ("random", 256, 2100, 8, 512, 128), ("few", 256, 513, 16, 1032, 64), ("contiguous", 256, 1, 1, 8, 16),
           ("random", 32, 2000, 4, 2048, 512), ("padded", 256, 300, 8, 72, 16),
           # the largest tiles: rows that are whole steps and rows that are not
           ("random", 16, 9000, 2, 2048, 256), ("padded", 10, 9001, 2, 2056, 144)]


@pytest.mark.parametrize("kind,E,T,k,N,K", GROUPED)
@pytest.mark.parametrize("typ", ["bf16", "i8"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_grouped_exact(torch, kind, E, T, k, N, K, typ, out):
    """Small integers, exact sums: every named row bit for bit, every other row as it was."""
    G.say(f"[grouped] {kind} E={E} T={T} k={k} N={N} K={K} {typ} {out}")
    g = B.gen(E * 31 + T + N)
    off, counts, rows, P = layout(torch, g, kind, E, T, k)
    R = T * k
    a_div = 1 if kind == "contiguous" else k
    a_rows = (R - 1) // a_div + 1
    i8 = typ == "i8"
    lim = 127 if i8 else 8
    ty = torch.int8 if i8 else torch.bfloat16
    a, b = B.ints(g, (a_rows, K), -lim, lim, ty), B.ints(g, (E, N, K), -lim, lim, ty)
    sa, sb = (B.powers(g, (a_rows,)), B.powers(g, (E, N))) if i8 else (None, None)
    # two rows more than R, and some named by nobody: they keep their bits
    c = torch.full((R + 2, N), -777.25, dtype=dt(torch, out), device="cuda")
    if rows is not None:
        rows[::5] = torch.where(torch.arange(rows[::5].numel(), device="cuda") % 2 == 0, -1, R).int()
    if i8:
        moe.moe_grouped_gemm_i8(a, sa, b, sb, off, counts, rows, a_div, P, R, E, N, K, c)
    else:
        moe.moe_grouped_gemm(a, b, off, counts, rows, a_div, P, R, E, N, K, c)
    ref = torch.full_like(c, -777.25)
    named = B.grouped_positions(off.tolist(), None if counts is None else counts.tolist(),
                                None if rows is None else rows.tolist(), P, R)
    of = {}
    for e, i in named:
        of.setdefault(e, []).append(i)
    for e, ids in of.items():
        t = torch.tensor(ids, device="cuda")
        v = (a[t // a_div].double() @ b[e].double().t()).float()
        ref[t] = (v * sa[t // a_div][:, None] * sb[e] if i8 else v).to(c.dtype)
    same_bits(torch, c, ref, "c")


# every tile with rows of whole steps and without, with weights that pass the caches by and that do not
@pytest.mark.parametrize("kind,E,T,k,N,K", [("random", 64, 900, 4, 520, 384), ("random", 256, 12, 8, 2048, 512),
                                            ("few", 256, 16, 8, 4096, 272), ("random", 256, 32, 8, 1024, 1024),
                                            ("padded", 256, 300, 8, 1032, 1040), ("random", 256, 500, 8, 1024, 1024),
                                            ("random", 256, 1000, 8, 1024, 1024)])
@pytest.mark.parametrize("typ", ["bf16", "i8"])
def test_grouped_weight_streams(torch, kind, E, T, k, N, K, typ):
    test_grouped_exact(torch, kind, E, T, k, N, K, typ, "bf16")


@pytest.mark.parametrize("kind,E,T,k,N,K", [GROUPED[i] for i in (1, 5, 7, 9, 15)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_grouped_general_values(torch, kind, E, T, k, N, K, out):
    g = B.gen(E + T + K)
    off, counts, rows, P = layout(torch, g, kind, E, T, k)
    R, a_div = T * k, k
    a = torch.randn((R - 1) // a_div + 1, K, generator=g, device="cuda").to(torch.bfloat16)
    b = torch.randn(E, N, K, generator=g, device="cuda").to(torch.bfloat16)
    c = torch.full((R, N), float("nan"), dtype=dt(torch, out), device="cuda")
    moe.moe_grouped_gemm(a, b, off, counts, rows, a_div, P, R, E, N, K, c)
    assert not bool(c.isnan().any())
    for e in range(E):
        t = rows[int(off[e]):int(off[e + 1])].long()
        if t.numel():
            x, w = a[t // a_div].double(), b[e].double()
            ref, mag = x @ w.t(), x.abs() @ w.abs().t()
            # products are exact in fp32; each of the K additions rounds by at most a step of the running magnitude
            within(c[t], ref, K * 2 * B.U24 * mag + B.half_step(c.dtype) * ref.abs(), f"expert {e}")


def test_grouped_nonfinite_rows_stay_apart(torch):
    """An infinity or a NaN in one token's row reaches that token's outputs only, and one in an expert's weights
    that expert's rows only (row tails past K are zeros on both sides, not other rows' values)."""
    E, N, K = 3, 72, 200
    off = torch.tensor([0, 40, 41, 150], dtype=torch.int32, device="cuda")
    a = torch.ones(150, K, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda")
    a[7, K - 1], a[99, 0], b[1, 5, K - 1] = float("nan"), float("inf"), float("nan")
    c = torch.empty(150, N, device="cuda")
    moe.moe_grouped_gemm(a, b, off, None, None, 1, 150, 150, E, N, K, c)
    ref = torch.full_like(c, float(K))
    ref[7], ref[99], ref[40, 5] = float("nan"), float("inf"), float("nan")
    assert torch.equal(c.isnan(), ref.isnan()) and torch.equal(c.nan_to_num(), ref.nan_to_num())


def test_grouped_offsets_out_of_range_are_clipped(torch):
    """Offsets and counts come from the device: whatever they hold, only positions in [0, P) and rows in [0, R) are
    touched."""
    E, N, K, P = 4, 16, 16, 64
    a = torch.ones(P, K, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(E, N, K, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(P + 8, N, device="cuda")
    off = torch.tensor([-5, 10, 2000000000, -2000000000, 30], dtype=torch.int32, device="cuda")
    for counts in (None, torch.tensor([10, 2000000000, 7, -3], dtype=torch.int32, device="cuda")):
        moe.moe_grouped_gemm(a, b, off, counts, None, 1, P, P, E, N, K, c)
        torch.cuda.synchronize()
        assert bool(((c == 0) | (c == K)).all()) and bool((c[P:] == 0).all())


def test_many_more_positions_than_rows(torch):
    """A million positions for four rows of 16384 columns, the named ones first, inside and last: the tile goes by the
    rows, the item list by the positions (2^23 items of the smallest tile)."""
    P, R, N, K = (1 << 20) + 7, 4, 1 << 14, 16
    g = B.gen(77)
    a, b = B.ints(g, (R, K), -8, 8, torch.bfloat16), B.ints(g, (2, N, K), -8, 8, torch.bfloat16)
    rows = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    for pos, i in ((0, 2), (5, 0), (600_000, 3), (P - 1, 1)):
        rows[pos] = i
    off = torch.tensor([0, 5, P], dtype=torch.int32, device="cuda")
    c = torch.full((R, N), -777.0, device="cuda")
    moe.moe_grouped_gemm(a, b, off, None, rows, 1, P, R, 2, N, K, c)
    ref = torch.stack([a[i].double() @ b[0 if i == 2 else 1].double().t() for i in range(R)]).float()
    same_bits(torch, c, ref, "c")


@pytest.mark.parametrize("rows_of_a", [140_000, 270_000])
def test_large_a_offsets(torch, rows_of_a):
    """A rows beyond 2^31 and beyond 2^32 bytes, gathered and in order."""
    K, N, E, P = 16384, 64, 3, 300
    g = B.gen(rows_of_a)
    a = torch.zeros(rows_of_a, K, dtype=torch.int8, device="cuda")
    a[-P:] = B.ints(g, (P, K), -9, 9, torch.int8)
    sa, sb = torch.ones(rows_of_a, device="cuda"), torch.ones(E, N, device="cuda")
    b = B.ints(g, (E, N, K), -9, 9, torch.int8)
    rows = (torch.randperm(P, generator=g, device="cuda") + rows_of_a - P).int()
    off = torch.tensor([0, 100, 101, P], dtype=torch.int32, device="cuda")
    c = torch.zeros(rows_of_a, N, device="cuda")
    moe.moe_grouped_gemm_i8(a, sa, b, sb, off, None, rows, 1, P, rows_of_a, E, N, K, c)
    for e in range(E):
        t = rows[int(off[e]):int(off[e + 1])].long()
        assert torch.equal(c[t], (a[t].double() @ b[e].double().t()).float())
    assert int(torch.count_nonzero(c[:-P])) == 0


def test_large_offsets(torch):
    """An output and an A operand beyond 2^31 elements: addresses are 64 bits wide."""
    M, N, K = 5, 1 << 20, 16
    E = 140  # 140 * 2^20 * 16 codes: the last expert's weights lie beyond 2^31 bytes
    g = B.gen(3)
    b = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    b[E - 1] = B.ints(g, (N, K), -9, 9, torch.int8)
    sb = torch.ones(E, N, device="cuda")
    a, sa = B.ints(g, (M, K), -9, 9, torch.int8), torch.ones(M, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = M
    big = 2100  # rows of c: the named ones are the last, beyond 2^31 elements
    rows = torch.arange(big - M, big, dtype=torch.int32, device="cuda")
    c = torch.zeros(big, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_gemm_i8(a, sa, b, sb, off, None, rows, big, M, big, E, N, K, c)
    ref = (a[0].double() @ b[E - 1].double().t()).to(torch.bfloat16)
    for i in range(M):
        assert torch.equal(c[big - M + i], ref)
    assert int(torch.count_nonzero(c[:big - M])) == 0

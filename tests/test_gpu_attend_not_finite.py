"""Attention over caches that hold infinities and NaN: what they reach, and what they leave alone."""
import pytest

from tests import attend_ref as A
from tests import gpu_util as G
from tests.test_gpu_attend import Case, within

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


def reference(c, terms):
    """A.attention's values and bounds, the bounds 0 where the value is no number."""
    out, lse, b_out, b_lse = A.attention(c.q, c.k, c.v, c.ks, c.vs, c.pages.clamp(0, c.n_pages - 1), c.q_start, c.kv_len,
                                         c.Hq, c.Hkv, c.D, c.P, c.D ** -0.5, c.window, terms)
    end = int(c.q_start[-1])
    return [x[:end] for x in (out, lse, b_out.nan_to_num(0.0), b_lse.nan_to_num(0.0))]


def check(torch, c, terms):
    """An element whose row sees a value that is no number there is not finite, all others and lse are the reference's."""
    ref, rl, bo, bl = reference(c, terms)
    out, lse = c.run()
    end = int(c.q_start[-1])
    got = out[:end].view(end, c.Hq, c.D)
    lost = ref.isnan()
    assert bool((~got[lost].isfinite()).all())
    within(torch.where(lost, 0.0, got.double()), torch.where(lost, 0.0, ref), bo, "out")
    within(lse[:end], rl, bl, "lse")
    assert bool((out[end:] == -9.5).all()) and bool((lse[end:] == -9.5).all())
    return out, lse


def spot(c, s, key):
    """(page, place) of a sequence's key."""
    return int(c.pages[s, key // c.P]), key % c.P


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("lengths,D,where,window", [
    ([(1, 200), (1, 90)], 128, 5, 0),       # few rows, a wave's second tile behind the key's
    ([(1, 20000)], 64, 10001, 0),           # contexts shared out, in shares of one unit and of three
    ([(3, 20000), (2, 19000)], 256, 0, 0),
    ([(129, 1500), (40, 66)], 64, 3, 0),    # row tiles
    ([(300, 900)], 128, 700, 250)])         # rows before it, rows that see it, rows whose window has left it
def test_value_row_of_nan(torch, kind, lengths, D, where, window):
    """A token whose whole value row is NaN, as the cache holds one that had an infinity in it: lse, which does not
    depend on values, is that of all keys."""
    c = Case(torch, lengths, 4, 2, D, 16, kind, window, seed=21, poison=False)
    for s in range(c.S):
        page, place = spot(c, s, where)
        if kind == "bf16":
            c.v[page, 1, place] = NAN
        else:
            c.v[page, 1, place] = 0
            c.vs[page, 1, place] = NAN
    check(torch, c, 2 if c.T * 2 <= 32 * c.S else 1)


@pytest.mark.parametrize("lengths,D,window,keys", [
    ([(40, 40), (33, 20)], 128, 0, 1),       # the first row sees one key; rows that see none beside it
    ([(1, 1), (1, 90)], 64, 0, 1), ([(5, 200)], 256, 1, 200),  # few rows, with a window of one key
    ([(2, 30000)], 128, 0, 30000), ([(100, 9000)], 64, 0, 9000),  # contexts shared out
    ([(300, 300)], 64, 3, 150)])             # rows that see such keys alone, some of them, none
def test_scores_of_minus_infinity_alone(torch, lengths, D, window, keys):
    """The weights of a row whose scores are all -infinity are 0 / 0: out is NaN, lse -infinity.  Rows that see no key
    are 0."""
    c = Case(torch, lengths, 4, 2, D, 16, "bf16", window, seed=23, poison=False)
    q = c.q.view(c.T, 4, D)
    q[..., 7] = q[..., 7].abs() + 0.5
    at = torch.arange(min(keys, lengths[0][1]), device="cuda")
    c.k[c.pages[0].long()[at // c.P], :, at % c.P, 7] = -INF
    out, lse = check(torch, c, 2 if c.T * 2 <= 32 * c.S else 1)
    ref = reference(c, 1)[0]
    assert bool(ref.isnan().any()) and bool(out[:ref.shape[0]].view(ref.shape)[ref.isnan()].isnan().all())


SPOTS = [
    # lengths, heads, D, window, keys (as many as a sequence has are taken, some of them)
    ([(40, 40), (1, 300), (0, 70)], 4, 2, 64, 0, (0, 5, 39, 290)),       # few rows
    ([(9, 12000)], 2, 1, 128, 0, (3, 6001, 11993, 11999)),               # shared out
    ([(7, 3000), (2, 500)], 8, 2, 256, 40, (470, 2960, 2975, 2999)),
    ([(300, 900), (64, 64)], 4, 2, 64, 0, (7, 62, 601, 640, 899)),       # row tiles
    ([(300, 900)], 4, 2, 128, 130, (480, 500, 600, 601, 897)),
    ([(129, 700), (200, 200)], 2, 1, 256, 0, (11, 190, 580, 699)),
    ([(180, 9000)], 4, 1, 64, 0, (100, 8821, 8990)),                     # row tiles shared out
    ([(257, 257), (300, 431), (64, 64)] * 4, 64, 64, 128, 0, (0, 63, 64, 250, 420)),  # 256 rows a workgroup
    ([(520, 600), (520, 520)] * 2, 64, 64, 128, 70, (0, 100, 111, 300, 519)),
]


@pytest.mark.parametrize("kind,bad", [("bf16", NAN), ("bf16", INF), ("bf16", -INF), ("i8", NAN), ("i8", INF),
                                      ("e4m3", NAN), ("e4m3", "code")])
@pytest.mark.parametrize("lengths,Hq,Hkv,D,window,keys", SPOTS)
def test_values_that_are_no_numbers(torch, lengths, Hq, Hkv, D, window, keys, kind, bad):
    """Single elements (a code or bf16 value) or rows (a scale) of some keys: early ones that all rows see, ones beside
    the diagonal and the window's edge that some see.  What does not see them, or is another channel, keeps its bits."""
    c = Case(torch, lengths, Hq, Hkv, D, 16, kind, window, seed=25, poison=False)
    clean, cl = c.run()
    for s, (n, L) in enumerate(lengths):
        for i, key in enumerate(k for k in keys if k < L):
            page, place = spot(c, s, key)
            head, ch = (i + s) % Hkv, (17 * i + 5) % D
            if kind == "bf16":
                c.v[page, head, place, ch] = bad
            elif bad == "code":
                c.v.view(torch.uint8)[page, head, place, ch] = 0x7f + 0x80 * (i & 1)
            else:
                c.vs[page, head, place] = bad
    out, lse = check(torch, c, 2 if c.T * (Hq // Hkv) <= 32 * c.S else 1)
    lost = reference(c, 1)[0].isnan()
    assert bool(lost.any())
    got, was = (x[:lost.shape[0]].view(lost.shape) for x in (out, clean))
    assert torch.equal(got[~lost].view(torch.int16), was[~lost].view(torch.int16))
    assert torch.equal(lse, cl)


def test_opposite_infinities(torch):
    """Two infinities of opposite signs in a channel: rows that see one hold it, rows that see both are NaN."""
    for lengths, Hq in (([(40, 300)], 1), ([(200, 200)], 4)):
        c = Case(torch, lengths, Hq, 1, 64, 16, "bf16", seed=27, poison=False)
        n, L = lengths[0]
        a, b = L - 30, L - 12
        for key, v in ((a, INF), (b, -INF)):
            page, place = spot(c, 0, key)
            c.v[page, 0, place, 9] = v
        out, _ = c.run()
        x = out[:n].view(n, Hq, 64)[..., 9].float()
        pos = torch.arange(L - n, L, device="cuda")
        assert bool(x[pos < a].isfinite().all()) and bool((x[(pos >= a) & (pos < b)] == INF).all())
        assert bool(x[pos >= b].isnan().all())


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_they_cost_little(torch, kind):
    """A prompt behind a token with a value that is no number is as fast as any, but for the tiles that some of the rows
    see in part; with one in every key it stays within some ten times."""
    c = Case(torch, [(4096, 4096)], 8, 1, 128, 64, kind, seed=29, poison=False)
    ws = c.workspace()

    def time():
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            c.run(workspace=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    clean = time()
    page, place = spot(c, 0, 3)
    if kind == "bf16":
        c.v[page, 0, place, 5] = NAN
    else:
        c.vs[page, 0, place] = NAN
    early = time()
    if kind == "bf16":
        c.v[..., 5] = NAN
    else:
        c.vs.fill_(NAN)
    every = time()
    G.say(f"[not finite] {kind}: clean {clean * 1e3:.0f} us, an early key {early * 1e3:.0f}, every key {every * 1e3:.0f}")
    assert early < 3 * clean and every < 10 * clean

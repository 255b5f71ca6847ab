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

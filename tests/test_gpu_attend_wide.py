"""Attention in workgroups of 256 rows (two groups of waves half a step apart), which large prompts of 128-element heads
over a bf16 cache take, against the 64-bit reference."""
import pytest

from tests import gpu_util as G
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu

D = 128
# Tiles of one, two and three steps, row tiles that end inside a wave or leave waves without rows, tokens whose heads
# lie in two workgroups, single tokens and sequences without rows beside them.
GROUPED = [(1, 1), (33, 33), (64, 64), (65, 65), (0, 40), (128, 128), (129, 129), (257, 257), (300, 900), (1, 500), (2, 0),
           (5, 3), (31, 31), (700, 700), (1000, 1200), (1400, 1400)]
SINGLE = [(760, 900), (1, 1), (33, 33), (65, 65), (129, 129), (257, 257), (300, 900), (512, 512)]
ODD = [(1500, 1600), (1, 70), (900, 900), (905, 1000)]
CASES = [  # lengths, Hq, Hkv, page, window
    (GROUPED, 32, 4, 64, 0), (GROUPED, 32, 4, 16, 50), (SINGLE, 64, 64, 32, 0), (SINGLE, 64, 64, 16, 300),
    (ODD, 40, 8, 128, 0), (ODD, 40, 8, 64, 1), (ODD, 40, 8, 16, 129)]
SPARE = 3  # rows behind the last sequence


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


@pytest.mark.parametrize("lengths,Hq,Hkv,P,window", CASES)
def test_wide(torch, lengths, Hq, Hkv, P, window):
    """Garbage in every slot that no row sees; the same bits again."""
    c = Case(torch, lengths, Hq, Hkv, D, P, "bf16", window, seed=31, spare_rows=SPARE, q_scale=3.0)
    out, lse = c.run()
    c.check(out, lse)
    for _ in range(3):
        again, l2 = c.run()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), l2.view(torch.int32))


@pytest.mark.parametrize("lengths,Hq,Hkv,P", [(GROUPED, 32, 4, 16), (SINGLE, 64, 64, 16)])
def test_wide_pages_that_are_none(torch, lengths, Hq, Hkv, P):
    """Rows that see a key without a page are NaN, all others keep their bits."""
    c = Case(torch, lengths, Hq, Hkv, D, P, "bf16", seed=33, spare_rows=SPARE, poison=False)
    clean, cl = c.run()
    starts = c.q_start.tolist()
    lost = torch.zeros(starts[-1], dtype=torch.bool, device="cuda")
    for s, (n, L) in enumerate(lengths):
        at = L * 2 // 3 // P  # keys P at .. of the sequences that have them
        if n == 0 or L < 60:
            continue
        c.pages[s, at] = -1 if s & 1 else c.n_pages + s
        lost[starts[s] + max(0, at * P - (L - n)):starts[s + 1]] = True
    out, lse = c.run()
    end = starts[-1]
    assert bool(out[:end][lost].isnan().all()) and bool(lse[:end][lost].isnan().all())
    assert torch.equal(out[:end][~lost], clean[:end][~lost]) and torch.equal(lse[:end][~lost], cl[:end][~lost])
    assert bool((out[end:] == -9.5).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_wide_keys_that_are_no_numbers(torch, bad):
    """Rows before such a key keep their bits; a score of -infinity is a weight of 0, one of NaN or infinity makes a row
    NaN."""
    c = Case(torch, GROUPED, 32, 4, D, 16, "bf16", seed=35, spare_rows=SPARE, poison=False)
    c.q.view(c.T, 32, D)[..., 7].abs_().add_(0.25)
    clean, _ = c.run()
    starts = c.q_start.tolist()
    sees = torch.zeros(starts[-1], dtype=torch.bool, device="cuda")
    for s, (n, L) in enumerate(GROUPED):
        if n == 0 or L < 100:
            continue
        key = L - n // 2 - 1
        c.k[int(c.pages[s, key // 16]), 1, key % 16, 7] = bad
        sees[starts[s] + max(0, key - (L - n)):starts[s + 1]] = True
    out, lse = c.run()
    end = starts[-1]
    a, b = (x[:end].view(end, 4, 8, D) for x in (out, clean))
    assert torch.equal(a[:, [0, 2, 3]], b[:, [0, 2, 3]]) and torch.equal(a[~sees], b[~sees])
    if bad == -float("inf"):
        # a weight of 0, as that of a score of -10^28 beside others of some units: the same bits
        c.k.masked_fill_(c.k == bad, -1e30)
        zero, zl = c.run()
        assert torch.equal(out, zero) and torch.equal(lse, zl) and bool(out.isfinite().all())
    else:
        assert bool(a[sees][:, 1].isnan().all())

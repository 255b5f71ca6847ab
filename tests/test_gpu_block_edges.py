"""Calls of the operators around the layer that stand at the edge of what their documentation allows."""
import pytest

from sparse_moe_layer_03_amd import moe
from tests import block_ref as B
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


# off (the last entry ends the last expert's run where no counts are given) and counts of 300 positions: runs that
# begin before the first position, end behind the last one, or lie outside; none names a position twice
RANGES = {
    "begins before": ([-5, 10, 150, 400, 0], [9, 100, 7, 20]),
    "ends behind": ([0, 40, 90, 299, 310], None),
    "before and behind, no counts": ([-70, 33, 200, 260, 1000], None),
    "lowest and highest": ([INT_MIN, 20, INT_MIN, 100, INT_MAX], [INT_MAX, 30, 5, INT_MAX]),
    "negative counts": ([0, 60, 100, 200, 250], [-1, 10, INT_MIN, 60]),
    "lowest as an end": ([40, INT_MIN, 7, INT_MAX, -3], None),
}


@pytest.mark.parametrize("name", list(RANGES))
@pytest.mark.parametrize("typ", ["bf16", "i8"])
def test_runs_are_cut_to_the_positions(torch, name, typ):
    """Expert e owns positions off[e] .. off[e] + n_e - 1, and of them those in [0, P) are computed: each by its own
    row and expert, exactly, and no other row of c changes."""
    G.say(f"[ranges] {name} {typ}")
    off, counts = RANGES[name]
    E, N, K, P = 4, 72, 48, 300
    g = B.gen(P)
    ty, lim = (torch.int8, 100) if typ == "i8" else (torch.bfloat16, 8)
    a, b = B.ints(g, (P, K), -lim, lim, ty), B.ints(g, (E, N, K), -lim, lim, ty)
    perm = torch.randperm(P, generator=g, device="cuda").int()
    i32 = dict(dtype=torch.int32, device="cuda")
    d_off = torch.tensor(off, **i32)
    d_counts = None if counts is None else torch.tensor(counts, **i32)
    for rows in (None, perm):
        c = torch.full((P, N), -777.25, device="cuda")
        if typ == "i8":
            sa, sb = torch.ones(P, device="cuda"), torch.ones(E, N, device="cuda")
            moe.moe_grouped_gemm_i8(a, sa, b, sb, d_off, d_counts, rows, 1, P, P, E, N, K, c)
        else:
            moe.moe_grouped_gemm(a, b, d_off, d_counts, rows, 1, P, P, E, N, K, c)
        ref = torch.full_like(c, -777.25)
        named = set()
        for e in range(E):
            end = off[e + 1] if counts is None else off[e] + counts[e]
            at = list(range(max(off[e], 0), min(end, P)))
            assert not named & set(at)
            named |= set(at)
            if at:
                i = torch.tensor(at, device="cuda") if rows is None else rows[at].long()
                ref[i] = (a[i].double() @ b[e].double().t()).float()
        assert torch.equal(c, ref), (c != ref).nonzero()[:4].tolist()

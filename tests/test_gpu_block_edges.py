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


def test_rows_beyond_one_grid_dimension(torch):
    """More rows than workgroups of four go into the launch's first dimension: norms and 8-bit rows, the last row and
    the rows at the seam compared, one row behind the last left as it was."""
    H, T = 16, (1 << 22) + 5
    g = B.gen(22)
    x = B.ints(g, (T, H), -8, 8, torch.bfloat16)
    q, s = torch.full((T + 1, H), 99, dtype=torch.int8, device="cuda"), torch.full((T + 1,), -1.0, device="cuda")
    moe.moe_quantize_i8(x, T, H, q, s)
    a = B.row_scales(x.double())
    assert bool(((s[:T].double() - a).abs() <= 2 * B.U24 * a).all())
    assert bool(((q[:T].double() - x.double() / a[:, None]).abs() <= 0.5 + 127 * 4 * B.U24).all())
    assert bool((q[T] == 99).all()) and float(s[T]) == -1.0
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    r, u = torch.full((T + 1, H), 77, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    moe.moe_block_norm(x, x, None, None, w, T, H, r, u, None, None)
    assert torch.equal(r[:T], x + x) and bool((r[T] == 77).all())
    _, ref, _, bound = B.block_norm(x, x, None, None, w, 1.0, 1.0, 0.0, 1e-6)
    assert bool(((u.double() - ref).abs() <= bound + B.U8 * ref.abs()).all())


def test_calls_on_two_streams_and_in_two_graphs(torch):
    """Calls share no memory of the library's: two streams at once, and two graphs replayed at once, give the results
    of one call after the other."""
    g = B.gen(5)
    bf, H, N, E, P = torch.bfloat16, 512, 1032, 8, 700
    off = torch.tensor([0, 3, 90, 91, 91, 300, 301, 640, P], dtype=torch.int32, device="cuda")

    def problem():
        r, y, w = (torch.randn(*s, generator=g, device="cuda").to(bf) for s in ((P, H), (P, H), (H,)))
        wq, ws = B.ints(g, (E, N, H), -127, 127, torch.int8), torch.rand(E, N, generator=g, device="cuda")
        wd = torch.randn(E, N, H, generator=g, device="cuda").to(bf)
        out = dict(x=torch.empty_like(r), q=torch.empty(P, H, dtype=torch.int8, device="cuda"),
                   s=torch.empty(P, device="cuda"), c=torch.empty(P, N, dtype=bf, device="cuda"),
                   d=torch.empty(P, N, dtype=bf, device="cuda"), e=torch.empty(P, N, dtype=bf, device="cuda"))

        def run():
            moe.moe_block_norm(r, y, None, None, w, P, H, None, out["x"], out["q"], out["s"])
            moe.moe_grouped_gemm_i8(out["q"], out["s"], wq, ws, off, None, None, 1, P, P, E, N, H, out["c"])
            moe.moe_grouped_gemm(out["x"], wd, off, None, None, 1, P, P, E, N, H, out["d"])
            moe.moe_gemm_i8(out["q"], out["s"], wq[0], ws[0], None, out["c"], P, N, H, out["e"])
        run()
        torch.cuda.synchronize()
        return out, {k: v.clone() for k, v in out.items()}, run
    both = [problem(), problem()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for (_, _, run), st in zip(both, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            run()
        graphs.append(graph)
    for i in range(6):
        for out, _, _ in both:
            for v in out.values():
                v.zero_()
        torch.cuda.synchronize()
        for (_, _, run), st, graph in zip(both, streams, graphs):
            with torch.cuda.stream(st):
                graph.replay() if i & 1 else run()
        torch.cuda.synchronize()
        for out, want, _ in both:
            for k in out:
                assert torch.equal(out[k], want[k]), (i, k)

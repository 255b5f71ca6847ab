"""The operators around the layer as they are used together: the 8-bit layer, the residual block, streams and graphs."""
import numpy as np
import pytest

from sparse_moe_layer_03_amd import moe, synth
from sparse_moe_layer_03_amd.layer import DeviceLayer, PrefillRunner
from tests import block_ref as B
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

SMALL = dict(H=512, E=16, k=4, I=256, bias="normal")


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


def layer(I_s, i8=True, **over):
    wl = synth.Workload("block", T=600, I_s=I_s, **{**SMALL, **over})
    inp = synth.make_inputs(wl, seed=3)
    return inp, DeviceLayer.from_inputs(inp, i8=i8), DeviceLayer.from_inputs(inp)


def product(codes, scale, wq, ws):
    return codes.double() @ wq.double().t() * scale.double()[:, None] * ws.double()


def check_product(got, ref, what):
    """One product of 8-bit rows: exact sum, rounded to fp32, two scales, one rounding to bf16."""
    d = (got.double() - ref).abs()
    assert bool((d <= (4 * B.U24 + B.U8) * ref.abs()).all()), what


def check_codes(q, scale, h, rel, what, factor=None):
    s = B.row_scales(h)
    f = 1.0 if factor is None else factor.double()
    assert bool(((scale.double() - s * f).abs() <= (rel + 4 * B.U24) * s * f + 1e-45).all()), what + " scale"
    v = h / s[:, None]
    assert bool(((q.double() - v).abs() <= 0.5 + 127 * (2 * rel + 4 * B.U24)).all()), what + " codes"


def silu_rel(gu):
    return (float(gu.double().abs().clamp_max(128).max()) + 8) * 2 * B.U24


@pytest.mark.parametrize("I_s", [0, 128])
@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_i8_layer_stages(torch, T, I_s):
    """Every stage of the 8-bit forward against its formula in 64 bits, from the codes the stage before it left."""
    inp, lay, plain = layer(I_s)
    G.say(f"[i8 layer] T={T} I_s={I_s}")
    s, q = lay.shapes, lay.q
    x = G.to_dev_x(inp)[:T].contiguous()
    y = lay.forward(x)
    torch.cuda.synchronize()
    b = lay._i8_buffers(T)
    # the routing is the layer's own
    stages = plain.alloc_stage_buffers(T)
    plain.run_route(x, stages)
    assert torch.equal(b["ids"], stages["ids"]) and torch.equal(b["w"], stages["w"])
    assert torch.equal(lay.forward_ids(T), stages["ids"])
    check_codes(b["xq"], b["xs"], x.double(), 0.0, "x")
    ids = b["ids"].reshape(-1).long()
    tok = torch.arange(T * s.k, device="cuda") // s.k
    gq, gs = q["gu"].view(s.E, 2 * s.I, s.H), q["gu_scale"].view(s.E, 2 * s.I)
    dq, ds = q["down"].view(s.E, s.H, s.I), q["down_scale"].view(s.E, s.H)
    for e in range(s.E):
        a = (ids == e).nonzero().reshape(-1)
        if a.numel():
            check_product(b["gu"][a], product(b["xq"][tok[a]], b["xs"][tok[a]], gq[e], gs[e]), f"gate/up {e}")
            check_product(b["o"][a], product(b["hq"][a], b["hs"][a], dq[e], ds[e]), f"down {e}")
    check_codes(b["hq"], b["hs"], B.swiglu(b["gu"]), silu_rel(b["gu"]), "h")
    o = b["o"].double().view(T, s.k, s.H)
    ref = (o * b["w"].double()[:, :, None]).sum(1)
    mag = (o.abs() * b["w"].double()[:, :, None]).sum(1)
    if I_s:
        check_product(b["s_gu"], product(b["xq"], b["xs"], q["s_gu"], q["s_gu_scale"]), "shared gate/up")
        check_codes(b["s_hq"], b["s_hs"], B.swiglu(b["s_gu"]), silu_rel(b["s_gu"]), "shared h", b["s"])
        sh = product(b["s_hq"], b["s_hs"], q["s_down"], q["s_down_scale"])
        # the combine's sum is rounded to bf16 before the shared term joins it
        tol = B.U8 * ref.abs() * (1 + B.U8) + B.U8 * (ref + sh).abs() + 4 * s.k * B.U24 * mag + 4 * B.U24 * sh.abs()
        ref = ref + sh
    else:
        tol = B.U8 * ref.abs() + 4 * s.k * B.U24 * mag
    assert bool(((y.double() - ref).abs() <= tol * (1 + 2 * B.U8)).all()), "y"


def test_weight_codes(torch):
    """The layer's weight codes are those of moe_quantize_i8 on the bf16 matrices, gate rows before up rows."""
    _, lay, _ = layer(128)
    s, W, q = lay.shapes, lay.w, lay.q
    gu = torch.cat([W["w_gate"], W["w_up"]], dim=1).reshape(-1, s.H)
    check_codes(q["gu"], q["gu_scale"], gu.double(), 0.0, "gate/up")
    check_codes(q["down"], q["down_scale"], W["w_down"].reshape(-1, s.I).double(), 0.0, "down")
    check_codes(q["s_down"], q["s_down_scale"], W["ws_down"].double(), 0.0, "shared down")


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("T", [1, 7, 130])
def test_forward_block(torch, T, i8):
    """A block of the residual stream is the norm followed by the layer: twice in a row, the second block taking the
    first one's output through a norm, a gate and scales."""
    inp, lay, plain = layer(128, i8=i8)
    g = B.gen(T)
    s = lay.shapes
    bf = torch.bfloat16
    w = [(1 + 0.1 * torch.randn(s.H, generator=g, device="cuda")).to(bf) for _ in range(3)]
    gate = torch.rand(s.H, generator=g, device="cuda").to(bf)
    r = G.to_dev_x(inp)[:T].contiguous()
    r0 = r.clone()
    kw = dict(w_post=w[1], gate=gate, r_scale=0.9, y_scale=0.5, eps=1e-5)
    y1 = lay.forward_block(r, None, w[0])
    assert torch.equal(r, r0)
    y2 = lay.forward_block(r, y1, w[2], **kw)
    # the same by hand
    def step(r, y, w_pre, **kw):
        x, ro = torch.empty_like(r), torch.empty_like(r)
        xq, xs = torch.empty(T, s.H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_block_norm(r, y, kw.pop("w_post", None), kw.pop("gate", None), w_pre, T, s.H, ro, x,
                           xq if i8 else None, xs if i8 else None, **kw)
        if not i8:
            return ro, plain.forward(x)
        b = lay._i8_buffers(T)
        b["xq"].copy_(xq), b["xs"].copy_(xs)
        return ro, lay._forward_i8(x, torch.empty_like(x), quantized=True)
    ra, ya = step(r0, None, w[0])
    assert torch.equal(ya, y1)
    rb, yb = step(ra, y1, w[2], **dict(kw))
    assert torch.equal(rb, r) and torch.equal(yb, y2)
    ref, _, br, _ = B.block_norm(r0, y1, w[1], gate, w[2], 0.9, 0.5, 0.0, 1e-5)
    assert bool(((r.double() - ref).abs() <= br + B.U8 * ref.abs()).all())


def test_i8_empty_and_shrinking_batches(torch):
    """No tokens is a no-op, and a smaller batch after a larger one reuses the workspace without a trace of it."""
    inp, lay, _ = layer(128)
    x = G.to_dev_x(inp)
    want = {T: DeviceLayer.from_inputs(inp, i8=True).forward(x[:T].contiguous()) for T in (3, 64)}
    assert lay.forward(x[:0]).shape == (0, SMALL["H"])
    for T in (600, 64, 3, 64):
        y = lay.forward(x[:T].contiguous())
        if T in want:
            assert torch.equal(y, want[T]), T
    r = x[:0].clone()
    assert lay.forward_block(r, None, torch.ones(SMALL["H"], dtype=torch.bfloat16, device="cuda")).shape[0] == 0


def test_i8_refusals(torch):
    inp, lay, _ = layer(0)
    with pytest.raises(ValueError):
        DeviceLayer.from_inputs(inp, fp8=True, i8=True)
    with pytest.raises(ValueError):
        PrefillRunner(lay)


def test_side_stream(torch):
    """The same bits on another stream, given as a stream and as a raw handle, while the default one is busy."""
    inp, lay, _ = layer(128)
    x = G.to_dev_x(inp)[:200].contiguous()
    w = torch.ones(SMALL["H"], dtype=torch.bfloat16, device="cuda")
    y = lay.forward(x)
    r = x.clone()
    z = lay.forward_block(r, y, w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for handle in (st, st.cuda_stream):
        r2, out = x.clone(), torch.zeros_like(y)
        torch.cuda.synchronize()
        junk = torch.randn(4096, 4096, device="cuda")
        junk = junk @ junk
        lay.forward(x, out, stream=handle)
        st.synchronize()
        assert torch.equal(out, y)
        z2 = lay.forward_block(r2, y, w, out=torch.zeros_like(y), stream=handle)
        st.synchronize()
        assert torch.equal(z2, z) and torch.equal(r2, r)
        del junk


def test_weights_are_ready_for_any_stream(torch):
    """The constructor's quantisation has ended when it returns, also behind other work of its stream."""
    wl = synth.Workload("block", T=8, I_s=128, **SMALL)
    inp = synth.make_inputs(wl, seed=4)
    junk = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        junk = junk @ junk * 1e-3
    lay = DeviceLayer.from_inputs(inp, i8=True)
    assert torch.cuda.current_stream().query()
    st = torch.cuda.Stream()
    x = G.to_dev_x(inp).contiguous()
    torch.cuda.synchronize()
    y = lay.forward(x, torch.zeros_like(x), stream=st)
    torch.cuda.synchronize()
    assert torch.equal(y, lay.forward(x))


def test_graph_replays(torch):
    """A captured block replayed with new inputs, eager work between the replays; two graphs of two layers in turn."""
    inp, lay, _ = layer(128)
    other = DeviceLayer.from_inputs(inp, i8=True)
    all_x = G.to_dev_x(inp)
    w = torch.ones(SMALL["H"], dtype=torch.bfloat16, device="cuda")
    T = 70

    def capture(lay):
        r, y, out = (torch.zeros(T, SMALL["H"], dtype=torch.bfloat16, device="cuda") for _ in range(3))
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            lay.forward_block(r, y, w, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            lay.forward_block(r, y, w, out=out)
        return graph, r, y, out
    graphs = [capture(lay), capture(other)]
    eager = DeviceLayer.from_inputs(inp, i8=True)
    for i in range(5):
        graph, r, y, out = graphs[i & 1]
        a, b = all_x[i * 50:i * 50 + T].clone(), all_x[i * 40 + 7:i * 40 + 7 + T].clone()
        r.copy_(a), y.copy_(b)
        graph.replay()
        want = eager.forward_block(a, b, w)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(r, a), f"replay {i}"
        float((want.float() @ want.float().t()).sum())  # the program's own eager work


@pytest.mark.parametrize("T", [1, 33, 1024, 4096])
def test_products_over_align(torch, T):
    """moe_align's outputs passed on as they are, at the full layer's shape: gate/up rows gathered by token, down rows
    by assignment, bf16 and 8-bit, on integers (every element exact)."""
    H, E, k, I = 2048, 256, 8, 512
    g = B.gen(T)
    n = T * k
    score = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    ids = score.topk(k, dim=1).indices.int().contiguous()
    rows = moe.moe_align_max_rows(T, E, k)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, off, srt = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(rows, **i32)
    inv, nt = torch.empty(n, **i32), torch.empty(2, **i32)
    tiles = torch.empty(2 * moe.moe_align_max_tiles(T, E, k), **i32)
    scratch = torch.empty(moe.moe_align_scratch_size(T, E, k), dtype=torch.uint8, device="cuda")
    moe.moe_align(ids, T, E, k, counts, off, srt, inv, tiles, nt, scratch, scratch.numel())
    flat = ids.reshape(-1).long()
    for dtype, lim in ((torch.int8, 100), (torch.bfloat16, 8)):
        for N, K, a_div in ((2 * I, H, k), (H, I, 1)):
            a = B.ints(g, ((n - 1) // a_div + 1, K), -lim, lim, dtype)
            w = B.ints(g, (E, N, K), -lim, lim, dtype)
            c = torch.full((n, N), float("nan"), device="cuda")
            if dtype is torch.int8:
                sa, sb = B.powers(g, (a.shape[0],)), B.powers(g, (E, N))
                moe.moe_grouped_gemm_i8(a, sa, w, sb, off, counts, srt, a_div, rows, n, E, N, K, c)
            else:
                moe.moe_grouped_gemm(a, w, off, counts, srt, a_div, rows, n, E, N, K, c)
            for e in range(E):
                at = (flat == e).nonzero().reshape(-1)
                if at.numel():
                    ref = (a[at // a_div].double() @ w[e].double().t()).float()
                    if dtype is torch.int8:
                        ref = ref * sa[at // a_div][:, None] * sb[e]
                    assert torch.equal(c[at], ref), (dtype, N, e)

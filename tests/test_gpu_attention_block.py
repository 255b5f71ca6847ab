"""The attention half of a block (DeviceAttention) and a whole block, chained on a residual stream, against 64-bit
references; chunks and single tokens, streams, captured steps."""
import math

import numpy as np
import pytest

from sparse_moe_layer_03_amd import moe, synth
from sparse_moe_layer_03_amd.layer import DeviceAttention, DeviceLayer, bf16_to_numpy_bits
from tests import attend_ref as A
from tests import block_ref as B
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, P = 512, 8, 2, 64, 16


@pytest.fixture(scope="module")
def torch():
    return G.torch_cuda()


def weights(torch, seed=0, bias=True):
    g = B.gen(seed, "cpu")

    def bits(*shape, scale):
        return bf16_to_numpy_bits((torch.randn(*shape, generator=g) * scale).to(torch.bfloat16))
    w = {"w_qkv": bits((HQ + 2 * HKV) * D, H, scale=H ** -0.5), "w_o": bits(H, HQ * D, scale=(HQ * D) ** -0.5),
         "q_norm": bits(D, scale=0.2), "k_norm": bits(D, scale=0.2)}
    if bias:
        w["b_qkv"] = torch.randn((HQ + 2 * HKV) * D, generator=g).numpy()
        w["b_o"] = torch.randn(H, generator=g).numpy()
    return w


def attention(torch, cache, seed=0, n_pages=64, window=0, bias=True):
    freq, ms = moe.moe_rope_frequencies(D, 1e4, moe.ROPE_YARN, 4.0, 64)
    return DeviceAttention(weights(torch, seed, bias), HQ, HKV, D, n_pages, P, cache, freq, ms, window=window, w_add=1.0)


class Book:
    """Which pages the sequences own and how long they are, and the device tensors of a step."""

    def __init__(self, torch, n_seq, max_pages, n_pages):
        self.torch = torch
        self.table = torch.randperm(n_pages)[:n_seq * max_pages].view(n_seq, max_pages).int()
        self.len = [0] * n_seq

    def step(self, new):
        torch = self.torch
        pos, slots, start = [], [], [0]
        for s, n in enumerate(new):
            for i in range(self.len[s], self.len[s] + n):
                pos.append(i)
                slots.append(int(self.table[s, i // P]) * P + i % P)
            self.len[s] += n
            start.append(start[-1] + n)
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return t(pos), t(slots), self.table.cuda(), t(start), t(self.len)


def reference(torch, att, x, hist, step, new):
    """[T, H] in float64 from the rows as bf16 products leave them; hist[s]: the sequence's cached k and v so far (as
    the cache holds them)."""
    pos, _, _, start, kv = step
    w = {k: None if v is None else v.double() for k, v in att.w.items()}
    rows = x.double() @ w["w_qkv"].t().contiguous()
    if att.b["b_qkv"] is not None:
        rows = rows + att.b["b_qkv"].double()
    T = x.shape[0]
    q, k, v = rows.split([HQ * D, HKV * D, HKV * D], dim=1)
    q = A.rope(q.view(T, HQ, D), att.w["q_norm"], 1.0, att.eps, pos, att.freq, att.mscale, att.rot, False)[0]
    k = A.rope(k.view(T, HKV, D), att.w["k_norm"], 1.0, att.eps, pos, att.freq, att.mscale, att.rot, False)[0]
    v = v.view(T, HKV, D)
    out = torch.zeros(T, HQ, D, dtype=torch.float64, device="cuda")
    at = 0
    for s, n in enumerate(new):
        if n == 0:
            continue
        hk, hv = hist.get(s, (k[:0], v[:0]))
        hist[s] = hk, hv = torch.cat([hk, k[at:at + n]]), torch.cat([hv, v[at:at + n]])
        L = hk.shape[0]
        i, j = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        seen = (j <= i) & (j > i - att.window if att.window else True)
        for h in range(HQ):
            g = h // (HQ // HKV)
            sc = (q[at:at + n, h] @ hk[:, g].t().contiguous()) * D ** -0.5
            p = torch.softmax(torch.where(seen, sc, -math.inf), -1)
            out[at:at + n, h] = p @ hv[:, g].contiguous()
        at += n
    y = out.view(T, HQ * D) @ w["w_o"].t().contiguous()
    return y if att.b["b_o"] is None else y + att.b["b_o"].double()


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


# The product's rows, q, k, v and attention's output are rounded to bf16 (half a step, 2^-8, each at random: an rms of
# 2^-8 / sqrt 3 / 1.4 at most for a value); scores of some magnitude 3 turn the q and k errors into weights' errors of
# sqrt 2 * 3 * 0.0017 before averaging over keys.  Together below 2^-6.  8-bit keys and values carry the quantisation's
# error besides: rows of normal values up to some 3.5 standard deviations, i8 steps of 3.5 / 127 (rms over sqrt 12:
# 0.8%), e4m3 half steps of 2^-4 at random (3.1 / sqrt 3 / 1.4 = 2.6%), on k through the scores and on v: below 3 times
# these.
BOUND = {"bf16": 2.0 ** -6, "i8": 0.04, "e4m3": 0.1}
STEPS = [[33, 0, 70, 5], [1, 1, 1, 1], [1, 40, 0, 2], [1, 1, 1, 1], [3, 2, 1, 4]]


@pytest.mark.parametrize("cache,window", [("bf16", 0), ("i8", 0), ("e4m3", 0), ("bf16", 20)])
def test_steps(torch, cache, window):
    """Chunks and single tokens of four sequences, step by step over one cache."""
    att = attention(torch, cache, window=window)
    book, hist, g = Book(torch, 4, 10, att.n_pages), {}, B.gen(3)
    for new in STEPS:
        step = book.step(new)
        T = sum(new)
        x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        y = att.forward(x, *step)
        ref = reference(torch, att, x, hist, step, new)
        assert rel(y, ref) < BOUND[cache], (cache, new, rel(y, ref))
        add = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
        # the same step again writes the same slots
        again = att.forward(x, *step, add=add)
        assert rel(again, ref + add.double()) < BOUND[cache]
        assert torch.equal(att.forward(x, *step), y)


def test_chunks_of_one_prompt(torch):
    """A prompt in one chunk, in chunks, and token by token gives the same rows up to roundings."""
    T = 50
    x = torch.randn(T, H, generator=B.gen(8), device="cuda").to(torch.bfloat16)
    rows = []
    for sizes in ([50], [20, 1, 29], [1] * 50):
        att = attention(torch, "bf16")
        book = Book(torch, 1, 8, att.n_pages)
        at, ys = 0, []
        for n in sizes:
            ys.append(att.forward(x[at:at + n], *book.step([n])))
            at += n
        rows.append(torch.cat(ys))
    for other in rows[1:]:
        assert rel(other, rows[0].double()) < BOUND["bf16"]


@pytest.mark.parametrize("i8", [False, True])
def test_blocks_on_a_residual_stream(torch, i8):
    """Two blocks, attention and experts each, chained through their norms: the stream holds every block's output but
    the last, and a row's result does not depend on the other sequences of its batch."""
    wl = synth.Workload("block", T=16, H=H, E=8, k=2, I=128, I_s=128, bias="normal")
    moes = [DeviceLayer.from_inputs(synth.make_inputs(wl, seed=s), i8=i8) for s in (1, 2)]
    atts = [attention(torch, "i8" if i8 else "bf16", seed=s) for s in (5, 6)]
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    g = B.gen(12)
    r0 = torch.randn(24, H, generator=g, device="cuda")

    def run(r, step):
        y, parts = None, []
        for att, layer in zip(atts, moes):
            y = att.forward_block(r, y, one, *step)
            parts.append(y)
            y = layer.forward_block(r, y, one)
            parts.append(y)
        return y, parts
    book = Book(torch, 3, 4, atts[0].n_pages)
    step = book.step([9, 1, 14])
    r = r0.clone()
    y, parts = run(r, step)
    assert bool(y.isfinite().all())
    want = r0.double()
    for p in parts[:-1]:
        want = want + p.double()
    assert bool(((r.double() - want).abs() <= 4 * B.U24 * sum(p.double().abs() for p in parts) + 4 * B.U24 * r0.abs()).all())
    alone = Book(torch, 1, 4, atts[0].n_pages)
    r1 = r0[10:].clone()
    y1, _ = run(r1, alone.step([14]))
    assert rel(y1, y[10:].double()) < 0.05  # tiles and experts' loads differ, and a near tie may choose another expert


def test_padded_batch(torch):
    """Rows of no sequence are finite and their own, whatever the workspace held, so that the experts may follow; the
    other rows are as without them."""
    wl = synth.Workload("block", T=16, H=H, E=8, k=2, I=128, I_s=128, bias="normal")
    layer = DeviceLayer.from_inputs(synth.make_inputs(wl, seed=1))
    att, plain = attention(torch, "i8", seed=5), attention(torch, "i8", seed=5)
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    g = B.gen(33)
    r0 = torch.randn(8, H, generator=g, device="cuda")
    book = Book(torch, 3, 4, att.n_pages)
    pos, slots, table, start, lens = book.step([1, 1, 1])
    pad = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    got = []
    for fill in (0, 255):  # 255: NaN in every type
        att.forward(r0.to(torch.bfloat16), torch.cat([pos, pad]), torch.cat([slots, pad]), table, start, lens)
        att._ws.fill_(fill)
        r = r0.clone()
        y = att.forward_block(r, None, one, torch.cat([pos, pad]), torch.cat([slots, pad]), table, start, lens)
        z = layer.forward_block(r, y, one)
        assert bool(y.isfinite().all()) and bool(z.isfinite().all()) and bool(r.isfinite().all())
        got.append(y)
    assert torch.equal(*got)
    want = plain.forward_block(r0[:3].clone(), None, one, pos, slots, table, start, lens)
    assert rel(got[0][:3], want.double()) < BOUND["i8"]


def test_captured_steps_and_streams(torch):
    """A decode step captured once and replayed over a growing context, eager steps of another size between; the same
    on a stream of its own, whose pool holds what it allocates."""
    S = 3
    att, plain = attention(torch, "e4m3"), attention(torch, "e4m3")
    book, book2 = Book(torch, S, 8, att.n_pages), None
    book2 = Book(torch, S, 8, att.n_pages)
    book2.table = book.table
    g = B.gen(21)
    x0 = torch.randn(60, H, generator=g, device="cuda").to(torch.bfloat16)
    att.forward(x0, *book.step([20, 20, 20]))
    plain.forward(x0, *book2.step([20, 20, 20]))
    x = torch.empty(S, H, dtype=torch.bfloat16, device="cuda")
    fixed = [t.clone() for t in book.step([1, 1, 1])]
    book2.step([1, 1, 1])
    x.copy_(x0[:S])
    y = torch.empty(S, H, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att.forward(x, *fixed, out=y)
    assert att._ws_captured
    graph.replay()
    want = plain.forward(x, *fixed)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    for t in range(4):
        x.copy_(x0[3 * t:3 * t + 3])
        step = book.step([1, 1, 1])
        for a, b in zip(fixed, step):
            a.copy_(b)
        graph.replay()
        want = plain.forward(x, *step)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        # a larger eager call needs a larger workspace: the captured one is kept
        if t == 1:
            other = Book(torch, 1, 20, att.n_pages)
            other.table = torch.arange(att.n_pages - 20, att.n_pages).view(1, 20).int()
            keep = [c.clone() for c in (att.k_cache.view(torch.uint8), att.v_cache.view(torch.uint8))]
            ks = [c.clone() for c in (att.k_scale, att.v_scale)]
            att.forward(torch.randn(300, H, generator=g, device="cuda").to(torch.bfloat16), *other.step([300]))
            att.k_cache.view(torch.uint8).copy_(keep[0]), att.v_cache.view(torch.uint8).copy_(keep[1])
            att.k_scale.copy_(ks[0]), att.v_scale.copy_(ks[1])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    fresh = attention(torch, "bf16")
    b = Book(torch, 1, 8, fresh.n_pages)
    s1 = b.step([30])
    ref = attention(torch, "bf16").forward(x0[:30], *s1)
    torch.cuda.synchronize()
    got = fresh.forward(x0[:30], *s1, stream=st)
    at = got.data_ptr()
    pool = next(s["stream"] for s in torch.cuda.memory_snapshot() if 0 <= at - s["address"] < s["total_size"])
    assert pool == st.cuda_stream
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


def test_refusals(torch):
    att = attention(torch, "bf16")
    book = Book(torch, 2, 4, att.n_pages)
    step = book.step([3, 2])
    x = torch.zeros(5, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x[:, :256], torch.zeros(5, 2 * H, dtype=torch.bfloat16, device="cuda"), x.cpu()):
        with pytest.raises(ValueError):
            att.forward(bad, *step)
    for i, name in enumerate(("pos", "slots", "pages", "q_start", "kv_len")):
        broken = list(step)
        broken[i] = step[i].long()
        with pytest.raises(ValueError, match=f"^{name} is"):
            att.forward(x, *broken)
        broken[i] = torch.cat([step[i], step[i]])
        with pytest.raises(ValueError):
            att.forward_block(x.clone(), None, w, *broken)
    with pytest.raises(ValueError, match="^out has shape"):
        att.forward(x, *step, out=torch.zeros(4, H, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="^cache is"):
        attention(torch, "fp16")
    with pytest.raises(ValueError, match="^w_o has shape"):
        DeviceAttention(dict(weights(torch), w_o=np.zeros((H, 64), np.uint16)), HQ, HKV, D, 4)
    empty = att.forward(x[:0], *book.step([0, 0]))
    assert empty.shape == (0, H)

"""Argument checks of the operators around the layer: refused before anything touches a GPU."""
import os

import pytest

from sparse_moe_layer_03_amd import moe

P = 1 << 12  # an aligned pointer that is never dereferenced
NO_GPU = not os.path.exists("/dev/kfd")


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def call(fn, base, order, **kw):
    a = dict(base)
    a.update(kw)
    assert set(a) == set(order)
    return fn(*[a[n] for n in order])


NORM_ORDER = ("r", "r_type", "y", "w_post", "gate", "gate_rows", "r_scale", "y_scale", "w_pre", "w_add", "eps", "T",
              "H", "r_out", "x", "q", "q_scale", "stream")
NORM = dict(r=P, r_type=0, y=P, w_post=None, gate=None, gate_rows=1, r_scale=1.0, y_scale=1.0, w_pre=P, w_add=0.0,
            eps=1e-6, T=4, H=64, r_out=P, x=P, q=None, q_scale=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(H=24), "SHAPE"),
    (dict(H=16400), "SHAPE"), (dict(r_type=2), "SHAPE"), (dict(eps=-1e-6), "SHAPE"), (dict(eps=float("nan")), "SHAPE"),
    (dict(y=None, w_post=P), "SHAPE"), (dict(y=None, gate=P), "SHAPE"), (dict(gate=P, gate_rows=3), "SHAPE"),
    (dict(q=P), "NULL"), (dict(q_scale=P), "NULL"), (dict(w_pre=None), "NULL"), (dict(x=None), "NULL"),
    (dict(r_out=None, x=None, w_pre=None), "NULL"), (dict(r=None), "NULL"),
    (dict(r=P + 2), "ALIGN"), (dict(y=P + 8), "ALIGN"), (dict(w_pre=P + 8), "ALIGN"), (dict(r_out=P + 4), "ALIGN"),
    (dict(q=P + 8, q_scale=P), "ALIGN"), (dict(q=P, q_scale=P + 4), "ALIGN"), (dict(gate=P + 2), "ALIGN"),
    (dict(T=0, r=None), "OK"),
])
def test_block_norm_refusals(L, kw, status):
    want = getattr(moe, "MOE_" + status if status == "OK" else "MOE_ERR_" + status)
    assert call(L.moe_block_norm, NORM, NORM_ORDER, **kw) == want
    assert status == "OK" or "moe_block_norm" in moe.last_error()


ROWS = dict(x=P, R=4, K=64, q=P, scale=P, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), "SHAPE"), (dict(R=(1 << 28) + 1), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=24), "SHAPE"),
    (dict(K=32784), "SHAPE"), (dict(x=None), "NULL"), (dict(q=None), "NULL"), (dict(scale=None), "NULL"),
    (dict(x=P + 2), "ALIGN"), (dict(q=P + 8), "ALIGN"), (dict(scale=P + 4), "ALIGN"), (dict(R=0, x=None), "OK"),
])
def test_quantize_and_swiglu_refusals(L, kw, status):
    want = getattr(moe, "MOE_" + status if status == "OK" else "MOE_ERR_" + status)
    assert call(L.moe_quantize_i8, ROWS, ("x", "R", "K", "q", "scale", "stream"), **kw) == want
    for gate in (None, P):
        a = dict(ROWS, gate=gate)
        assert call(L.moe_swiglu_i8, a, ("x", "gate", "R", "K", "q", "scale", "stream"), **kw) == want


def test_swiglu_row_gate_alignment(L):
    assert L.moe_swiglu_i8(P, P + 2, 4, 64, P, P, None) == moe.MOE_ERR_ALIGN


GEMM_ORDER = ("a", "a_scale", "b", "b_scale", "bias", "add", "M", "N", "K", "c", "c_type", "stream")
GEMM = dict(a=P, a_scale=P, b=P, b_scale=P, bias=None, add=None, M=4, N=16, K=32, c=P, c_type=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), "SHAPE"), (dict(M=(1 << 28) + 1), "SHAPE"), (dict(N=0), "SHAPE"), (dict(N=12), "SHAPE"),
    (dict(N=(1 << 20) + 8), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=24), "SHAPE"), (dict(K=65552), "SHAPE"),
    (dict(c_type=2), "SHAPE"), (dict(a=None), "NULL"), (dict(a_scale=None), "NULL"), (dict(b=None), "NULL"),
    (dict(b_scale=None), "NULL"), (dict(c=None), "NULL"), (dict(a=P + 8), "ALIGN"), (dict(b_scale=P + 4), "ALIGN"),
    (dict(bias=P + 4), "ALIGN"), (dict(add=P + 2), "ALIGN"), (dict(c=P + 2), "ALIGN"), (dict(M=0, a=None), "OK"),
])
def test_gemm_i8_refusals(L, kw, status):
    want = getattr(moe, "MOE_" + status if status == "OK" else "MOE_ERR_" + status)
    assert call(L.moe_gemm_i8, GEMM, GEMM_ORDER, **kw) == want


GROUP_ORDER = ("off", "counts", "rows", "a_div", "P", "R", "E", "N", "K", "c", "c_type", "stream")
GROUP = dict(off=P, counts=None, rows=None, a_div=1, P=8, R=8, E=4, N=16, K=32, c=P, c_type=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(P=-1), "SHAPE"), (dict(R=-1), "SHAPE"), (dict(P=(1 << 28) + 1), "SHAPE"), (dict(E=0), "SHAPE"),
    (dict(E=257), "SHAPE"), (dict(N=20), "SHAPE"), (dict(K=20), "SHAPE"), (dict(K=65552), "SHAPE"),
    (dict(a_div=0), "SHAPE"), (dict(c_type=-1), "SHAPE"), (dict(off=None), "NULL"), (dict(c=None), "NULL"),
    (dict(off=P + 2), "ALIGN"), (dict(counts=P + 1), "ALIGN"), (dict(rows=P + 2), "ALIGN"), (dict(c=P + 8), "ALIGN"),
    (dict(P=0), "OK"), (dict(R=0), "OK"),
])
def test_grouped_refusals(L, kw, status):
    want = getattr(moe, "MOE_" + status if status == "OK" else "MOE_ERR_" + status)
    assert call(lambda *a: L.moe_grouped_gemm(P, P, *a), GROUP, GROUP_ORDER, **kw) == want
    assert call(lambda *a: L.moe_grouped_gemm_i8(P, P, P, P, *a), GROUP, GROUP_ORDER, **kw) == want


def test_outputs_beyond_the_item_list(L):
    """Positions times columns above 2^37, whether or not the output rows are as many."""
    assert call(L.moe_gemm_i8, GEMM, GEMM_ORDER, M=1 << 28, N=520) == moe.MOE_ERR_SHAPE
    for kw in (dict(P=1 << 28, N=520), dict(P=(1 << 17) + 1, N=1 << 20)):
        assert call(lambda *a: L.moe_grouped_gemm(P, P, *a), GROUP, GROUP_ORDER, **kw) == moe.MOE_ERR_SHAPE
        assert call(lambda *a: L.moe_grouped_gemm_i8(P, P, P, P, *a), GROUP, GROUP_ORDER, **kw) == moe.MOE_ERR_SHAPE


def test_grouped_missing_operands(L):
    tail = [GROUP[n] for n in GROUP_ORDER]
    assert L.moe_grouped_gemm(None, P, *tail) == moe.MOE_ERR_NULL
    assert L.moe_grouped_gemm(P, P + 8, *tail) == moe.MOE_ERR_ALIGN
    for at in range(4):
        ops = [P] * 4
        ops[at] = None
        assert L.moe_grouped_gemm_i8(*ops, *tail) == moe.MOE_ERR_NULL
        ops[at] = P + 4
        assert L.moe_grouped_gemm_i8(*ops, *tail) == moe.MOE_ERR_ALIGN
    # 8 is a fine row length in bf16 and none in 8-bit integers
    tail[GROUP_ORDER.index("K")] = 8
    assert L.moe_grouped_gemm_i8(P, P, P, P, *tail) == moe.MOE_ERR_SHAPE


@pytest.mark.skipif(not NO_GPU, reason="host without a GPU only")
def test_valid_calls_without_gpu_report_arch(L):
    assert call(L.moe_block_norm, NORM, NORM_ORDER) == moe.MOE_ERR_ARCH
    assert L.moe_quantize_i8(P, 4, 64, P, P, None) == moe.MOE_ERR_ARCH
    assert L.moe_swiglu_i8(P, None, 4, 64, P, P, None) == moe.MOE_ERR_ARCH
    assert call(L.moe_gemm_i8, GEMM, GEMM_ORDER) == moe.MOE_ERR_ARCH
    tail = [GROUP[n] for n in GROUP_ORDER]
    assert L.moe_grouped_gemm(P, P, *tail) == moe.MOE_ERR_ARCH
    assert L.moe_grouped_gemm_i8(P, P, P, P, *tail) == moe.MOE_ERR_ARCH


def test_wrappers_refuse_what_pointers_cannot_show():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for args in ((x.float(), 4, 64, q, s), (x, 5, 64, q, s), (x.t(), 4, 64, q, s), (x, 4, 64, q.short(), s),
                 (x, 4, 64, q, s.double())):
        with pytest.raises(ValueError):
            moe.moe_quantize_i8(*args)
    with pytest.raises(ValueError, match="is on cpu"):
        moe.moe_quantize_i8(x, 4, 64, q, s)
    with pytest.raises(ValueError, match="c is torch.float16"):
        moe.moe_gemm_i8(q, s, q, s, None, None, 4, 8, 64, x.half())
    with pytest.raises(ValueError, match="r is torch.float16"):
        moe.moe_block_norm(x.half(), None, None, None, None, 4, 64, x.half(), None, None, None)

"""Argument checks of the operators around attention, refused before anything touches a GPU, and their host arithmetic."""
import math
import os

import pytest
import torch

from sparse_moe_layer_03_amd import moe

P = 1 << 12  # an aligned pointer that is never dereferenced
NO_GPU = not os.path.exists("/dev/kfd")


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def status(name):
    return moe.MOE_OK if name == "OK" else getattr(moe, "MOE_ERR_" + name)


def call(fn, base, kw):
    assert set(kw) <= set(base)
    return fn(*{**base, **kw}.values())


NAN, INF = float("nan"), float("inf")
ROPE = dict(x=P, x_ld=256, w=P, w_add=0.0, eps=1e-6, pos=P, freq=P, mscale=1.0, T=4, heads=2, D=128, rot=64, pairs=0,
            out=P, out_ld=256, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(heads=1025), "SHAPE"),
    (dict(D=0), "SHAPE"), (dict(D=12), "SHAPE"), (dict(D=264, x_ld=528, out_ld=528), "SHAPE"), (dict(rot=-2), "SHAPE"),
    (dict(rot=63), "SHAPE"), (dict(rot=130), "SHAPE"), (dict(pairs=2), "SHAPE"), (dict(eps=-1.0), "SHAPE"),
    (dict(eps=NAN), "SHAPE"), (dict(mscale=INF), "SHAPE"), (dict(mscale=NAN), "SHAPE"), (dict(x_ld=248), "SHAPE"),
    (dict(x_ld=260), "SHAPE"), (dict(out_ld=0), "SHAPE"), (dict(out_ld=264), "SHAPE"), (dict(x_ld=(1 << 32) + 8), "SHAPE"),
    (dict(x=None), "NULL"), (dict(out=None), "NULL"), (dict(pos=None), "NULL"), (dict(freq=None), "NULL"),
    (dict(x=P + 8), "ALIGN"), (dict(out=P + 2), "ALIGN"), (dict(w=P + 8), "ALIGN"), (dict(pos=P + 2), "ALIGN"),
    (dict(freq=P + 4), "ALIGN"), (dict(T=0, x=None, out=None), "OK"),
])
def test_rope_refusals(L, kw, want):
    assert call(L.moe_rope, ROPE, kw) == status(want)
    assert want == "OK" or "moe_rope" in moe.last_error()


WRITE = dict(q=P, q_ld=512, w_q=None, q_out=P, q_out_ld=512, k=P, k_ld=256, w_k=P, v=P, v_ld=256, w_add=0.0, eps=1e-6,
             pos=P, freq=P, mscale=1.0, slots=P, T=4, Hq=4, Hkv=2, D=128, rot=128, pairs=1, type=2, n_pages=8, P=16,
             k_cache=P, v_cache=P, k_scale=P, v_scale=P, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "SHAPE"), (dict(D=20), "SHAPE"), (dict(rot=129), "SHAPE"), (dict(pairs=-1), "SHAPE"),
    (dict(type=1), "SHAPE"), (dict(type=4), "SHAPE"), (dict(Hkv=0), "SHAPE"), (dict(Hq=-1), "SHAPE"),
    (dict(Hq=1025), "SHAPE"), (dict(P=8), "SHAPE"), (dict(P=48), "SHAPE"), (dict(P=2048), "SHAPE"),
    (dict(n_pages=0), "SHAPE"), (dict(n_pages=(1 << 26) + 1), "SHAPE"), (dict(k_ld=248), "SHAPE"),
    (dict(v_ld=252), "SHAPE"), (dict(q_ld=504), "SHAPE"), (dict(q_out_ld=8), "SHAPE"), (dict(q_out_ld=520), "SHAPE"),
    (dict(Hq=0), "SHAPE"), (dict(Hq=0, q=None, q_out=None, w_q=P), "SHAPE"), (dict(type=0), "SHAPE"),
    (dict(q=None), "NULL"), (dict(q_out=None), "NULL"), (dict(k=None), "NULL"), (dict(v=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(k_cache=None), "NULL"), (dict(v_cache=None), "NULL"),
    (dict(k_scale=None), "NULL"), (dict(type=3, v_scale=None), "NULL"), (dict(pos=None), "NULL"),
    (dict(freq=None), "NULL"), (dict(k=P + 8), "ALIGN"), (dict(v_cache=P + 8), "ALIGN"), (dict(slots=P + 2), "ALIGN"),
    (dict(k_scale=P + 2), "ALIGN"), (dict(w_k=P + 2), "ALIGN"), (dict(T=0, k=None, slots=None), "OK"),
])
def test_cache_write_refusals(L, kw, want):
    assert call(L.moe_cache_write, WRITE, kw) == status(want)


READ = dict(k_cache=P, v_cache=P, k_scale=P, v_scale=P, type=3, n_pages=8, P=16, slots=P, n=4, Hkv=2, D=128, k=P, v=P,
            out_type=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), "SHAPE"), (dict(n=(1 << 24) + 1), "SHAPE"), (dict(D=4), "SHAPE"), (dict(type=1), "SHAPE"),
    (dict(P=17), "SHAPE"), (dict(out_type=2), "SHAPE"), (dict(Hkv=2000), "SHAPE"), (dict(type=0), "SHAPE"),
    (dict(slots=None), "NULL"), (dict(k=None), "NULL"), (dict(v_cache=None), "NULL"), (dict(v_scale=None), "NULL"),
    (dict(k=P + 8), "ALIGN"), (dict(slots=P + 1), "ALIGN"), (dict(n=0, slots=None), "OK"),
])
def test_cache_read_refusals(L, kw, want):
    assert call(L.moe_cache_read, READ, kw) == status(want)


ATTEND = dict(q=P, q_ld=512, k_cache=P, v_cache=P, k_scale=None, v_scale=None, type=0, pages=P, q_start=P, kv_len=P, T=8,
              S=2, Hq=4, Hkv=2, D=128, n_pages=8, P=16, max_pages=4, scale=0.1, window=0, out=P, out_ld=512, lse=None,
              workspace=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(S=-1), "SHAPE"), (dict(S=(1 << 21) + 1), "SHAPE"),
    (dict(Hq=5), "SHAPE"), (dict(Hq=0), "SHAPE"), (dict(Hkv=0), "SHAPE"), (dict(D=96), "SHAPE"), (dict(D=512), "SHAPE"),
    (dict(T=1 << 24, Hq=128, q_ld=1 << 14, out_ld=1 << 14), "SHAPE"), (dict(type=1), "SHAPE"), (dict(P=24), "SHAPE"),
    (dict(n_pages=0), "SHAPE"), (dict(max_pages=0), "SHAPE"), (dict(max_pages=(1 << 26) + 1), "SHAPE"),
    (dict(scale=0.0), "SHAPE"), (dict(scale=-1.0), "SHAPE"), (dict(scale=NAN), "SHAPE"), (dict(scale=INF), "SHAPE"),
    (dict(window=-1), "SHAPE"), (dict(q_ld=504), "SHAPE"), (dict(out_ld=516), "SHAPE"), (dict(k_scale=P), "SHAPE"),
    (dict(q=None), "NULL"), (dict(k_cache=None), "NULL"), (dict(pages=None), "NULL"), (dict(q_start=None), "NULL"),
    (dict(kv_len=None), "NULL"), (dict(out=None), "NULL"), (dict(type=2, k_scale=P), "NULL"),
    (dict(max_pages=4096, workspace=None), "NULL"), (dict(max_pages=4096, workspace=P + 8), "ALIGN"),
    (dict(max_pages=4096, ws_bytes=1000), "WORKSPACE"), (dict(q=P + 8), "ALIGN"), (dict(out=P + 4), "ALIGN"),
    (dict(lse=P + 2), "ALIGN"), (dict(pages=P + 2), "ALIGN"), (dict(T=0, q=None), "OK"), (dict(S=0, pages=None), "OK"),
])
def test_attention_refusals(L, kw, want):
    assert call(L.moe_attention, ATTEND, kw) == status(want)


def test_attention_in_place_refusal(L):
    assert call(L.moe_attention, ATTEND, dict(out_ld=520)) == moe.MOE_ERR_SHAPE
    assert "in place" in moe.last_error()


def test_attention_workspace(L):
    """What the query says is enough and one byte less is refused; sizes out of range need nothing."""
    size = moe.moe_attention_workspace_size
    for T, S, Hq, Hkv, D, keys in ((1, 1, 8, 1, 128, 1 << 17), (64, 64, 32, 4, 128, 8192), (40, 1, 4, 4, 256, 4096),
                                   (300, 2, 16, 2, 64, 1 << 15), (5, 5, 1, 1, 64, 1 << 30)):
        n = size(T, S, Hq, Hkv, D, keys)
        assert n > 0
        kw = dict(T=T, S=S, Hq=Hq, Hkv=Hkv, D=D, q_ld=Hq * D, out_ld=Hq * D, P=1024, max_pages=keys // 1024)
        assert call(L.moe_attention, ATTEND, dict(kw, ws_bytes=n - 1)) == moe.MOE_ERR_WORKSPACE
        if NO_GPU:
            assert call(L.moe_attention, ATTEND, dict(kw, ws_bytes=n)) == moe.MOE_ERR_ARCH
    assert size(0, 1, 8, 1, 128, 4096) == size(1, 0, 8, 1, 128, 4096) == size(1, 1, 8, 3, 128, 4096) == 0
    assert size(1, 1, 8, 1, 128, -1) == size(1, 1, 8, 1, 128, (1 << 30) + 1) == 0
    assert size(8192, 1, 32, 4, 128, 8192) == 0  # enough row tiles for every CU


GEMM = dict(a=P, b=P, bias=None, act=0, add=None, M=4, N=16, K=32, c=P, c_type=0, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), "SHAPE"), (dict(M=(1 << 28) + 1), "SHAPE"), (dict(N=0), "SHAPE"), (dict(N=12), "SHAPE"),
    (dict(N=(1 << 20) + 8), "SHAPE"), (dict(K=0), "SHAPE"), (dict(K=20), "SHAPE"), (dict(K=65544), "SHAPE"),
    (dict(M=1 << 28, N=520), "SHAPE"), (dict(c_type=2), "SHAPE"), (dict(act=3), "SHAPE"), (dict(act=-1), "SHAPE"),
    (dict(a=None), "NULL"), (dict(b=None), "NULL"), (dict(c=None), "NULL"), (dict(a=P + 8), "ALIGN"),
    (dict(b=P + 2), "ALIGN"), (dict(bias=P + 4), "ALIGN"), (dict(add=P + 2), "ALIGN"), (dict(c=P + 8), "ALIGN"),
    (dict(M=0, a=None), "OK"),
])
def test_gemm_refusals(L, kw, want):
    assert call(L.moe_gemm, GEMM, kw) == status(want)


@pytest.mark.skipif(not NO_GPU, reason="host without a GPU only")
def test_valid_calls_without_gpu_report_arch(L):
    for fn, base in ((L.moe_rope, ROPE), (L.moe_cache_write, WRITE), (L.moe_cache_read, READ), (L.moe_attention, ATTEND),
                     (L.moe_gemm, GEMM)):
        assert call(fn, base, {}) == moe.MOE_ERR_ARCH
    assert call(L.moe_rope, ROPE, dict(rot=0, pos=None, freq=None)) == moe.MOE_ERR_ARCH
    assert call(L.moe_cache_write, WRITE, dict(Hq=0, q=None, q_out=None, q_ld=0, q_out_ld=0)) == moe.MOE_ERR_ARCH


# ------------------------------------------------------------------ frequencies
def test_frequencies():
    rot, base = 64, 1e4
    plain, ms = moe.moe_rope_frequencies(rot, base)
    want = torch.tensor([base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)], dtype=torch.float64)
    assert ms == 1.0 and torch.allclose(plain, want, rtol=1e-14, atol=0)
    lin, ms = moe.moe_rope_frequencies(rot, base, moe.ROPE_LINEAR, 8.0)
    assert ms == 1.0 and torch.allclose(lin, want / 8, rtol=1e-14, atol=0)
    ntk, ms = moe.moe_rope_frequencies(rot, base, moe.ROPE_NTK, 8.0)
    # the fastest pair as it was, the slowest interpolated by the whole factor
    assert ms == 1.0 and float(ntk[0]) == float(plain[0]) and abs(float(ntk[-1] / plain[-1]) * 8 - 1) < 1e-12
    yarn, ms = moe.moe_rope_frequencies(rot, base, moe.ROPE_YARN, 8.0, 4096)
    assert abs(ms - (0.1 * math.log(8) + 1)) < 1e-7
    turns = want * 4096
    r = yarn / want
    # two pairs' width around the bounds is the ramp's own rounding to whole pairs
    step = base ** (2 / rot)
    assert bool((r[turns > 32 * step] == 1).all()) and bool(((r[turns < 1 / step] * 8 - 1).abs() < 1e-12).all())
    assert bool((r[:-1] >= r[1:]).all())


@pytest.mark.parametrize("args", [(0, 1e4), (3, 1e4), (258, 1e4), (64, 1.0), (64, NAN), (64, INF), (64, 1e4, 4),
                                  (64, 1e4, -1), (64, 1e4, 1, 0.5), (64, 1e4, 2, NAN), (2, 1e4, 2, 2.0),
                                  (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, INF, 4096.0)])
def test_frequency_refusals(args):
    with pytest.raises(moe.MoEError):
        moe.moe_rope_frequencies(*args)


# ------------------------------------------------------------------ the Python entry points
class Reached(Exception):
    """A call has passed its checks and asks for the library."""


@pytest.fixture
def no_gpu_needed(monkeypatch):
    def lib():
        raise Reached
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(moe, "_device", lambda: 0)
    monkeypatch.setattr(moe, "lib", lib)


BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32
T, HQ, HKV, D, NP, PG, S, MP = 4, 4, 2, 64, 3, 16, 2, 2


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


CACHE = dict(k_cache=z(NP, HKV, PG, D, dtype=torch.int8), v_cache=z(NP, HKV, PG, D, dtype=torch.int8),
             k_scale=z(NP, HKV, PG, dtype=F32), v_scale=z(NP, HKV, PG, dtype=F32))
ANGLES = dict(pos=z(T, dtype=I32), freq=z(D // 2, dtype=torch.float64))
CALLS = {
    "moe_rope": dict(x=z(T, HQ * D), w_norm=z(D), **ANGLES, T=T, heads=HQ, D=D, rot=D, pairs=0, out=z(T, HQ * D)),
    "moe_cache_write": dict(q=z(T, HQ * D), w_q=z(D), q_out=z(T, HQ * D), k=z(T, HKV * D), w_k=z(D), v=z(T, HKV * D),
                            **ANGLES, slots=z(T, dtype=I32), T=T, Hq=HQ, Hkv=HKV, D=D, rot=D, pairs=0, **CACHE,
                            n_pages=NP, P=PG),
    "moe_cache_read": dict(**CACHE, slots=z(T, dtype=I32), n=T, Hkv=HKV, D=D, n_pages=NP, P=PG, k=z(T, HKV, D),
                           v=z(T, HKV, D)),
    "moe_attention": dict(q=z(T, HQ * D), **CACHE, pages=z(S, MP, dtype=I32), q_start=z(S + 1, dtype=I32),
                          kv_len=z(S, dtype=I32), T=T, S=S, Hq=HQ, Hkv=HKV, D=D, n_pages=NP, P=PG, max_pages=MP,
                          out=z(T, HQ * D), workspace=z(64, dtype=torch.uint8), lse=z(T, HQ, dtype=F32)),
    "moe_gemm": dict(a=z(T, D), b=z(8, D), bias=z(8, dtype=F32), add=z(T, 8), M=T, N=8, K=D, c=z(T, 8)),
}
TENSORS = [(f, n) for f, a in CALLS.items() for n, t in a.items() if torch.is_tensor(t)]


@pytest.mark.parametrize("fn,name", TENSORS)
def test_wrong_tensors(no_gpu_needed, fn, name):
    """Each tensor too short, of another type, or not in order is refused by its name."""
    args, t = CALLS[fn], CALLS[fn][name]
    with pytest.raises(Reached):
        getattr(moe, fn)(**args)
    bad = [t.flatten()[:-1], t.double() if t.dtype != torch.float64 else t.float()]
    if t.dim() > 1:
        bad.append(t.transpose(0, -1))
    for b in bad if name != "workspace" else []:
        with pytest.raises(ValueError, match=f"^{name} |^v_cache |^v "):
            getattr(moe, fn)(**{**args, name: b})


def test_strided_rows(no_gpu_needed):
    """q, k, v and outputs may be columns of wider rows, heads apart or not; a table may not."""
    wide = z(T, 3 * HQ * D)
    for fn, names in (("moe_rope", ("x", "out")), ("moe_attention", ("q", "out")), ("moe_cache_write", ("q", "q_out"))):
        for name in names:
            for t in (wide[:, 8:8 + HQ * D], z(T, HQ, D), z(T + 2, HQ * D), z(2 * T, HQ * D)[::2]):
                with pytest.raises(Reached):
                    getattr(moe, fn)(**{**CALLS[fn], name: t})
            for t in (wide[:, ::3], z(HQ * D, T).t(), z(T, HQ * D + 8)):
                with pytest.raises(ValueError, match=f"^{name} "):
                    getattr(moe, fn)(**{**CALLS[fn], name: t})
    assert moe._rows("q", wide[:, 8:8 + HQ * D], T, HQ * D)[1] == 3 * HQ * D
    assert moe._rows("q", wide[:1, 8:8 + HQ * D], 1, HQ * D)[1] == HQ * D
    with pytest.raises(ValueError, match="^pages "):
        moe.moe_attention(**{**CALLS["moe_attention"], "pages": z(S, 2 * MP, dtype=I32)[:, ::2]})


def test_cache_types(no_gpu_needed):
    for dt in (torch.float16, torch.uint8, torch.float8_e5m2):
        with pytest.raises(ValueError, match="^k_cache is "):
            moe.moe_cache_read(**{**CALLS["moe_cache_read"], "k_cache": z(NP, HKV, PG, D).to(dt)})
    with pytest.raises(ValueError, match="^v_cache is "):
        moe.moe_cache_read(**{**CALLS["moe_cache_read"], "v_cache": z(NP, HKV, PG, D)})
    with pytest.raises(ValueError, match="^k_cache must be a tensor"):
        moe.moe_cache_read(**{**CALLS["moe_cache_read"], "k_cache": P})
    with pytest.raises(ValueError, match="^workspace must be a tensor"):
        moe.moe_attention(**{**CALLS["moe_attention"], "workspace": P})


def test_another_device(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1)
    monkeypatch.setattr(moe, "_device", lambda: 0)
    for fn in CALLS:
        with pytest.raises(ValueError, match="is on GPU 1; the current one is 0"):
            getattr(moe, fn)(**CALLS[fn])

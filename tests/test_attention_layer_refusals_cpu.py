"""DeviceAttention refuses what its kernels do not take when it is built, or before anything of a step is enqueued."""
import contextlib

import numpy as np
import pytest
import torch

from sparse_moe_layer_03_amd import moe
from sparse_moe_layer_03_amd.layer import DeviceAttention

H, HQ, HKV, D = 64, 4, 2, 64
BF = torch.bfloat16


@pytest.fixture
def no_gpu_needed(monkeypatch):
    """Tensors of the host pass for those of the current GPU."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(moe, "_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: type("S", (), {"synchronize": lambda s: None})())


def build(Hq=HQ, Hkv=HKV, D=D, H=H, n_pages=4, drop=(), **kw):
    w = {"w_qkv": np.zeros(((Hq + 2 * Hkv) * D, H), np.uint16), "w_o": np.zeros((H, Hq * D), np.uint16)}
    for key in drop:
        del w[key]
    return DeviceAttention(w, Hq, Hkv, D, n_pages, device="cpu", **kw)


def turns(n, dtype=torch.float64):
    return torch.zeros(n, dtype=dtype)


@pytest.mark.parametrize("kw", [
    {}, dict(cache="i8", page=16, window=7, scale=0.3), dict(cache="e4m3", freq=turns(D // 2)), dict(freq=turns(8)),
    dict(Hq=6, Hkv=3, D=128), dict(Hq=1, Hkv=1, D=256, pairs=moe.ROPE_INTERLEAVED, page=1024)])
def test_built(no_gpu_needed, kw):
    att = build(**kw)
    assert att.k_cache.shape == (4, att.Hkv, att.page, att.D)


@pytest.mark.parametrize("kw,match", [
    (dict(D=96), "D=96"), (dict(D=8), "D=8"), (dict(D=512), "D=512"), (dict(Hq=6, Hkv=4), "Hq=6"),
    (dict(Hq=0), "Hq=0"), (dict(Hkv=0, Hq=4), "Hkv=0"), (dict(page=24), "P=24"), (dict(page=8), "P=8"),
    (dict(page=2048), "P=2048"), (dict(n_pages=0), "n_pages=0"), (dict(n_pages=(1 << 24) + 1), "n_pages="),
    (dict(window=-1), "window"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"),
    (dict(scale=float("nan")), "scale"), (dict(eps=-1e-6), "eps"), (dict(mscale=float("inf")), "mscale"),
    (dict(pairs=2), "pairs=2"), (dict(H=20), "K=20"), (dict(H=4), "K=4"),
    (dict(freq=turns(D)), "rot=128"), (dict(freq=turns(32, torch.float32)), "freq"),
    (dict(freq=turns(32).view(2, 16)), "freq"), (dict(drop=("w_qkv",)), "w_qkv"), (dict(drop=("w_o",)), "w_o"),
])
def test_not_built(no_gpu_needed, kw, match):
    with pytest.raises((ValueError, moe.MoEError), match=match):
        build(**kw)


I32 = torch.int32
STEP = dict(pos=torch.zeros(6, dtype=I32), slots=torch.zeros(6, dtype=I32), pages=torch.zeros(2, 3, dtype=I32),
            q_start=torch.zeros(3, dtype=I32), kv_len=torch.zeros(2, dtype=I32))


class Enqueued(Exception):
    """A call has passed all checks."""


@pytest.fixture
def att(no_gpu_needed, monkeypatch):
    def enqueued(*a, **kw):
        raise Enqueued
    for name in ("moe_gemm", "moe_block_norm", "moe_cache_write", "moe_attention"):
        monkeypatch.setattr(moe, name, enqueued)
    monkeypatch.setattr(DeviceAttention, "_note_stream", lambda self, stream: None)
    return build(freq=turns(D // 2))


def calls(att, **kw):
    """The two ways to a step."""
    x, r, w = torch.zeros(6, H, dtype=BF), torch.zeros(6, H), torch.zeros(H, dtype=BF)
    step = {**STEP, **kw}
    return (lambda: att.forward(x, **step)), (lambda: att.forward_block(r, x, w, **step))


def test_step_passes(att):
    for call in calls(att) + calls(att, pages=torch.zeros(0, 3, dtype=I32), q_start=torch.zeros(1, dtype=I32),
                                   kv_len=torch.zeros(0, dtype=I32)):
        with pytest.raises(Enqueued):
            call()


@pytest.mark.parametrize("kw,match", [
    (dict(pos=None), "pos is missing"), (dict(slots=None), "slots is missing"), (dict(pages=None), "pages is missing"),
    (dict(q_start=None), "q_start is missing"), (dict(kv_len=None), "kv_len is missing"),
    (dict(pages=torch.zeros(2, 0, dtype=I32)), "pages has no columns"),
    (dict(pages=torch.zeros(6, dtype=I32)), "pages has shape"), (dict(pages=torch.tensor(0, dtype=I32)), "pages has shape"),
    (dict(kv_len=torch.tensor(2, dtype=I32)), "pages has shape|kv_len has shape"),
    # 2^24 + 64 pages of 64 tokens a sequence; without memory of their own
    (dict(pages=torch.zeros(1, 1, dtype=I32).expand(2, (1 << 24) + 64)), "pages"),
])
def test_step_refused(att, kw, match):
    for call in calls(att, **kw):
        with pytest.raises((ValueError, moe.MoEError), match=match):
            call()


def test_step_of_too_many(att, monkeypatch):
    """What the size query refuses: sequences times key heads above 2^22, longer tables, more rows than it takes."""
    monkeypatch.setattr(DeviceAttention, "_check_tensors", lambda self, *t: None)

    class Like:
        def __init__(self, *shape):
            self.shape = shape

        def dim(self):
            return len(self.shape)
    S = (1 << 21) + 1
    for kw in (dict(kv_len=Like(S), pages=Like(S, 3)), dict(pages=Like(2, (1 << 24) + 1))):
        for call in calls(att, **kw):
            with pytest.raises(moe.MoEError):
                call()


def test_scales_under_another_default_type(no_gpu_needed):
    was = torch.get_default_dtype()
    torch.set_default_dtype(BF)
    try:
        att = build(cache="i8")
    finally:
        torch.set_default_dtype(was)
    assert att.k_scale.dtype is att.v_scale.dtype is torch.float32

"""Device-resident MoE layer: weights and workspace in HBM, calls into libmoe355.

PyTorch is used for device memory and streams only; every step of the layer
runs in the HIP kernels behind ``moe.py``.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import Dict, Optional

import numpy as np

from . import moe

BF16_KEYS = ("w_router", "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down", "w_sg")
FP8_KEYS = ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")


def to_device_bf16(a: Optional[np.ndarray], device):
    """uint16 bf16 bit patterns -> torch.bfloat16 tensor on ``device`` (bits unchanged)."""
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16))
    return t.to(device).view(torch.bfloat16)


def bf16_to_numpy_bits(t) -> np.ndarray:
    import torch
    return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)


@dataclass
class Shapes:
    H: int
    E: int
    k: int
    I: int
    I_s: int


class DeviceLayer:
    """The layer's weights on one GPU plus a reusable workspace.

    ``fp8``: also upload the FP8 expert weights (``<key>_fp8`` codes and
    ``<key>_scale`` row scales of ``weights``); ``forward`` then calls
    ``moe_forward_fp8``.  ``q4``: likewise the 4-bit weights (``<key>_q4``
    codes and ``<key>_q4scale`` fp16 group scales) and ``moe_forward_q4``.
    ``i8``: the expert weights are quantised on the GPU to 8-bit integers with
    a scale per output row, and ``forward`` runs the experts in 8-bit integers
    with a scale per token, by the grouped products (see ``_forward_i8``).

    Calls of one layer share its workspace: one on another stream than the
    last has to be ordered behind it, and so have replays of captured calls.
    A workspace that a captured call used is kept as long as the layer.  What
    a call allocates belongs to the pool of the stream it is given (the
    current one by default).
    """

    def __init__(self, weights: Dict[str, np.ndarray], k: int, device="cuda:0", fp8: bool = False,
                 q4: bool = False, i8: bool = False):
        import torch
        if fp8 + q4 + i8 > 1:
            raise ValueError("choose one of fp8, q4 and i8")
        self.device = torch.device(device)
        self.fp8 = fp8
        self.q4 = q4
        self.i8 = i8
        self.w = {key: to_device_bf16(weights.get(key), self.device) for key in BF16_KEYS}
        self.q = {}
        if fp8:
            for key in FP8_KEYS:
                c, sc = weights.get(key + "_fp8"), weights.get(key + "_scale")
                self.q[key] = None if c is None else torch.from_numpy(np.ascontiguousarray(c, np.uint8)).to(self.device)
                self.q[key + "_scale"] = (None if sc is None else
                                          torch.from_numpy(np.ascontiguousarray(sc, np.float32)).to(self.device))
        if q4:
            for key in FP8_KEYS:
                c, sc = weights.get(key + "_q4"), weights.get(key + "_q4scale")
                self.q[key + "_q4"] = (None if c is None else
                                       torch.from_numpy(np.ascontiguousarray(c, np.uint8)).to(self.device))
                self.q[key + "_q4scale"] = (None if sc is None else torch.from_numpy(
                    np.ascontiguousarray(sc, np.uint16).view(np.int16)).to(self.device))
        b = weights.get("bias")
        self.bias = None if b is None else torch.from_numpy(np.ascontiguousarray(b, np.float32)).to(self.device)
        E, I, H = weights["w_gate"].shape
        I_s = 0 if weights.get("ws_gate") is None else weights["ws_gate"].shape[0]
        self.shapes = Shapes(H=H, E=E, k=k, I=I, I_s=I_s)
        self._ws = None
        self._ws_bytes = 0
        self._ws_streams = []  # handles of the streams the current workspace has been used on since it was allocated
        self._ws_captured = False  # whether a captured call has used it
        self._ws_kept = []  # earlier workspaces that graphs still write on replay
        self._i8_views = None  # (workspace address, T, the views forward uses) of 8-bit layers
        if i8:
            self._quantize_weights()

    @classmethod
    def from_inputs(cls, inp, device="cuda:0", fp8: bool = False, q4: bool = False, i8: bool = False):
        return cls(inp, inp["wl"].k, device, fp8=fp8, q4=q4, i8=i8)

    def _quantize_weights(self):
        """8-bit codes and row scales of the expert weights, gate and up rows of an expert one after the other."""
        import torch
        s, W = self.shapes, self.w

        def rows(a, n, K):
            q = torch.empty((n, K), dtype=torch.int8, device=self.device)
            sc = torch.empty(n, dtype=torch.float32, device=self.device)
            moe.moe_quantize_i8(a, n, K, q, sc)
            return q, sc

        def stacked(gate, up, E, I, K):
            (g, gs), (u, us) = rows(gate, E * I, K), rows(up, E * I, K)
            return (torch.cat([g.view(E, I, K), u.view(E, I, K)], dim=1).view(E * 2 * I, K),
                    torch.cat([gs.view(E, I), us.view(E, I)], dim=1).reshape(-1))
        with torch.cuda.device(self.device):
            self.q["gu"], self.q["gu_scale"] = stacked(W["w_gate"], W["w_up"], s.E, s.I, s.H)
            self.q["down"], self.q["down_scale"] = rows(W["w_down"], s.E * s.H, s.I)
            if s.I_s:
                self.q["s_gu"], self.q["s_gu_scale"] = stacked(W["ws_gate"], W["ws_up"], 1, s.I_s, s.H)
                self.q["s_down"], self.q["s_down_scale"] = rows(W["ws_down"], s.H, s.I_s)
            # as the grouped products take them
            self._i8_experts = (self.q["gu"].view(s.E, 2 * s.I, s.H), self.q["gu_scale"].view(s.E, 2 * s.I),
                                self.q["down"].view(s.E, s.H, s.I), self.q["down_scale"].view(s.E, s.H))
            # the first forward may run on any stream
            torch.cuda.current_stream().synchronize()

    def workspace(self, T: int):
        s = self.shapes
        need = moe.moe_workspace_size(T, s.H, s.E, s.k, s.I, s.I_s)
        if need == 0 and T > 0:
            raise moe.MoEError(moe.MOE_ERR_SHAPE, "unsupported shapes")
        return self._reserve(need)

    def _reserve(self, need: int):
        import torch
        if self._ws is None or self._ws_bytes < need:
            if self._ws is not None:
                # the caching allocator tracks only the allocating stream: keep the old buffer from being
                # handed out again before work already enqueued on the other streams that used it is done
                for st in self._ws_streams:
                    self._ws.record_stream(torch.cuda.ExternalStream(st, device=self.device))
                if self._ws_captured:
                    self._ws_kept.append(self._ws)
            self._ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
            self._ws_bytes = max(need, 256)
            self._ws_streams = []
            self._ws_captured = False
        return self._ws, self._ws_bytes

    def _pool(self, stream):
        """The context in which memory for work on ``stream`` (None, a torch stream or a raw handle) is allocated: a
        block of the current stream's pool may still be in use by work pending there."""
        import torch
        if stream is None:
            return contextlib.nullcontext()
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device) if isinstance(stream, int)
                                 else stream)

    def _output(self, T: int, stream):
        """[T, H] for the kernels on ``stream`` to write; once dropped, reused only behind the current stream's work at
        that time, which may read it."""
        import torch
        with self._pool(stream):
            y = torch.empty((T, self.shapes.H), dtype=torch.bfloat16, device=self.device)
        if stream is not None:
            y.record_stream(torch.cuda.current_stream(self.device))
        return y

    def _note_stream(self, stream):
        """Remember what the workspace is used by: the stream (None, a torch stream or a raw handle), a capture."""
        import torch
        st = moe._stream(stream)
        if st not in self._ws_streams:
            self._ws_streams.append(st)
        if not self._ws_captured:
            with self._pool(stream):
                self._ws_captured = torch.cuda.is_current_stream_capturing()

    def _check_tensors(self, *tensors):
        """Refuses, before anything is enqueued, tensors given as (name, tensor, shapes, dtypes) that the kernels would
        misread or write astray: another shape, type, order or device than the layer's, which is the current one."""
        at = self.w["w_router"].get_device()
        for name, t, shapes, dtypes in tensors:
            if t.dtype in dtypes and t.shape in shapes and t.is_contiguous() and t.get_device() == at >= 0:
                continue
            if t.dtype not in dtypes:
                raise ValueError(f"{name} is {t.dtype}; expected {' or '.join(map(str, dtypes))}")
            if t.shape not in shapes:
                raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {' or '.join(map(str, shapes))}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            raise ValueError(f"{name} is on {t.device}, the layer on {self.w['w_router'].device}")
        if at != moe._device():
            raise ValueError(f"the layer is on GPU {at}; the current one is {moe._device()}")

    def forward(self, x, y=None, stream=None):
        """y = layer(x); x is a [T, H] bfloat16 device tensor."""
        import torch
        s = self.shapes
        T = x.shape[0]
        if self.i8:
            rows, bf = ((T, s.H),), (torch.bfloat16,)
            self._check_tensors(("x", x, rows, bf), *([] if y is None else [("y", y, rows, bf)]))
            if y is None:
                y = self._output(T, stream)
            return self._forward_i8(x, y, stream)
        if y is None:
            y = self._output(T, stream)
        with self._pool(stream):
            ws, nbytes = self.workspace(T)
        self._note_stream(stream)
        W = self.w
        if self.q4:
            q = self.q
            moe.moe_forward_q4(x, W["w_router"], self.bias, q["w_gate_q4"], q["w_gate_q4scale"], q["w_up_q4"],
                               q["w_up_q4scale"], q["w_down_q4"], q["w_down_q4scale"], q["ws_gate_q4"],
                               q["ws_gate_q4scale"], q["ws_up_q4"], q["ws_up_q4scale"], q["ws_down_q4"],
                               q["ws_down_q4scale"], W["w_sg"], T, s.H, s.E, s.k, s.I, s.I_s, y, ws, nbytes, stream)
            return y
        if self.fp8:
            q = self.q
            moe.moe_forward_fp8(x, W["w_router"], self.bias, q["w_gate"], q["w_gate_scale"], q["w_up"],
                                q["w_up_scale"], q["w_down"], q["w_down_scale"], q["ws_gate"], q["ws_gate_scale"],
                                q["ws_up"], q["ws_up_scale"], q["ws_down"], q["ws_down_scale"], W["w_sg"],
                                T, s.H, s.E, s.k, s.I, s.I_s, y, ws, nbytes, stream)
            return y
        moe.moe_forward(x, W["w_router"], self.bias, W["w_gate"], W["w_up"], W["w_down"], W["ws_gate"], W["ws_up"],
                        W["ws_down"], W["w_sg"], T, s.H, s.E, s.k, s.I, s.I_s, y, ws, nbytes, stream)
        return y

    def forward_ids(self, T: int):
        """The expert ids [T, k] (int32, rank order) the last forward of T tokens selected, read back
        from the workspace."""
        import torch
        s = self.shapes
        if self.i8:
            return self._i8_buffers(T)["ids"]
        off = moe.moe_forward_ids_offset(T, s.H, s.E, s.k, s.I, s.I_s)
        return self._ws[off:off + T * s.k * 4].view(torch.int32).view(T, s.k)

    # ---------------------------------------------------------------- 8-bit experts
    def _i8_buffers(self, T: int):
        """The 8-bit forward's intermediates for T tokens, views of the layer's workspace.  The last ones are kept:
        laying them out takes 43 us of the host's time, more than one token's launches."""
        import torch
        v = self._i8_views
        if v is not None and v[1] == T and v[0] == self._ws.data_ptr():
            return v[2]
        s = self.shapes
        n, E = T * s.k, s.E
        i32, f32, i8, bf, u8 = torch.int32, torch.float32, torch.int8, torch.bfloat16, torch.uint8
        rows = moe.moe_align_max_rows(T, E, s.k)
        want = {"ids": (i32, T, s.k), "w": (f32, T, s.k), "s": (f32, T), "counts": (i32, E), "pad_off": (i32, E + 1),
                "sorted": (i32, rows), "inv": (i32, n), "tiles": (i32, 2 * moe.moe_align_max_tiles(T, E, s.k)),
                "n_tiles": (i32, 2), "scratch": (u8, moe.moe_align_scratch_size(T, E, s.k)),
                "route_scratch": (u8, moe.moe_route_scratch_size(T, s.H, E)),
                "xq": (i8, T, s.H), "xs": (f32, T), "gu": (bf, n, 2 * s.I), "hq": (i8, n, s.I), "hs": (f32, n),
                "o": (bf, n, s.H)}
        if s.I_s:
            want.update({"s_gu": (bf, T, 2 * s.I_s), "s_hq": (i8, T, s.I_s), "s_hs": (f32, T)})
        at, place = 0, {}
        for name, (dtype, *shape) in want.items():
            nbytes = int(np.prod(shape)) * dtype.itemsize
            place[name] = (at, nbytes)
            at += -(-nbytes // 256) * 256
        ws, _ = self._reserve(at)
        views = {name: ws[place[name][0]:place[name][0] + place[name][1]].view(dtype).view(*shape)
                 for name, (dtype, *shape) in want.items()}
        self._i8_views = (ws.data_ptr(), T, views)
        return views

    def _forward_i8(self, x, y, stream=None, quantized=False):
        """The layer with its experts in 8-bit integers: routing on the bf16 tokens, then per token one quantisation
        (unless ``xq`` and ``xs`` hold it already), the gate and up rows as one grouped product over the tokens of
        each expert, SwiGLU quantised per assignment, the grouped down product, and the combine.  The shared
        expert's products are dense; its gate multiplies the scales of its SwiGLU rows, and its down product adds
        the routed experts' output, which has been rounded to bf16 once by the combine."""
        s, q = self.shapes, self.q
        T = x.shape[0]
        if T == 0:
            return y
        with self._pool(stream):
            b = self._i8_buffers(T)
        self._note_stream(stream)
        n, E = T * s.k, s.E
        moe.moe_route(x, self.w["w_router"], self.bias, self.w["w_sg"], T, s.H, E, s.k, b["ids"], b["w"],
                      b["s"] if s.I_s else None, None, stream, scratch=b["route_scratch"])
        moe.moe_align(b["ids"], T, E, s.k, b["counts"], b["pad_off"], b["sorted"], b["inv"], b["tiles"],
                      b["n_tiles"], b["scratch"], b["scratch"].numel(), stream)
        if not quantized:
            moe.moe_quantize_i8(x, T, s.H, b["xq"], b["xs"], stream)
        P = b["sorted"].numel()
        gu, gu_scale, down, down_scale = self._i8_experts
        moe.moe_grouped_gemm_i8(b["xq"], b["xs"], gu, gu_scale, b["pad_off"], b["counts"], b["sorted"], s.k,
                                P, n, E, 2 * s.I, s.H, b["gu"], stream)
        moe.moe_swiglu_i8(b["gu"], None, n, s.I, b["hq"], b["hs"], stream)
        moe.moe_grouped_gemm_i8(b["hq"], b["hs"], down, down_scale, b["pad_off"], b["counts"], b["sorted"],
                                1, P, n, E, s.H, s.I, b["o"], stream)
        moe.moe_combine(b["o"], b["w"], None, None, None, T, s.H, s.k, 0, y, stream)
        if s.I_s:
            moe.moe_gemm_i8(b["xq"], b["xs"], q["s_gu"], q["s_gu_scale"], None, None, T, 2 * s.I_s, s.H, b["s_gu"],
                            stream)
            moe.moe_swiglu_i8(b["s_gu"], b["s"], T, s.I_s, b["s_hq"], b["s_hs"], stream)
            moe.moe_gemm_i8(b["s_hq"], b["s_hs"], q["s_down"], q["s_down_scale"], None, y, T, s.H, s.I_s, y, stream)
        return y

    def forward_block(self, r, y, w_pre, w_post=None, gate=None, r_scale: float = 1.0, y_scale: float = 1.0,
                      w_add: float = 0.0, eps: float = 1e-6, out=None, stream=None):
        """The layer as a block of a residual stream: r (in place) takes the previous block's output y (None: it has
        none) through moe_block_norm, and the layer runs on the normalised rows.  Returns the layer's output, which
        the next block's moe_block_norm adds to r.  8-bit layers take the norm's quantised rows as they are.
        r is [T, H] bf16 or fp32; y and out are [T, H], w_pre and w_post [H], gate [H] or [T, H], all bf16."""
        import torch
        s = self.shapes
        bf = torch.bfloat16
        T = r.shape[0]
        rows, one = ((T, s.H),), ((s.H,), (1, s.H))
        given = (("r", r, rows, (bf, torch.float32)), ("y", y, rows, (bf,)), ("w_pre", w_pre, one, (bf,)),
                 ("w_post", w_post, one, (bf,)), ("gate", gate, one + rows, (bf,)), ("out", out, rows, (bf,)))
        self._check_tensors(*(g for g in given if g[1] is not None))
        if out is None:
            out = self._output(T, stream)
        with self._pool(stream):
            x = torch.empty((T, s.H), dtype=bf, device=self.device)
            b = self._i8_buffers(T) if self.i8 and T > 0 else {"xq": None, "xs": None}
        moe.moe_block_norm(r, y, w_post, gate, w_pre, T, s.H, r, x, b["xq"], b["xs"], r_scale, y_scale, w_add, eps,
                           stream)
        if not self.i8:
            return self.forward(x, out, stream)
        return self._forward_i8(x, out, stream, quantized=True)

    # ---------------------------------------------------------------- stages
    def alloc_stage_buffers(self, T: int):
        import torch
        s = self.shapes
        dev = self.device
        max_rows = moe.moe_align_max_rows(T, s.E, s.k)
        max_tiles = moe.moe_align_max_tiles(T, s.E, s.k)
        i32 = dict(dtype=torch.int32, device=dev)
        return {
            "ids": torch.empty((T, s.k), **i32),
            "w": torch.empty((T, s.k), dtype=torch.float32, device=dev),
            "s": torch.empty(max(T, 1), dtype=torch.float32, device=dev),
            "logits": torch.empty((T, s.E), dtype=torch.float32, device=dev),
            "counts": torch.empty(s.E, **i32),
            "pad_off": torch.empty(s.E + 1, **i32),
            "sorted": torch.empty(max_rows, **i32),
            "inv": torch.empty(T * s.k, **i32),
            "tiles": torch.empty(2 * max_tiles, **i32),
            "n_tiles": torch.empty(2, **i32),
            "scratch": torch.empty(moe.moe_align_scratch_size(T, s.E, s.k), dtype=torch.uint8, device=dev),
            "route_scratch": torch.empty(moe.moe_route_scratch_size(T, s.H, s.E), dtype=torch.uint8, device=dev),
            "h": torch.empty((max_rows, s.I), dtype=torch.bfloat16, device=dev),
            "h_s": torch.empty((T, s.I_s), dtype=torch.bfloat16, device=dev) if s.I_s else None,
            "o": torch.empty((T * s.k, s.H), dtype=torch.bfloat16, device=dev),
            "y": torch.empty((T, s.H), dtype=torch.bfloat16, device=dev),
        }

    def run_route(self, x, b, stream=None, streamed=True):
        """streamed: the form moe_forward runs (W_router copied in operand order into scratch, then
        the streamed router); else the one-launch router with W_router staged through LDS."""
        s = self.shapes
        T = x.shape[0]
        moe.moe_route(x, self.w["w_router"], self.bias, self.w["w_sg"], T, s.H, s.E, s.k, b["ids"], b["w"],
                      b["s"] if s.I_s else None, b["logits"], stream, scratch=b["route_scratch"] if streamed else None)

    def run_align(self, T, b, stream=None):
        s = self.shapes
        moe.moe_align(b["ids"], T, s.E, s.k, b["counts"], b["pad_off"], b["sorted"], b["inv"],
                      b["tiles"], b["n_tiles"], b["scratch"], b["scratch"].numel(), stream)

    def run_gate_up(self, x, b, stream=None):
        s = self.shapes
        T = x.shape[0]
        W = self.w
        moe.moe_grouped_gate_up(x, W["w_gate"], W["w_up"], W["ws_gate"], W["ws_up"], b["sorted"], b["tiles"],
                                b["n_tiles"], T, s.H, s.E, s.k, s.I, s.I_s, b["h"], b["h_s"], stream)

    def run_down(self, T, b, stream=None):
        s = self.shapes
        moe.moe_grouped_down(b["h"], self.w["w_down"], b["sorted"], b["tiles"], b["n_tiles"], T, s.H, s.E, s.k,
                             s.I, b["o"], stream)

    def run_combine(self, T, b, stream=None):
        s = self.shapes
        moe.moe_combine(b["o"], b["w"], b["h_s"], self.w["ws_down"], b["s"] if s.I_s else None, T,
                        s.H, s.k, s.I_s, b["y"], stream)

    def run_stages(self, x, b=None, stream=None, ids=None, w=None, s=None):
        """All prefill stages one by one (same kernels as ``forward``); returns the buffers.

        ``ids`` ([T, k] int32), ``w`` ([T, k] fp32) and ``s`` ([T] fp32) device
        tensors, when given, replace the router's outputs before the align
        stage, so align, the grouped GEMMs and the combine can be driven with
        crafted expert loads.
        """
        T = x.shape[0]
        if b is None:
            b = self.alloc_stage_buffers(T)
        self.run_route(x, b, stream)
        if ids is not None:
            b["ids"].copy_(ids)
        if w is not None:
            b["w"].copy_(w)
        if s is not None:
            b["s"][:T].copy_(s)
        self.run_align(T, b, stream)
        self.run_gate_up(x, b, stream)
        self.run_down(T, b, stream)
        self.run_combine(T, b, stream)
        return b


class PrefillRunner:
    """Prefill of any length through per-bucket HIP graphs (moe_prefill_runner_*) for a DeviceLayer's
    weights: its FP8 codes when the layer was built with ``fp8``, else its BF16 weights.  The layer
    must outlive the runner."""

    PAGE_BUCKETS = (1024, 2048, 4096, 8192)

    def __init__(self, layer: DeviceLayer, buckets=PAGE_BUCKETS):
        s = layer.shapes
        W = layer.w
        self.layer = layer
        self.buckets = tuple(buckets)
        self.handle = None
        if layer.q4:
            raise ValueError("the prefill runner takes BF16 or FP8 weights (4-bit weights serve T <= %d)"
                             % moe.Q4_MAX_T)
        if layer.i8:
            raise ValueError("the prefill runner takes BF16 or FP8 weights")
        if layer.fp8:
            q = layer.q
            self.handle = moe.moe_prefill_runner_create_fp8(
                W["w_router"], layer.bias, q["w_gate"], q["w_gate_scale"], q["w_up"], q["w_up_scale"], q["w_down"],
                q["w_down_scale"], q["ws_gate"], q["ws_gate_scale"], q["ws_up"], q["ws_up_scale"], q["ws_down"],
                q["ws_down_scale"], W["w_sg"], s.H, s.E, s.k, s.I, s.I_s, list(self.buckets))
        else:
            self.handle = moe.moe_prefill_runner_create(W["w_router"], layer.bias, W["w_gate"], W["w_up"],
                                                        W["w_down"], W["ws_gate"], W["ws_up"], W["ws_down"],
                                                        W["w_sg"], s.H, s.E, s.k, s.I, s.I_s, list(self.buckets))

    def plan(self, T: int):
        return moe.moe_bucket_plan(T, list(self.buckets))

    def run(self, x, y=None, stream=None):
        """y = layer(x) for a [T, H] bfloat16 device tensor, segment by segment."""
        T = x.shape[0]
        if y is None:
            y = self.layer._output(T, stream)
        moe.moe_prefill_runner_run(self.handle, x, T, y, stream)
        return y

    def close(self):
        """Free the runner's buffers and graphs (after its last run has completed)."""
        if self.handle:
            import torch
            torch.cuda.synchronize(self.layer.device)
            moe.moe_prefill_runner_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

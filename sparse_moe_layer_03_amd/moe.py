"""Thin Python binding of libmoe355 (include/moe.h).

Argument marshalling only: every function takes PyTorch tensors that live on
the GPU, passes their data pointers and the current HIP stream to the C ABI
function of the same name, and raises ``MoEError`` on a non-zero status.
All arithmetic happens in the HIP kernels.  There is no fallback: if the
library has not been built, importing and calling fails loudly.
"""
from __future__ import annotations

import ctypes as C
import math
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE355_LIB names another build of this library to load (the sanitizer build of the CPU tests)
LIB_PATH = os.environ.get("MOE355_LIB") or os.path.join(_PKG, "libmoe355.so")

MOE_OK = 0
MOE_ERR_NULL = -1
MOE_ERR_SHAPE = -2
MOE_ERR_ALIGN = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_ARCH = -5
MOE_ERR_HIP = -6
SMALL_BATCH_MAX_T = 32  # MOE_SMALL_BATCH_MAX_T: moe_forward's small-batch path covers 2 <= T <= this
Q4_MAX_T = 32  # MOE_Q4_MAX_T: moe_forward_q4 covers 1 <= T <= this

EXPORTS = (
    "moe_status_str", "moe_last_error", "moe_align_tile_rows", "moe_align_small_tile_rows", "moe_align_max_rows",
    "moe_align_max_big_tiles", "moe_align_max_tiles", "moe_workspace_size", "moe_forward_ids_offset", "moe_forward", "moe_route", "moe_route_scratch_size", "moe_route_from_logits", "moe_align_scratch_size",
    "moe_align", "moe_grouped_gate_up", "moe_grouped_down", "moe_combine", "moe_forward_fp8", "moe_e4m3_to_f32", "moe_forward_q4",
    "moe_bucket_plan", "moe_prefill_runner_create", "moe_prefill_runner_create_fp8", "moe_prefill_runner_run", "moe_prefill_runner_destroy",
    "moe_forward_noalloc", "moe_workspace_sections",
    "moe_block_norm", "moe_quantize_i8", "moe_swiglu_i8", "moe_gemm_i8", "moe_grouped_gemm", "moe_grouped_gemm_i8",
)
BF16 = 0  # MOE_BF16, MOE_F32: types of a residual stream and of a product's output
F32 = 1
NOALLOC_WS_BYTES = 64 << 20  # MOE_NOALLOC_WS_BYTES: the fixed workspace of moe_forward_noalloc


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_str(status)}: {message}")
        self.status = status


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_moe_layer_03_amd.build`")
        L = C.CDLL(LIB_PATH)
        p, i, z, i64, f = C.c_void_p, C.c_int, C.c_size_t, C.c_int64, C.c_float
        sig = {
            "moe_status_str": ([i], C.c_char_p),
            "moe_last_error": ([], C.c_char_p),
            "moe_align_tile_rows": ([i, i, i], i),
            "moe_align_small_tile_rows": ([i, i, i], i),
            "moe_align_max_rows": ([i, i, i], i64),
            "moe_align_max_big_tiles": ([i, i, i], i64),
            "moe_align_max_tiles": ([i, i, i], i64),
            "moe_workspace_size": ([i, i, i, i, i, i], z),
            "moe_forward_ids_offset": ([i, i, i, i, i, i], z),
            "moe_workspace_sections": ([i, i, i, i, i, i, p, p, i], i),
            "moe_forward": ([p] * 10 + [i] * 6 + [p, p, z, p], i),
            "moe_forward_noalloc": ([p] * 10 + [i] * 6 + [p, p], i),
            "moe_route": ([p, p, p, p, i, i, i, i, p, p, p, p, p, z, p], i),
            "moe_route_scratch_size": ([i, i, i], z),
            "moe_route_from_logits": ([p, i, i, i, p, p, p], i),
            "moe_align_scratch_size": ([i, i, i], z),
            "moe_align": ([p, i, i, i, p, p, p, p, p, p, p, z, p], i),
            "moe_grouped_gate_up": ([p] * 8 + [i] * 6 + [p, p, p], i),
            "moe_grouped_down": ([p] * 5 + [i] * 5 + [p, p], i),
            "moe_combine": ([p] * 5 + [i] * 4 + [p, p], i),
            "moe_forward_fp8": ([p] * 16 + [i] * 6 + [p, p, z, p], i),
            "moe_e4m3_to_f32": ([p, p, i64, p], i),
            "moe_forward_q4": ([p] * 16 + [i] * 6 + [p, p, z, p], i),
            "moe_bucket_plan": ([i, p, i, p, p, i, p], i),
            "moe_prefill_runner_create": ([p] * 9 + [i] * 5 + [p, i, p], i),
            "moe_prefill_runner_create_fp8": ([p] * 15 + [i] * 5 + [p, i, p], i),
            "moe_prefill_runner_run": ([p, p, i, p, p], i),
            "moe_prefill_runner_destroy": ([p], i),
            "moe_block_norm": ([p, i, p, p, p, i, f, f, p, f, f, i, i, p, p, p, p, p], i),
            "moe_quantize_i8": ([p, i, i, p, p, p], i),
            "moe_swiglu_i8": ([p, p, i, i, p, p, p], i),
            "moe_gemm_i8": ([p] * 6 + [i] * 3 + [p, i, p], i),
            "moe_grouped_gemm": ([p] * 5 + [i] * 6 + [p, i, p], i),
            "moe_grouped_gemm_i8": ([p] * 7 + [i] * 6 + [p, i, p], i),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def last_error() -> str:
    return lib().moe_last_error().decode()


def _check(rc: int):
    if rc != MOE_OK:
        raise MoEError(rc, last_error())


def _p(t) -> Optional[int]:
    """Device pointer of a tensor (None stays NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _raw_stream(_device())


# The current device and its current stream: torch's own functions behind the public ones, which take a tenth of their
# time.  Bound at the first call, when torch has initialised the GPU.
def _device() -> int:
    global _device, _raw_stream
    import torch
    at = torch.cuda.current_device()
    get, raw = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get is not None and raw is not None:
        _device, _raw_stream = get, raw
    return at


def _raw_stream(device: int) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


# ------------------------------------------------------------- sizes
def moe_align_tile_rows(T: int, E: int, k: int) -> int:
    return lib().moe_align_tile_rows(T, E, k)


def moe_align_small_tile_rows(T: int, E: int, k: int) -> int:
    return lib().moe_align_small_tile_rows(T, E, k)


def moe_align_max_rows(T: int, E: int, k: int) -> int:
    return lib().moe_align_max_rows(T, E, k)


def moe_align_max_big_tiles(T: int, E: int, k: int) -> int:
    return lib().moe_align_max_big_tiles(T, E, k)


def moe_align_max_tiles(T: int, E: int, k: int) -> int:
    return lib().moe_align_max_tiles(T, E, k)


def moe_workspace_size(T: int, H: int, E: int, k: int, I: int, I_s: int) -> int:
    return lib().moe_workspace_size(T, H, E, k, I, I_s)


def moe_forward_ids_offset(T: int, H: int, E: int, k: int, I: int, I_s: int) -> int:
    return lib().moe_forward_ids_offset(T, H, E, k, I, I_s)


def moe_workspace_sections(T: int, H: int, E: int, k: int, I: int, I_s: int):
    """[(offset, bytes)] of the workspace sections moe_forward carves for these sizes (host only)."""
    L = lib()
    n = L.moe_workspace_sections(T, H, E, k, I, I_s, None, None, 0)
    if n <= 0:
        return []
    off = (C.c_size_t * n)()
    nb = (C.c_size_t * n)()
    L.moe_workspace_sections(T, H, E, k, I, I_s, off, nb, n)
    return [(int(off[i]), int(nb[i])) for i in range(n)]


def moe_align_scratch_size(T: int, E: int, k: int) -> int:
    return lib().moe_align_scratch_size(T, E, k)


# ------------------------------------------------------------- stages
def moe_forward(x, w_router, router_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, w_sg,
                T, H, E, k, I, I_s, y, workspace, ws_bytes: int, stream=None):
    _check(lib().moe_forward(_p(x), _p(w_router), _p(router_bias), _p(w_gate), _p(w_up), _p(w_down),
                             _p(ws_gate), _p(ws_up), _p(ws_down), _p(w_sg), T, H, E, k, I, I_s,
                             _p(y), _p(workspace), ws_bytes, _stream(stream)))


def moe_forward_noalloc(x, w_router, router_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, w_sg,
                        T, H, E, k, I, I_s, y, stream=None):
    _check(lib().moe_forward_noalloc(_p(x), _p(w_router), _p(router_bias), _p(w_gate), _p(w_up), _p(w_down),
                                     _p(ws_gate), _p(ws_up), _p(ws_down), _p(w_sg), T, H, E, k, I, I_s,
                                     _p(y), _stream(stream)))


def moe_forward_fp8(x, w_router, router_bias, q_gate, sc_gate, q_up, sc_up, q_down, sc_down,
                    qs_gate, ssc_gate, qs_up, ssc_up, qs_down, ssc_down, w_sg,
                    T, H, E, k, I, I_s, y, workspace, ws_bytes: int, stream=None):
    _check(lib().moe_forward_fp8(_p(x), _p(w_router), _p(router_bias), _p(q_gate), _p(sc_gate), _p(q_up),
                                 _p(sc_up), _p(q_down), _p(sc_down), _p(qs_gate), _p(ssc_gate), _p(qs_up),
                                 _p(ssc_up), _p(qs_down), _p(ssc_down), _p(w_sg), T, H, E, k, I, I_s,
                                 _p(y), _p(workspace), ws_bytes, _stream(stream)))


def moe_forward_q4(x, w_router, router_bias, q_gate, s_gate, q_up, s_up, q_down, s_down,
                   qs_gate, ss_gate, qs_up, ss_up, qs_down, ss_down, w_sg,
                   T, H, E, k, I, I_s, y, workspace, ws_bytes: int, stream=None):
    _check(lib().moe_forward_q4(_p(x), _p(w_router), _p(router_bias), _p(q_gate), _p(s_gate), _p(q_up),
                                _p(s_up), _p(q_down), _p(s_down), _p(qs_gate), _p(ss_gate), _p(qs_up),
                                _p(ss_up), _p(qs_down), _p(ss_down), _p(w_sg), T, H, E, k, I, I_s,
                                _p(y), _p(workspace), ws_bytes, _stream(stream)))


def moe_e4m3_to_f32(codes, out, n: int, stream=None):
    _check(lib().moe_e4m3_to_f32(_p(codes), _p(out), n, _stream(stream)))


def moe_bucket_plan(T: int, buckets):
    """(segment bucket sizes, real tokens per segment) covering T tokens (host only)."""
    nb = len(buckets)
    barr = (C.c_int * max(nb, 1))(*buckets)
    n = C.c_int(0)
    cap = 64
    while True:
        sb, sl = (C.c_int * cap)(), (C.c_int * cap)()
        rc = lib().moe_bucket_plan(T, barr, nb, sb, sl, cap, C.byref(n))
        if rc == MOE_ERR_SHAPE and n.value > cap:
            cap = n.value
            continue
        _check(rc)
        return list(sb[:n.value]), list(sl[:n.value])


def moe_prefill_runner_create(w_router, router_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, w_sg,
                              H, E, k, I, I_s, buckets) -> int:
    """Opaque runner handle (an int); free it with moe_prefill_runner_destroy."""
    nb = len(buckets)
    barr = (C.c_int * max(nb, 1))(*buckets)
    out = C.c_void_p()
    _check(lib().moe_prefill_runner_create(_p(w_router), _p(router_bias), _p(w_gate), _p(w_up), _p(w_down),
                                           _p(ws_gate), _p(ws_up), _p(ws_down), _p(w_sg), H, E, k, I, I_s,
                                           barr, nb, C.byref(out)))
    return out.value


def moe_prefill_runner_create_fp8(w_router, router_bias, q_gate, sc_gate, q_up, sc_up, q_down, sc_down,
                                  qs_gate, ssc_gate, qs_up, ssc_up, qs_down, ssc_down, w_sg,
                                  H, E, k, I, I_s, buckets) -> int:
    """Runner over FP8 expert weights (codes and row scales as moe_forward_fp8)."""
    nb = len(buckets)
    barr = (C.c_int * max(nb, 1))(*buckets)
    out = C.c_void_p()
    _check(lib().moe_prefill_runner_create_fp8(_p(w_router), _p(router_bias), _p(q_gate), _p(sc_gate), _p(q_up),
                                               _p(sc_up), _p(q_down), _p(sc_down), _p(qs_gate), _p(ssc_gate),
                                               _p(qs_up), _p(ssc_up), _p(qs_down), _p(ssc_down), _p(w_sg),
                                               H, E, k, I, I_s, barr, nb, C.byref(out)))
    return out.value


def moe_prefill_runner_run(runner: int, x, T: int, y, stream=None):
    _check(lib().moe_prefill_runner_run(runner, _p(x), T, _p(y), _stream(stream)))


def moe_prefill_runner_destroy(runner: Optional[int]):
    _check(lib().moe_prefill_runner_destroy(runner))


def moe_route_scratch_size(T, H, E):
    return lib().moe_route_scratch_size(T, H, E)


def moe_route(x, w_router, router_bias, w_sg, T, H, E, k, ids, w, s, logits, stream=None, scratch=None):
    """scratch (a device tensor of moe_route_scratch_size bytes or more) selects the streamed form."""
    nbytes = scratch.numel() * scratch.element_size() if scratch is not None else 0
    _check(lib().moe_route(_p(x), _p(w_router), _p(router_bias), _p(w_sg), T, H, E, k,
                           _p(ids), _p(w), _p(s), _p(logits), _p(scratch), nbytes, _stream(stream)))


def moe_route_from_logits(logits, T, E, k, ids, w, stream=None):
    _check(lib().moe_route_from_logits(_p(logits), T, E, k, _p(ids), _p(w), _stream(stream)))


def moe_align(ids, T, E, k, counts, pad_off, sorted_rows, inv, tiles, n_tiles, scratch, scratch_bytes,
              stream=None):
    _check(lib().moe_align(_p(ids), T, E, k, _p(counts), _p(pad_off), _p(sorted_rows),
                           _p(inv), _p(tiles), _p(n_tiles), _p(scratch), scratch_bytes, _stream(stream)))


def moe_grouped_gate_up(x, w_gate, w_up, ws_gate, ws_up, sorted_rows, tiles, n_tiles, T, H, E, k, I, I_s,
                        h, h_s, stream=None):
    _check(lib().moe_grouped_gate_up(_p(x), _p(w_gate), _p(w_up), _p(ws_gate), _p(ws_up), _p(sorted_rows),
                                     _p(tiles), _p(n_tiles), T, H, E, k, I, I_s, _p(h), _p(h_s),
                                     _stream(stream)))


def moe_grouped_down(h, w_down, sorted_rows, tiles, n_tiles, T, H, E, k, I, o, stream=None):
    _check(lib().moe_grouped_down(_p(h), _p(w_down), _p(sorted_rows), _p(tiles), _p(n_tiles), T, H, E, k, I,
                                  _p(o), _stream(stream)))


def moe_combine(o, w, h_s, ws_down, s, T, H, k, I_s, y, stream=None):
    _check(lib().moe_combine(_p(o), _p(w), _p(h_s), _p(ws_down), _p(s), T, H, k, I_s, _p(y),
                             _stream(stream)))


# ------------------------------------------------------------- operators around the layer
def _args(*tensors):
    """Device pointers of tensors, given as (name, tensor, dtype, shape) (None stays NULL, raw pointers pass, except for
    r, c and gate, whose type or size the calls read).  Refuses what the C ABI cannot tell from the right tensor:
    another type, another shape (see _fits), strides, or another device than the current one (whose stream the call is
    enqueued on)."""
    out = []
    dev = None
    for name, t, dtype, shape in tensors:
        if t is None or t.__class__ is int:
            out.append(t)
        elif (t.dtype is dtype and (t.shape == shape or _fits(name, t, shape)) and t.is_contiguous()
              and (at := t.get_device()) >= 0):
            if at != dev:
                dev = _device()
                if at != dev:
                    raise ValueError(f"{name} is on GPU {at}; the current one is {dev}")
            out.append(t.data_ptr())
        else:
            raise ValueError(_fault(name, t, dtype, shape))
    return out


def _fits(name, t, shape) -> bool:
    """Whether a tensor of another shape holds one of this shape from its first element on: it is flat or its rows are
    as long, and it has as many elements or more (the norms' weights: as many)."""
    n = math.prod(shape)
    if name in ("w_post", "w_pre"):
        return t.numel() == n
    return t.numel() >= n and (len(shape) == 1 or t.dim() < 2 or t.shape[-1] == shape[-1])


def _fault(name, t, dtype, shape) -> str:
    n = math.prod(shape)
    if t.dtype is not dtype:
        return f"{name} is {t.dtype}; expected {dtype}"
    if t.numel() < n:
        return f"{name} has {t.numel()} elements; {n} needed"
    if not t.is_contiguous():
        return f"{name} must be contiguous"
    if not _fits(name, t, shape):
        if len(shape) == 1:
            return f"{name} has {t.numel()} elements; expected {n}"
        return f"{name} has rows of {t.shape[-1]} elements; expected {shape[-1]}"
    return f"{name} is on {t.device}, not on a GPU"


def _type(name, t):
    """(MOE_BF16 or MOE_F32, the torch type) of a residual stream or a product's output (None: the library's to
    report)."""
    import torch
    if t.__class__ is int:
        raise ValueError(f"{name} must be a tensor: its type is the call's")
    if t is None or t.dtype is torch.bfloat16:
        return BF16, torch.bfloat16
    if t.dtype is torch.float32:
        return F32, torch.float32
    raise ValueError(f"{name} is {t.dtype}; expected torch.bfloat16 or torch.float32")


def moe_block_norm(r, y, w_post, gate, w_pre, T, H, r_out, x, q, q_scale, r_scale: float = 1.0, y_scale: float = 1.0,
                   w_add: float = 0.0, eps: float = 1e-6, stream=None):
    """The type of r (bf16 or fp32) is that of r_out; gate has H elements (one row for all tokens) or T * H."""
    import torch
    bf, rows = torch.bfloat16, (T, H)
    r_type, rt = _type("r", r)
    if gate.__class__ is int:
        raise ValueError("gate must be a tensor: its size tells one row from T")
    one = gate is None or gate.numel() == H
    r, y, w_post, gate, w_pre, r_out, x, q, q_scale = _args(
        ("r", r, rt, rows), ("y", y, bf, rows), ("w_post", w_post, bf, (H,)),
        ("gate", gate, bf, (H,) if one else rows), ("w_pre", w_pre, bf, (H,)), ("r_out", r_out, rt, rows),
        ("x", x, bf, rows), ("q", q, torch.int8, rows), ("q_scale", q_scale, torch.float32, (T,)))
    _check(lib().moe_block_norm(r, r_type, y, w_post, gate, 1 if one else T, r_scale, y_scale, w_pre, w_add, eps, T, H,
                                r_out, x, q, q_scale, _stream(stream)))


def moe_quantize_i8(x, R, K, q, scale, stream=None):
    import torch
    x, q, scale = _args(("x", x, torch.bfloat16, (R, K)), ("q", q, torch.int8, (R, K)),
                        ("scale", scale, torch.float32, (R,)))
    _check(lib().moe_quantize_i8(x, R, K, q, scale, _stream(stream)))


def moe_swiglu_i8(gu, row_gate, R, I, q, scale, stream=None):
    import torch
    gu, row_gate, q, scale = _args(
        ("gu", gu, torch.bfloat16, (R, 2 * I)), ("row_gate", row_gate, torch.float32, (R,)),
        ("q", q, torch.int8, (R, I)), ("scale", scale, torch.float32, (R,)))
    _check(lib().moe_swiglu_i8(gu, row_gate, R, I, q, scale, _stream(stream)))


def moe_gemm_i8(a, a_scale, b, b_scale, bias, add, M, N, K, c, stream=None):
    """The type of c (bf16 or fp32) is the output's."""
    import torch
    i8, f32 = torch.int8, torch.float32
    c_type, ct = _type("c", c)
    a, a_scale, b, b_scale, bias, add, c = _args(
        ("a", a, i8, (M, K)), ("a_scale", a_scale, f32, (M,)), ("b", b, i8, (N, K)),
        ("b_scale", b_scale, f32, (N,)), ("bias", bias, f32, (N,)), ("add", add, torch.bfloat16, (M, N)),
        ("c", c, ct, (M, N)))
    _check(lib().moe_gemm_i8(a, a_scale, b, b_scale, bias, add, M, N, K, c, c_type, _stream(stream)))


def _a_rows(a_div, R):
    return (R - 1) // a_div + 1 if R > 0 and a_div > 0 else 0


def moe_grouped_gemm(a, b, off, counts, rows, a_div, P, R, E, N, K, c, stream=None):
    """The type of c (bf16 or fp32) is the output's."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    c_type, ct = _type("c", c)
    a, b, off, counts, rows, c = _args(
        ("a", a, bf, (_a_rows(a_div, R), K)), ("b", b, bf, (E, N, K)), ("off", off, i32, (E + 1,)),
        ("counts", counts, i32, (E,)), ("rows", rows, i32, (P,)), ("c", c, ct, (R, N)))
    _check(lib().moe_grouped_gemm(a, b, off, counts, rows, a_div, P, R, E, N, K, c, c_type, _stream(stream)))


def moe_grouped_gemm_i8(a, a_scale, b, b_scale, off, counts, rows, a_div, P, R, E, N, K, c, stream=None):
    """The type of c (bf16 or fp32) is the output's."""
    import torch
    i8, f32, i32 = torch.int8, torch.float32, torch.int32
    c_type, ct = _type("c", c)
    n = _a_rows(a_div, R)
    a, a_scale, b, b_scale, off, counts, rows, c = _args(
        ("a", a, i8, (n, K)), ("a_scale", a_scale, f32, (n,)), ("b", b, i8, (E, N, K)),
        ("b_scale", b_scale, f32, (E, N)), ("off", off, i32, (E + 1,)), ("counts", counts, i32, (E,)),
        ("rows", rows, i32, (P,)), ("c", c, ct, (R, N)))
    _check(lib().moe_grouped_gemm_i8(a, a_scale, b, b_scale, off, counts, rows, a_div, P, R, E, N, K, c, c_type,
                                     _stream(stream)))

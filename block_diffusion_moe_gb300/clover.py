"""ctypes binding of libclover (include/clover.h).

Argument marshalling only: every step of the denoising path runs in the CUDA
library. PyTorch supplies device memory and the current stream. There is no
CPU or PyTorch fallback: if the library is missing, loading fails.

A call with stream= behaves as inside `with torch.cuda.stream(stream)`: what it
allocates, results included, belongs to that stream. The caller orders its
inputs before the call, and tells the allocator (Tensor.record_stream) of a
tensor that is dropped while a stream other than its own still uses it.
"""
from __future__ import annotations

import ctypes
import operator
import os

import torch

from . import synth

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libclover.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_WORKSPACE_TOO_SMALL = -2
ERR_CUDA = -3
ERR_NOT_CONVERGED = -4
ERR_UNSUPPORTED_SHAPE = -5
ERR_DEVICE_TIMEOUT = -6


class CloverError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"clover error {code}: {msg}")
        self.code = code


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("vocab", ctypes.c_int32), ("mask_id", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("coreset_top_p", ctypes.c_float)]


class MoeLayer(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p), ("gate_up", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("sh_gate_up", ctypes.c_void_p), ("sh_down", ctypes.c_void_p),
                ("gate_up_q", ctypes.c_void_p), ("gate_up_s", ctypes.c_void_p), ("down_q", ctypes.c_void_p),
                ("down_s", ctypes.c_void_p), ("sh_gate_up_q", ctypes.c_void_p), ("sh_gate_up_s", ctypes.c_void_p),
                ("sh_down_q", ctypes.c_void_p), ("sh_down_s", ctypes.c_void_p)]


class Routing(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_rank", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


_i32, _i64, _ptr_t, _size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t

EXPORTS = {
    "clover_moe_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "clover_moe_block_step": (ctypes.c_int, [ctypes.POINTER(Dims), ctypes.POINTER(MoeLayer), ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "clover_head_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "clover_lmhead_unmask": (ctypes.c_int, [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_float, ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_size_t, ctypes.c_void_p]),
    "clover_lmhead_unmask_static": (ctypes.c_int, [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.c_void_p,
                                                   ctypes.c_void_p, ctypes.c_float, ctypes.c_int32, ctypes.c_void_p,
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                   ctypes.c_int32, ctypes.c_void_p]),
    "clover_lmhead_unmask_static_status": (ctypes.c_int, [ctypes.c_void_p]),
    "clover_quantize_q4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "clover_accept_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "clover_lmhead_accept": (ctypes.c_int, [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_float,
                                            ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_size_t, ctypes.c_void_p]),
    "clover_denoise_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "clover_denoise_hidden_offset": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "clover_denoise_step": (ctypes.c_int, [ctypes.POINTER(Dims), ctypes.POINTER(MoeLayer), ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "clover_denoise_block": (ctypes.c_int, [ctypes.POINTER(Dims), ctypes.POINTER(MoeLayer), ctypes.c_int32,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_float, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                            ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "clover_workspace_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "clover_profile_expert_events": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32]),
    "clover_last_error": (ctypes.c_int32, [ctypes.c_char_p, ctypes.c_size_t]),
    "clover_version": (ctypes.c_int32, []),
    "clover_route_workspace_bytes": (_size, [ctypes.POINTER(Routing), _i32]),
    "clover_route": (ctypes.c_int, [ctypes.POINTER(Routing), _ptr_t, _i32, _i64, _ptr_t, _i32, _ptr_t, _ptr_t, _ptr_t,
                                    _ptr_t, _ptr_t, _ptr_t, _size, _ptr_t]),
    "clover_fp4_scale_bytes": (_size, [_i32, _i32, _i32, _i32]),
    "clover_fp4_grouped_scale_bytes": (_size, [_i32, _i32, _i32, _i32]),
    "clover_quantize_fp4": (ctypes.c_int, [_i32, _ptr_t, _i32, _i64, _i32, _i32, _i32, _i32, _ptr_t, _ptr_t, _ptr_t]),
    "clover_quantize_fp4_rows": (ctypes.c_int, [_i32, _ptr_t, _i32, _i64, _i32, _i32, _i32, _ptr_t, _i32, _i32,
                                                _ptr_t, _i32, _ptr_t, _ptr_t, _ptr_t]),
    "clover_dequantize_fp4": (ctypes.c_int, [_i32, _ptr_t, _ptr_t, _i32, _i32, _i32, _i32, _ptr_t, _i32, _ptr_t,
                                             _ptr_t]),
    "clover_fp4_product_workspace_bytes": (_size, []),
    "clover_fp4_product_shared_workspace": (ctypes.c_int, [ctypes.POINTER(_ptr_t)]),
    "clover_fp4_product": (ctypes.c_int, [_i32, _ptr_t, _ptr_t, _i32, _ptr_t, _ptr_t, _ptr_t, _i32, _i32, _i32,
                                          ctypes.c_float, _ptr_t, _i32, _ptr_t, _ptr_t, _size, _ptr_t]),
    "clover_moe_combine": (ctypes.c_int, [_ptr_t, _i32, _ptr_t, _ptr_t, _ptr_t, _ptr_t, _ptr_t, _i32, _i32, _i32,
                                          _ptr_t]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Loads libclover.so (built by __graft_entry__.build()). Raises if it is
    missing: there is no fallback implementation."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libclover.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    buf = ctypes.create_string_buffer(512)
    lib().clover_last_error(buf, 512)
    return buf.value.decode()


def _check(rc: int):
    if rc != OK:
        raise CloverError(rc, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _as_current(stream, t):
    """Makes `stream`, of the device that holds t, the current one for the rest of a call, so that what the call
    allocates belongs to the stream it runs on: a block of another stream's may still be in use there, is filled there,
    and goes back to it when the call drops it."""
    if stream.device != t.device:
        raise CloverError(ERR_INVALID_ARG, f"the stream is of {stream.device}, the tensors are on {t.device}")
    return torch.cuda.stream(stream)


def make_dims(d: synth.Dims, coreset_top_p: float = 0.0) -> Dims:
    return Dims(d.hidden, d.n_experts, d.top_k, d.d_ff, d.vocab, d.mask_id, d.rms_eps, coreset_top_p)


class Q4Layer:
    """A layer whose expert weights are in the low-bit format
    (clover_quantize_q4): codes uint8 and scales int16 (bf16 bits), device
    tensors; the router stays bf16."""

    def __init__(self, router_w, router_bias, gate_up_q, gate_up_s, down_q, down_s, sh_gate_up_q, sh_gate_up_s,
                 sh_down_q, sh_down_s):
        self.router_w, self.router_bias = router_w, router_bias
        self.gate_up_q, self.gate_up_s, self.down_q, self.down_s = gate_up_q, gate_up_s, down_q, down_s
        self.sh_gate_up_q, self.sh_gate_up_s, self.sh_down_q, self.sh_down_s = (sh_gate_up_q, sh_gate_up_s,
                                                                                sh_down_q, sh_down_s)


def quantize_q4(w, stream=None):
    """bf16 [n_mats][rows][cols] (or [rows][cols]) -> (codes uint8
    [..][rows][cols/2], scales int16 [..][cols/64][rows]) on the device."""
    if stream is not None:
        with _as_current(stream, w):
            return quantize_q4(w)
    assert w.is_cuda and w.dtype == torch.bfloat16 and w.is_contiguous()
    shape = tuple(w.shape)
    w3 = w.view(1, *shape) if w.dim() == 2 else w
    n, rows, cols = w3.shape
    q = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=w.device)
    sc = torch.empty((n, cols // 64, rows), dtype=torch.int16, device=w.device)
    _check(lib().clover_quantize_q4(_ptr(w3), n, rows, cols, _ptr(q), _ptr(sc), _stream()))
    if w.dim() == 2:
        return q[0], sc[0]
    return q, sc


def quantize_layer_q4(L: synth.Layer, stream=None) -> Q4Layer:
    gq, gs = quantize_q4(L.gate_up, stream)
    dq, ds = quantize_q4(L.down, stream)
    sgq, sgs = quantize_q4(L.sh_gate_up, stream)
    sdq, sds = quantize_q4(L.sh_down, stream)
    return Q4Layer(L.router_w, L.router_bias, gq, gs, dq, ds, sgq, sgs, sdq, sds)


def make_layer(L) -> MoeLayer:
    if L.router_bias is not None:
        assert L.router_bias.is_cuda and L.router_bias.dtype == torch.float32
    bias = None if L.router_bias is None else L.router_bias.data_ptr()
    if isinstance(L, Q4Layer):
        ts = (L.gate_up_q, L.gate_up_s, L.down_q, L.down_s, L.sh_gate_up_q, L.sh_gate_up_s, L.sh_down_q, L.sh_down_s)
        for t in ts:
            assert t.is_cuda and t.is_contiguous()
        return MoeLayer(L.router_w.data_ptr(), bias, None, None, None, None, *[t.data_ptr() for t in ts])
    for t in (L.router_w, L.gate_up, L.down, L.sh_gate_up, L.sh_down):
        assert t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()
    return MoeLayer(L.router_w.data_ptr(), bias, L.gate_up.data_ptr(), L.down.data_ptr(), L.sh_gate_up.data_ptr(),
                    L.sh_down.data_ptr())


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zero-filled, 256-byte aligned device workspace (torch allocations are)."""
    if nbytes <= 0:
        raise CloverError(ERR_UNSUPPORTED_SHAPE, last_error())
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_workspace_bytes(d: synth.Dims, max_tokens: int) -> int:
    return lib().clover_moe_workspace_bytes(ctypes.byref(make_dims(d)), max_tokens)


def head_workspace_bytes(d: synth.Dims, max_tokens: int) -> int:
    return lib().clover_head_workspace_bytes(ctypes.byref(make_dims(d)), max_tokens)


def denoise_workspace_bytes(d: synth.Dims, max_tokens: int) -> int:
    return lib().clover_denoise_workspace_bytes(ctypes.byref(make_dims(d)), max_tokens)


def denoise_hidden(d: synth.Dims, ws: torch.Tensor, M: int) -> torch.Tensor:
    """The fp32 [M][H] residual stream the last denoise step left in `ws`
    (a view into the workspace)."""
    o = lib().clover_denoise_hidden_offset(ctypes.byref(make_dims(d)), M)
    if o == 0:
        raise CloverError(ERR_INVALID_ARG, last_error())
    return ws[o:o + M * d.hidden * 4].view(torch.float32).view(M, d.hidden)


def moe_block_step(d: synth.Dims, layer: synth.Layer, x_in: torch.Tensor, x_out: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, with_topk: bool = True, stream=None, coreset_top_p: float = 0.0):
    if stream is not None:
        with _as_current(stream, x_in):
            return moe_block_step(d, layer, x_in, x_out, ws, with_topk, coreset_top_p=coreset_top_p)
    M = x_in.shape[0]
    if x_out is None:
        x_out = torch.empty_like(x_in)
    if ws is None:
        ws = workspace(moe_workspace_bytes(d, M), x_in.device)
    idx = torch.empty((M, d.top_k), dtype=torch.int32, device=x_in.device) if with_topk else None
    w = torch.empty((M, d.top_k), dtype=torch.float32, device=x_in.device) if with_topk else None
    dims = make_dims(d, coreset_top_p)
    lay = make_layer(layer)
    _check(lib().clover_moe_block_step(ctypes.byref(dims), ctypes.byref(lay), _ptr(x_in), _ptr(x_out), _ptr(idx),
                                       _ptr(w), M, _ptr(ws), ws.numel(), _stream()))
    return x_out, idx, w


def lmhead_unmask(d: synth.Dims, head_w, x, tokens, masked, logit_scale=None, threshold: float = 0.95,
                  block: int = 32, ws=None, stream=None, out=None) -> dict:
    """Head statistics + unmask over M = x.shape[0] positions. `out` (a dict
    this function returned before, for the same M) is reused; the library
    writes every entry, including the committed count."""
    if stream is not None:
        with _as_current(stream, x):
            return lmhead_unmask(d, head_w, x, tokens, masked, logit_scale, threshold, block, ws, out=out)
    M = x.shape[0]
    dev = x.device
    if ws is None:
        ws = workspace(head_workspace_bytes(d, M), dev)
    if out is None:
        out = {"argmax": torch.empty(M, dtype=torch.int32, device=dev),
               "max_logit": torch.empty(M, dtype=torch.float32, device=dev),
               "lse": torch.empty(M, dtype=torch.float32, device=dev),
               "max_prob": torch.empty(M, dtype=torch.float32, device=dev),
               "n_committed": (torch.empty if M > 0 else torch.zeros)(1, dtype=torch.int32, device=dev)}
    dims = make_dims(d)
    _check(lib().clover_lmhead_unmask(ctypes.byref(dims), _ptr(head_w), _ptr(x), _ptr(logit_scale), threshold, block,
                                      _ptr(tokens), _ptr(masked), _ptr(out["argmax"]), _ptr(out["max_logit"]),
                                      _ptr(out["lse"]), _ptr(out["max_prob"]), _ptr(out["n_committed"]), M,
                                      _ptr(ws), ws.numel(), _stream()))
    return out


ACCEPT_EXACT = 0
ACCEPT_THRESHOLD = 1


def accept_workspace_bytes(d: synth.Dims, max_rows: int) -> int:
    return lib().clover_accept_workspace_bytes(ctypes.byref(make_dims(d)), max_rows)


def lmhead_accept(d: synth.Dims, head_w, x, draft, block: int, rule: int = ACCEPT_EXACT, ratio: float = 0.9,
                  delta: float = 0.6, logit_scale=None, ws=None, stream=None, out=None) -> dict:
    """Verify-pass head + accept test over M = x.shape[0] rows in blocks of
    `block` rows (block - 1 drafts + the boundary row). `out` (a dict this
    function returned before, for the same M and block) is reused."""
    if stream is not None:
        with _as_current(stream, x):
            return lmhead_accept(d, head_w, x, draft, block, rule, ratio, delta, logit_scale, ws, out=out)
    M = x.shape[0]
    dev = x.device
    if ws is None:
        ws = workspace(accept_workspace_bytes(d, M), dev)
    if out is None:
        f32 = lambda: torch.empty(M, dtype=torch.float32, device=dev)
        out = {"argmax": torch.empty(M, dtype=torch.int32, device=dev), "max_logit": f32(), "lse": f32(),
               "max_prob": f32(), "entropy": f32(), "p_draft": f32(),
               "accept_len": torch.empty(max(1, M // max(block, 1)), dtype=torch.int32, device=dev),
               "tokens": torch.empty(M, dtype=torch.int32, device=dev)}
    dims = make_dims(d)
    _check(lib().clover_lmhead_accept(ctypes.byref(dims), _ptr(head_w), _ptr(x), _ptr(logit_scale), _ptr(draft),
                                      rule, ratio, delta, block, _ptr(out["argmax"]), _ptr(out["max_logit"]),
                                      _ptr(out["lse"]), _ptr(out["max_prob"]), _ptr(out["entropy"]),
                                      _ptr(out["p_draft"]), _ptr(out["accept_len"]), _ptr(out["tokens"]), M,
                                      _ptr(ws), ws.numel(), _stream()))
    return out


class Model:
    """Device-resident weights of a stack of MoE sublayers plus embedding and
    head, with the ctypes layer array the denoise entry points take."""

    def __init__(self, d: synth.Dims, layers, embed, head_w, coreset_top_p: float = 0.0):
        self.d = d
        self.layers = list(layers)
        self.embed = embed
        self.head_w = head_w
        self.c_layers = (MoeLayer * max(1, len(self.layers)))(*[make_layer(L) for L in self.layers])
        self.c_dims = make_dims(d, coreset_top_p)


def denoise_step(m: Model, ctx, tokens, masked, logit_scale=None, threshold: float = 0.95, block: int = 32,
                 ws=None, stream=None):
    if stream is not None:
        with _as_current(stream, tokens):
            return denoise_step(m, ctx, tokens, masked, logit_scale, threshold, block, ws)
    M = tokens.shape[0]
    if ws is None:
        ws = workspace(denoise_workspace_bytes(m.d, M), tokens.device)
    _check(lib().clover_denoise_step(ctypes.byref(m.c_dims), m.c_layers, len(m.layers), _ptr(m.embed), _ptr(ctx),
                                     _ptr(m.head_w), _ptr(logit_scale), threshold, block, _ptr(tokens),
                                     _ptr(masked), M, _ptr(ws), ws.numel(), _stream()))
    return ws


def denoise_block(m: Model, ctx, tokens, masked, logit_scale=None, threshold: float = 0.95, block: int = 32,
                  max_steps: int = 32, ws=None, stream=None) -> int:
    if stream is not None:
        with _as_current(stream, tokens):
            return denoise_block(m, ctx, tokens, masked, logit_scale, threshold, block, max_steps, ws)
    M = tokens.shape[0]
    if ws is None:
        ws = workspace(denoise_workspace_bytes(m.d, M), tokens.device)
    steps = ctypes.c_int32(0)
    _check(lib().clover_denoise_block(ctypes.byref(m.c_dims), m.c_layers, len(m.layers), _ptr(m.embed), _ptr(ctx),
                                      _ptr(m.head_w), _ptr(logit_scale), threshold, block, _ptr(tokens),
                                      _ptr(masked), M, max_steps, ctypes.byref(steps), _ptr(ws), ws.numel(),
                                      _stream()))
    return steps.value


def workspace_status(ws: torch.Tensor, stream=None):
    _check(lib().clover_workspace_status(_ptr(ws), ws.numel(), _stream(stream)))


# ------------------------------------------- routed experts as separate calls
#
# Tensors are checked here (type, shape, layout, one device: the current one);
# values and limits are checked by the library. A refused argument raises
# CloverError with the library's codes.

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
FP4_NV = 0
FP4_MX = 1
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}
_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
_TYPES = {_F32: 0, _BF16: 1}
_UNGROUPED = {"idx", "w"}
_GROUPED = _UNGROUPED | {"offsets", "rows", "pos"}
# (calls of a few microseconds: the device and stream objects of torch.cuda cost as much as the launch)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _refuse(msg: str):
    raise CloverError(ERR_INVALID_ARG, msg)


def _counts(*values):
    """Refuses what would wrap on its way to the library's 32-bit arguments."""
    for v in values:
        if not -(1 << 31) <= v < 1 << 31:
            _refuse(f"{v}: a count past 32 bits")


def _tensor(name: str, t, dtype, shape, dev: int) -> int:
    """The pointer of a contiguous tensor of this type and shape on CUDA device `dev`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(f"{name}: need contiguous {dtype} {tuple(shape)} on cuda:{dev}, "
                f"got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _length(name: str, t) -> int:
    if t.dim() != 1:
        _refuse(f"{name}: need one dimension, got {tuple(t.shape)}")
    return t.shape[0]


def _on_current(name: str, t) -> int:
    """The index of the current CUDA device, which holds t."""
    dev = t.get_device()  # -1 on the host
    if dev < 0 or dev != _current_device():
        _refuse(f"{name} is on {t.device}, not on the current CUDA device")
    return dev


def _rows_of(name: str, t):
    """(device, pointer, type code, row stride in elements) of a 2-D fp32 or bf16 tensor with contiguous rows on the
    current device."""
    dev, kind, strides = _on_current(name, t), _TYPES.get(t.dtype), t.stride()
    if len(strides) != 2 or kind is None or (strides[1] != 1 and t.shape[1] > 1):
        _refuse(f"{name}: need a 2-D fp32 or bf16 tensor with contiguous rows, got {t.dtype} {tuple(t.shape)}, "
                f"strides {strides}")
    rows, cols = t.shape
    if rows > 1 << 29 or cols > 1 << 29:  # (past 32 bits a count would wrap on its way to the library)
        raise CloverError(ERR_UNSUPPORTED_SHAPE, f"{name}: {tuple(t.shape)} is past 2^29 rows or columns")
    return dev, t.data_ptr(), kind, (strides[0] if rows > 1 else max(strides[0], cols))


def _scratch(ws, dev: int):
    """(pointer, bytes) of a caller's workspace."""
    if ws.dtype is not _U8 or ws.get_device() != dev or not ws.is_contiguous():
        _refuse(f"ws: need contiguous uint8 on cuda:{dev}, got {ws.dtype} on {ws.device}, strides {ws.stride()}")
    return ws.data_ptr(), ws.numel()


def make_routing(n_experts: int, top_k: int, score: str = "softmax", n_groups: int = 1, top_groups: int | None = None,
                 group_rank: int = 1, renormalise: bool = True, scale: float = 1.0) -> Routing:
    """The selection rule of `route`. top_groups defaults to every group."""
    if score not in _SCORES:
        _refuse(f"score {score!r} is neither 'softmax' nor 'sigmoid'")
    top_groups = n_groups if top_groups is None else top_groups
    _counts(n_experts, top_k, n_groups, top_groups, group_rank)
    return Routing(n_experts, top_k, _SCORES[score], n_groups, top_groups, group_rank, int(bool(renormalise)), scale)


def route_workspace_bytes(r: Routing, max_tokens: int) -> int:
    _counts(max_tokens)
    return lib().clover_route_workspace_bytes(r, max_tokens)


def route(r: Routing, logits, bias=None, grouping: bool = True, ws=None, out=None, stream=None) -> dict:
    """Expert selection from router logits [M][E] (fp32 or bf16, rows may be strided) -> idx int32 [M][K], w fp32
    [M][K] and, with grouping, offsets int32 [E + 1], rows int32 [M * K], pos int32 [M][K]. `out` (a dict this
    function returned before, for the same shape) is reused."""
    if stream is not None:
        with _as_current(stream, logits):
            return route(r, logits, bias, grouping, ws, out)
    dev, p_logits, kind, ld = _rows_of("logits", logits)
    M, cols = logits.shape
    K, E = r.top_k, r.n_experts
    if cols != E:
        _refuse(f"logits have {cols} columns for {E} experts")
    slots = (M, K)
    p_bias = None if bias is None else _tensor("bias", bias, _F32, (E,), dev)
    if ws is None:
        ws = workspace(route_workspace_bytes(r, M), logits.device)
    if out is None:
        device = logits.device
        out = {"idx": torch.empty(slots, dtype=_I32, device=device), "w": torch.empty(slots, dtype=_F32, device=device)}
        if grouping:
            out["offsets"] = torch.empty(E + 1, dtype=_I32, device=device)
            out["rows"] = torch.empty(M * K, dtype=_I32, device=device)
            out["pos"] = torch.empty(slots, dtype=_I32, device=device)
    elif not (_GROUPED if grouping else _UNGROUPED) <= out.keys():
        _refuse(f"out holds {sorted(out)}, not what this call returns")
    p_off = p_rows = p_pos = None
    if grouping:
        p_off = _tensor("offsets", out["offsets"], _I32, (E + 1,), dev)
        p_rows = _tensor("rows", out["rows"], _I32, (M * K,), dev)
        p_pos = _tensor("pos", out["pos"], _I32, slots, dev)
    rc = lib().clover_route(r, p_logits, kind, ld, p_bias, M, _tensor("idx", out["idx"], _I32, slots, dev),
                            _tensor("w", out["w"], _F32, slots, dev), p_off, p_rows, p_pos, *_scratch(ws, dev),
                            _current_stream(dev))
    if rc != OK:
        _check(rc)
    return out


class Fp4:
    """Matrices in a microscaled 4-bit format: codes uint8 [rows][cols / 2] or [mats][rows][cols / 2], scale tiles
    uint8 (1-D), and the power of two the values are scaled by. With offsets (int32 [groups + 1]) the rows of one
    matrix form groups. The parts are checked against one another here, once, and cannot be replaced but for offsets
    and scale_exp."""

    __slots__ = ("scale_exp", "_fmt", "_device", "_mats", "_rows", "_cols", "_groups", "_offsets", "_shape", "_codes",
                 "_scales", "_at")
    # (the calls below read the fields themselves)
    fmt, device, mats, rows, cols, groups = (property(operator.attrgetter(f)) for f in (
        "_fmt", "_device", "_mats", "_rows", "_cols", "_groups"))

    def __init__(self, fmt: int, codes, scales, scale_exp: int = 0, offsets=None):
        if codes.dtype != _U8 or codes.dim() not in (2, 3) or not codes.is_contiguous():
            _refuse(f"codes: need contiguous uint8 [rows][cols / 2] or [mats][rows][cols / 2], got {codes.dtype} "
                    f"{tuple(codes.shape)}")
        if scales.dtype != _U8 or scales.device != codes.device or not scales.is_contiguous():
            _refuse(f"scales: need contiguous uint8 on {codes.device}, got {scales.dtype} {tuple(scales.shape)} on "
                    f"{scales.device}")
        self._fmt, self.scale_exp, self._device = fmt, scale_exp, codes.device
        self._shape, self._codes, self._scales, self._at = codes.shape, codes, scales, -1  # two tensors
        self._mats = codes.shape[0] if codes.dim() == 3 else 1
        self._rows, self._cols = codes.shape[-2], 2 * codes.shape[-1]
        self.offsets = offsets

    @classmethod
    def _new(cls, fmt, shape, scale_bytes, scale_exp, offsets, groups, device, mats, rows, cols):
        """Room for codes of this shape and as many scales, in one allocation: the codes, then the scales."""
        q = object.__new__(cls)
        at = (mats * rows * cols // 2 + 127) & -128
        q._codes = q._scales = torch.empty(at + scale_bytes, dtype=_U8, device=device)
        q._fmt, q.scale_exp, q._offsets, q._shape, q._at = fmt, scale_exp, offsets, shape, at
        q._device, q._mats, q._rows, q._cols, q._groups = device, mats, rows, cols, groups
        return q

    @property
    def codes(self):
        return self._codes if self._at < 0 else self._codes[:self._mats * self._rows * self._cols // 2].view(self._shape)

    @property
    def scales(self):
        return self._scales if self._at < 0 else self._scales[self._at:]

    def _pointers(self):
        p = self._codes.data_ptr()
        return p, (self._scales.data_ptr() if self._at < 0 else p + self._at)

    @property
    def offsets(self):
        return self._offsets

    @offsets.setter
    def offsets(self, offsets):
        self._offsets, self._groups = offsets, self._groups_of(offsets)

    def _groups_of(self, offsets):
        """The number of groups of these offsets, checked against the scales' room."""
        if offsets is not None:
            if len(self._shape) != 2:
                _refuse("rows in groups form one matrix")
            if offsets.dim() != 1 or offsets.dtype != torch.int32 or offsets.device != self._device \
                    or not offsets.is_contiguous():
                _refuse(f"offsets: need contiguous int32 [groups + 1] on {self._device}, got {offsets.dtype} "
                        f"{tuple(offsets.shape)} on {offsets.device}")
        groups = 0 if offsets is None else offsets.shape[0] - 1
        need = fp4_scale_bytes(self._fmt, self._mats, self._rows, self._cols, None if offsets is None else groups)
        have = self._scales.numel() - max(self._at, 0)
        if have < need:
            _refuse(f"scales: {have} bytes, need {need}")
        return groups


def fp4_scale_bytes(fmt: int, n_mats: int, rows: int, cols: int, n_groups: int | None = None) -> int:
    """Bytes of the scale tiles of n_mats matrices, or of `rows` rows in n_groups groups."""
    _counts(fmt, n_mats, rows, cols, n_groups or 0)
    if n_groups is None:
        n = lib().clover_fp4_scale_bytes(fmt, n_mats, rows, cols)
    else:
        n = lib().clover_fp4_grouped_scale_bytes(fmt, rows, n_groups, cols)
    if n == 0 and (n_groups is not None or (n_mats != 0 and rows != 0)):
        raise CloverError(ERR_UNSUPPORTED_SHAPE, last_error())
    return n


def quantize_fp4(x, fmt: int = FP4_NV, scale_exp: int = 0, offsets=None, src_rows=None, src_div: int = 1, out=None,
                 stream=None) -> Fp4:
    """fp32 or bf16 matrices [rows][cols] or [mats][rows][cols] -> Fp4. With offsets (int32 [groups + 1]) the rows form
    groups: row i comes from x row src_rows[i] // src_div (src_rows int32, default i), as `route` lists them. `out` (an
    Fp4 this function returned before, for the same shapes) is reused."""
    if stream is not None:
        with _as_current(stream, x):
            return quantize_fp4(x, fmt, scale_exp, offsets, src_rows, src_div, out)
    shape, grouped = x.shape, offsets is not None
    if len(shape) == 3:
        if grouped or not x.is_contiguous():
            _refuse("x: matrices must be contiguous, and grouped rows one matrix")
        dev, p_x, kind, ldx = _rows_of("x", x.flatten(0, 1))
    else:
        dev, p_x, kind, ldx = _rows_of("x", x)
    cols, rows, p_src = shape[-1], shape[-2], None
    _counts(fmt)
    if not (-64 <= scale_exp <= 64 and 1 <= src_div < 1 << 31):
        _refuse(f"scale_exp={scale_exp} outside [-64, 64], or src_div={src_div} below 1 or past 32 bits")
    if src_rows is not None:
        if not grouped:
            _refuse("src_rows without offsets")
        rows = _length("src_rows", src_rows)
        p_src = _tensor("src_rows", src_rows, _I32, (rows,), dev)
    codes_shape = shape[:-2] + (rows, cols // 2)
    n_groups = p_off = None
    if grouped:
        n_groups = _length("offsets", offsets) - 1
        p_off = _tensor("offsets", offsets, _I32, (n_groups + 1,), dev)
    if out is None:
        mats, device = shape[0] if len(shape) == 3 else 1, x.device
        n = fp4_scale_bytes(fmt, mats, rows, cols, n_groups)
        out = Fp4._new(fmt, codes_shape, n, scale_exp, offsets, n_groups or 0, device, mats, rows, cols)
    elif out._fmt != fmt or out._shape != codes_shape or out._device != x.device:
        _refuse(f"out holds {tuple(out._shape)} of format {out._fmt} on {out._device}")
    else:
        out._groups_of(offsets)
    if grouped:
        rc = lib().clover_quantize_fp4_rows(fmt, p_x, kind, ldx, shape[0], cols, scale_exp, p_src, src_div, rows, p_off,
                                            n_groups, *out._pointers(), _current_stream(dev))
    else:
        rc = lib().clover_quantize_fp4(fmt, p_x, kind, ldx, out._mats, rows, cols, scale_exp, *out._pointers(),
                                       _current_stream(dev))
    if rc != OK:
        _check(rc)
    out._offsets, out._groups, out.scale_exp = offsets, n_groups or 0, scale_exp
    return out


def dequantize_fp4(q: Fp4, out=None, stream=None):
    """The bf16 matrices the codes stand for (rows behind the last group left as they were)."""
    if stream is not None:
        with _as_current(stream, q):
            return dequantize_fp4(q, out)
    off = q._offsets
    dev = _on_current("q", q._codes)
    shape = q._shape[:-1] + (q._cols,)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q._device)
        p_out = out.data_ptr()
    else:
        p_out = _tensor("out", out, _BF16, shape, dev)
    rc = lib().clover_dequantize_fp4(q._fmt, *q._pointers(), q._mats, q._rows, q._cols, q.scale_exp,
                                     None if off is None else off.data_ptr(), q._groups, p_out, _current_stream(dev))
    if rc != OK:
        _check(rc)
    return out


def fp4_product_workspace_bytes() -> int:
    return lib().clover_fp4_product_workspace_bytes()


def _shared_workspace():
    """(pointer, bytes) of the library's own workspace for products on the current device."""
    p = ctypes.c_void_p()
    rc = lib().clover_fp4_product_shared_workspace(ctypes.byref(p))
    if rc != OK:
        _check(rc)
    return p.value, 256


def fp4_product_status(stream=None):
    """Synchronises the stream, then raises CloverError if a wait ran out in an `fp4_product` without ws on the current
    device since the last look (rows of its result are then missing)."""
    _check(lib().clover_workspace_status(*_shared_workspace(), _stream(stream)))


def fp4_product(a: Fp4, b: Fp4, swiglu: bool = False, alpha: float = 1.0, group_alpha=None, ws=None, out=None,
                stream=None):
    """Rows of `a` times the matrix of their group (a.offsets; without offsets one group of all rows): bf16
    [rows][N], or with swiglu silu(gate) * up, [rows][N / 2]. b holds one [N][cols] matrix per group, or with swiglu two
    of N / 2 rows (gate, up). The result is scaled by alpha, group_alpha (fp32 [groups]) and both operands' scale_exp;
    rows behind the last group are left as they were. ws (fp4_product_workspace_bytes(); calls may share it) holds the status
    that workspace_status reads; without one it is fp4_product_status that does."""
    if stream is not None:
        with _as_current(stream, a):
            return fp4_product(a, b, swiglu, alpha, group_alpha, ws, out)
    off, per = a._offsets, 2 if swiglu else 1
    dev = _on_current("a", a._codes)
    if len(a._shape) != 2 or b._offsets is not None:
        _refuse("a must be one matrix, and only its rows may form groups")
    if a._fmt != b._fmt or a._cols != b._cols or b._device != a._device:
        _refuse(f"a (format {a._fmt}, {a._cols} columns, {a._device}) does not match b (format {b._fmt}, {b._cols} columns, "
                f"{b._device})")
    rows, width = a._rows, b._rows
    groups = 1 if off is None else a._groups
    if b._mats != groups * per:
        _refuse(f"b holds {b._mats} matrices for {groups} groups, {per} each")
    if out is None:
        out = torch.empty((rows, width), dtype=_BF16, device=a._device)
        p_out = out.data_ptr()
    else:
        p_out = _tensor("out", out, _BF16, (rows, width), dev)
    p_alpha = None if group_alpha is None else _tensor("group_alpha", group_alpha, _F32, (groups,), dev)
    try:
        factor = alpha * 2.0 ** (a.scale_exp + b.scale_exp)
    except OverflowError:
        _refuse(f"alpha {alpha} and scale exponents {a.scale_exp}, {b.scale_exp}: past the largest number")
    rc = lib().clover_fp4_product(a._fmt, *a._pointers(), rows, *b._pointers(), None if off is None else off.data_ptr(),
                                  groups, width * per, a._cols, factor, p_alpha, int(swiglu), p_out,
                                  *(_shared_workspace() if ws is None else _scratch(ws, dev)), _current_stream(dev))
    if rc != OK:
        _check(rc)
    return out


def moe_combine(y, pos, w, x=None, shared=None, out=None, stream=None):
    """x + sum_k w[:, k] * y[pos[:, k]] + shared, fp32 [M][H]: y bf16 [rows][H], pos int32 and w fp32 [M][K] as `route`
    gives them, x fp32 and shared bf16 [M][H] or None. out may be x itself."""
    if stream is not None:
        with _as_current(stream, y):
            return moe_combine(y, pos, w, x, shared, out)
    if y.dim() != 2 or pos.dim() != 2 or max(y.shape + pos.shape) > 1 << 29:
        _refuse(f"y and pos must be matrices of at most 2^29 rows, got {tuple(y.shape)} and {tuple(pos.shape)}")
    dev = _on_current("y", y)
    slots, y_shape = pos.shape, y.shape
    (M, K), (n, H) = slots, y_shape
    full = (M, H)
    if out is None:
        out = torch.empty(full, dtype=_F32, device=y.device)
        p_out = out.data_ptr()
    else:
        p_out = _tensor("out", out, _F32, full, dev)
    rc = lib().clover_moe_combine(_tensor("y", y, _BF16, y_shape, dev), n, _tensor("pos", pos, _I32, slots, dev),
                                  _tensor("w", w, _F32, slots, dev),
                                  None if shared is None else _tensor("shared", shared, _BF16, full, dev),
                                  None if x is None else _tensor("x", x, _F32, full, dev), p_out, M, K, H,
                                  _current_stream(dev))
    if rc != OK:
        _check(rc)
    return out

"""ctypes binding of libmoe_b200.so (argument marshalling only).

Every function here checks shapes, dtypes and devices of torch tensors, passes
their device pointers and the current CUDA stream to the C ABI of the same
name, and turns a non-zero return code into MoeError. All computation happens
in the library's CUDA kernels; there is no other implementation to fall back
to, so a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_NO_DEVICE = range(6)
MOE_STATUS_NAN_LOGIT, MOE_STATUS_BAD_ROUTE, MOE_STATUS_TIMEOUT = 1, 2, 4
MOE_STATUS_MX_SATURATED, MOE_STATUS_MX_UNDERFLOW, MOE_STATUS_BAD_OFFSETS = 8, 16, 32
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_SILU = 0, 1, 2, 3, 4
MOE_PRODUCT_FORWARD, MOE_PRODUCT_DGRAD, MOE_PRODUCT_WGRAD = 0, 1, 2
MOE_FORM_FEW_ROWS, MOE_FORM_SINGLE, MOE_FORM_PAIR, MOE_FORM_SPLIT = 0, 1, 2, 3
MOE_PRECISION_BF16, MOE_PRECISION_MXFP8 = 0, 1
MOE_COMBINE_AUTO, MOE_COMBINE_SEPARATE, MOE_COMBINE_FUSED = 0, 1, 2
MOE_PREACT_RECOMPUTE, MOE_PREACT_SAVE = 0, 1
MOE_DTYPE_BF16, MOE_DTYPE_F32 = 0, 1
MOE_EXPERT_SWIGLU, MOE_EXPERT_IDENTITY, MOE_EXPERT_SCALE = 0, 1, 2
MOE_OP_ROUTE, MOE_OP_PERMUTE, MOE_OP_GROUPED_FFN, MOE_OP_LAYER, MOE_OP_BACKWARD = 0, 1, 2, 3, 4
MOE_GEMM_TILES_AUTO, MOE_GEMM_TILES_SINGLE, MOE_GEMM_TILES_PAIR = 0, 1, 2
MOE_LAYOUT_COMPACT, MOE_LAYOUT_PADDED = 0, 1
MOE_DISPATCH_AUTO, MOE_DISPATCH_COPY, MOE_DISPATCH_GATHER = 0, 1, 2
MOE_MAX_E, MOE_MAX_K, MOE_PACK_BLOCK = 256, 8, 128

EXPORTED = ("moe_workspace_size", "moe_status_string", "moe_version", "moe_pack_weights", "moe_route",
            "moe_permute", "moe_grouped_ffn", "moe_unpermute_combine", "moe_layer_forward",
            "moe_permute_static_scratch", "moe_layer_forward_timed", "moe_pack_weights_backward",
            "moe_layer_backward", "moe_mxfp8_quantize", "moe_mxfp8_weights_size", "moe_pack_weights_mxfp8",
            "moe_debug_stall_next_gemms", "moe_gemm_tiles_used", "moe_grouped_gemm", "moe_grouped_gemm_dgrad",
            "moe_grouped_gemm_wgrad", "moe_linear", "moe_linear_dgrad", "moe_linear_wgrad", "moe_act_backward",
            "moe_dropout", "moe_unpermute_combine_dropout", "moe_product_form_used")


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn} failed: {text} (code {code})")
        self.code = code


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("dtype", ctypes.c_int32), ("expert_kind", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("gemm_tiles", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("dispatch", ctypes.c_int32), ("precision", ctypes.c_int32), ("combine", ctypes.c_int32),
                ("preact", ctypes.c_int32)]

    def __repr__(self):
        return "MoeConfig(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"

    @property
    def torch_dtype(self):
        return torch.bfloat16 if self.dtype == MOE_DTYPE_BF16 else torch.float32


class MoeGemmConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64),
                ("w_stride", ctypes.c_int64), ("ldy", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("ldz", ctypes.c_int64)]


_lib = None
_lock = threading.Lock()

P = ctypes.c_void_p
I32 = ctypes.c_int32
SZ = ctypes.c_size_t
CFG = ctypes.POINTER(MoeConfig)
GCFG = ctypes.POINTER(MoeGemmConfig)
I64 = ctypes.c_int64
U64 = ctypes.c_uint64
F64 = ctypes.c_double

_SIGS = {
    "moe_workspace_size": (SZ, [CFG, I32]),
    "moe_status_string": (ctypes.c_char_p, [I32]),
    "moe_version": (I32, []),
    "moe_gemm_tiles_used": (I32, [CFG, P]),
    "moe_pack_weights": (I32, [CFG, P, P, P, P]),
    "moe_route": (I32, [CFG, P, P, P, P, P, P, P, SZ, P, P]),
    "moe_permute": (I32, [CFG, P, P, P, P, P, P, P, P, P, SZ, P, P]),
    "moe_grouped_ffn": (I32, [CFG, P, P, P, P, P, P, SZ, P, P]),
    "moe_unpermute_combine": (I32, [CFG, P, P, P, P, P, P]),
    "moe_layer_forward": (I32, [CFG, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P]),
    "moe_permute_static_scratch": (I32, [CFG, P, P, P, P, P, P, P, P, P, P]),
    "moe_layer_forward_timed": (I32, [CFG, P, P, P, P, P, P, P, P, P, P, P, SZ, P, P, P]),
    "moe_pack_weights_backward": (I32, [CFG, P, P, P, P, P]),
    "moe_layer_backward": (I32, [CFG, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P, SZ, P, P]),
    "moe_mxfp8_quantize": (I32, [P, I32, I32, P, P, P, P, P]),
    "moe_mxfp8_weights_size": (SZ, [CFG, I32]),
    "moe_pack_weights_mxfp8": (I32, [CFG, P, P, P, P, P, P]),
    "moe_debug_stall_next_gemms": (I32, [I32]),
    "moe_grouped_gemm": (I32, [GCFG, P, P, P, P, P, P, P, P, P]),
    "moe_grouped_gemm_dgrad": (I32, [GCFG, P, P, P, P, P, P, P, P]),
    "moe_grouped_gemm_wgrad": (I32, [GCFG, P, P, P, P, P, P, P]),
    "moe_linear": (I32, [GCFG, P, P, P, P, P, P, P, P]),
    "moe_linear_dgrad": (I32, [GCFG, P, P, P, P, P, P, P]),
    "moe_linear_wgrad": (I32, [GCFG, P, P, P, P, P, P]),
    "moe_act_backward": (I32, [GCFG, P, P, P, P]),
    "moe_dropout": (I32, [I32, I32, I32, P, I64, P, I64, P, I64, F64, P, U64, P]),
    "moe_product_form_used": (I32, [GCFG, I32, I32, P]),
    "moe_unpermute_combine_dropout": (I32, [CFG, P, P, P, P, F64, P, U64, P, P]),
}


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                                   "`python -m combine_router_gemm_softmax_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGS.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def config(T, d, E, k, d_ff, dtype="bf16", expert_kind="swiglu", capacity=-1, gemm_tiles="auto",
           layout="compact", dispatch="auto", precision="bf16", combine="auto", preact="recompute") -> MoeConfig:
    dt = {"bf16": MOE_DTYPE_BF16, "f32": MOE_DTYPE_F32, torch.bfloat16: MOE_DTYPE_BF16,
          torch.float32: MOE_DTYPE_F32}[dtype]
    kind = {"swiglu": MOE_EXPERT_SWIGLU, "identity": MOE_EXPERT_IDENTITY, "scale": MOE_EXPERT_SCALE}[expert_kind]
    tiles = {"auto": MOE_GEMM_TILES_AUTO, "single": MOE_GEMM_TILES_SINGLE, "pair": MOE_GEMM_TILES_PAIR}[gemm_tiles]
    lay = {"compact": MOE_LAYOUT_COMPACT, "padded": MOE_LAYOUT_PADDED}[layout]
    disp = {"auto": MOE_DISPATCH_AUTO, "copy": MOE_DISPATCH_COPY, "gather": MOE_DISPATCH_GATHER}[dispatch]
    prec = {"bf16": MOE_PRECISION_BF16, "mxfp8": MOE_PRECISION_MXFP8}[precision]
    comb = {"auto": MOE_COMBINE_AUTO, "separate": MOE_COMBINE_SEPARATE, "fused": MOE_COMBINE_FUSED}[combine]
    pre = {"recompute": MOE_PREACT_RECOMPUTE, "save": MOE_PREACT_SAVE}[preact]
    return MoeConfig(T, d, E, k, d_ff, dt, kind, capacity, tiles, lay, disp, prec, comb, pre)


def perm_rows(cfg) -> int:
    """Rows P of x_perm, y_perm and perm_src: T*k, or E*capacity in the padded layout."""
    return cfg.E * cfg.capacity if cfg.layout == MOE_LAYOUT_PADDED else cfg.T * cfg.k


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _check(t, shape, dtype, name):
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _rc(fn, code):
    if code != MOE_OK:
        raise MoeError(fn, code, lib().moe_status_string(code).decode())


def _dev(ref):
    return ref.device


def _check_expert_weights(cfg, w13, w_down):
    """bf16: w13_packed [E, 2F, d] and w_down [E, d, F]; MXFP8: the two uint8
    blobs of moe_pack_weights_mxfp8."""
    if cfg.precision == MOE_PRECISION_MXFP8:
        _check(w13, (moe_mxfp8_weights_size(cfg, 0),), torch.uint8, "w13 MXFP8 blob")
        _check(w_down, (moe_mxfp8_weights_size(cfg, 1),), torch.uint8, "w_down MXFP8 blob")
    else:
        _check(w13, (cfg.E, 2 * cfg.d_ff, cfg.d), cfg.torch_dtype, "w13_packed")
        _check(w_down, (cfg.E, cfg.d, cfg.d_ff), cfg.torch_dtype, "w_down")


def moe_workspace_size(cfg: MoeConfig, op: int) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(cfg), op))


def moe_gemm_tiles_used(cfg: MoeConfig) -> int:
    """MOE_GEMM_TILES_SINGLE or MOE_GEMM_TILES_PAIR: the grouped GEMMs' tile
    shape for cfg with AUTO resolved (host only)."""
    tiles = ctypes.c_int32(-1)
    _rc("moe_gemm_tiles_used", lib().moe_gemm_tiles_used(ctypes.byref(cfg), ctypes.byref(tiles)))
    return tiles.value


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream` (None: the current one). On another
    stream than the current one it comes from that stream's memory, where no
    earlier work of the current stream is still due, and is not handed out
    again before the current stream is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if current != stream:
        t.record_stream(current)
    return t


def workspace(cfg: MoeConfig, op: int, device, stream=None) -> torch.Tensor:
    """Memory for one `op` at a time; stream: another stream than the current one that the op will run on."""
    n = moe_workspace_size(cfg, op)
    return _empty((max(n, 256),), torch.uint8, device, stream)


def moe_pack_weights(cfg, w_gate, w_up, w13_packed=None, stream=None):
    dt = cfg.torch_dtype
    _check(w_gate, (cfg.E, cfg.d_ff, cfg.d), dt, "w_gate")
    _check(w_up, (cfg.E, cfg.d_ff, cfg.d), dt, "w_up")
    if w13_packed is None:
        w13_packed = _empty((cfg.E, 2 * cfg.d_ff, cfg.d), dt, _dev(w_gate), stream)
    _check(w13_packed, (cfg.E, 2 * cfg.d_ff, cfg.d), dt, "w13_packed")
    _rc("moe_pack_weights", lib().moe_pack_weights(ctypes.byref(cfg), _ptr(w_gate), _ptr(w_up), _ptr(w13_packed),
                                                   _stream(stream)))
    return w13_packed


def moe_route(cfg, h, w_router, bias=None, logits_out=None, topk_idx=None, topk_gate=None, status=None,
              stream=None):
    dt = cfg.torch_dtype
    dev = _dev(h)
    _check(h, (cfg.T, cfg.d), dt, "h")
    _check(w_router, (cfg.E, cfg.d), dt, "w_router")
    _check(bias, (cfg.E,), torch.float32, "bias")
    _check(logits_out, (cfg.T, cfg.E), torch.float32, "logits_out")
    if topk_idx is None:
        topk_idx = _empty((cfg.T, cfg.k), torch.int32, dev, stream)
    if topk_gate is None:
        topk_gate = _empty((cfg.T, cfg.k), torch.float32, dev, stream)
    _check(topk_idx, (cfg.T, cfg.k), torch.int32, "topk_idx")
    _check(topk_gate, (cfg.T, cfg.k), torch.float32, "topk_gate")
    _rc("moe_route", lib().moe_route(ctypes.byref(cfg), _ptr(h), _ptr(w_router), _ptr(bias), _ptr(logits_out),
                                     _ptr(topk_idx), _ptr(topk_gate), None, 0, _ptr(status), _stream(stream)))
    return topk_idx, topk_gate


def moe_permute(cfg, h, topk_idx, out=None, ws=None, status=None, stream=None):
    """Returns dict routed_counts, counts, offsets, dest_row, perm_src, x_perm."""
    dt = cfg.torch_dtype
    dev = _dev(h)
    A = perm_rows(cfg)
    _check(h, (cfg.T, cfg.d), dt, "h")
    _check(topk_idx, (cfg.T, cfg.k), torch.int32, "topk_idx")
    if out is None:
        out = dict(routed_counts=_empty(cfg.E, torch.int32, dev, stream),
                   counts=_empty(cfg.E, torch.int32, dev, stream),
                   offsets=_empty(cfg.E + 1, torch.int32, dev, stream),
                   dest_row=_empty((cfg.T, cfg.k), torch.int32, dev, stream),
                   perm_src=_empty(max(A, 1), torch.int32, dev, stream),
                   x_perm=_empty((max(A, 1), cfg.d), dt, dev, stream))
    if ws is None:
        ws = workspace(cfg, MOE_OP_PERMUTE, dev, stream)
    _rc("moe_permute", lib().moe_permute(
        ctypes.byref(cfg), _ptr(h), _ptr(topk_idx), _ptr(out["routed_counts"]), _ptr(out["counts"]),
        _ptr(out["offsets"]), _ptr(out["dest_row"]), _ptr(out["perm_src"]), _ptr(out["x_perm"]), _ptr(ws),
        ws.numel(), _ptr(status), _stream(stream)))
    return out


def moe_grouped_ffn(cfg, x_perm, offsets, w13_packed=None, w_down=None, y_perm=None, ws=None, status=None,
                    stream=None):
    dt = cfg.torch_dtype
    dev = _dev(x_perm)
    rows = x_perm.shape[0]
    if rows < max(perm_rows(cfg), 1):
        raise ValueError("x_perm needs perm_rows(cfg) rows")
    _check(offsets, (cfg.E + 1,), torch.int32, "offsets")
    if cfg.expert_kind == MOE_EXPERT_SWIGLU:
        _check_expert_weights(cfg, w13_packed, w_down)
    if y_perm is None:
        y_perm = _empty((rows, cfg.d), dt, dev, stream)
    if ws is None:
        ws = workspace(cfg, MOE_OP_GROUPED_FFN, dev, stream)
    _rc("moe_grouped_ffn", lib().moe_grouped_ffn(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(w13_packed), _ptr(w_down), _ptr(y_perm), _ptr(ws),
        ws.numel(), _ptr(status), _stream(stream)))
    return y_perm


def moe_unpermute_combine(cfg, y_perm, dest_row, topk_gate, y=None, status=None, stream=None):
    dt = cfg.torch_dtype
    _check(dest_row, (cfg.T, cfg.k), torch.int32, "dest_row")
    _check(topk_gate, (cfg.T, cfg.k), torch.float32, "topk_gate")
    if y is None:
        y = _empty((cfg.T, cfg.d), dt, _dev(y_perm), stream)
    _check(y, (cfg.T, cfg.d), dt, "y")
    _rc("moe_unpermute_combine", lib().moe_unpermute_combine(
        ctypes.byref(cfg), _ptr(y_perm), _ptr(dest_row), _ptr(topk_gate), _ptr(y), _ptr(status), _stream(stream)))
    return y


def moe_layer_forward(cfg, h, w_router, bias=None, w13_packed=None, w_down=None, y=None, topk_idx=None,
                      topk_gate=None, routed_counts=None, counts=None, ws=None, status=None, stream=None,
                      stage_events=None):
    """The whole layer; returns y. stage_events: None, or 5 torch.cuda.Event
    (or None) recorded before the router and after the router, the dispatch,
    the expert stage and the combine (moe_layer_forward_timed)."""
    dt = cfg.torch_dtype
    dev = _dev(h)
    _check(h, (cfg.T, cfg.d), dt, "h")
    _check(w_router, (cfg.E, cfg.d), dt, "w_router")
    _check(bias, (cfg.E,), torch.float32, "bias")
    if cfg.expert_kind == MOE_EXPERT_SWIGLU:
        _check_expert_weights(cfg, w13_packed, w_down)
    _check(topk_idx, (cfg.T, cfg.k), torch.int32, "topk_idx")
    _check(topk_gate, (cfg.T, cfg.k), torch.float32, "topk_gate")
    _check(routed_counts, (cfg.E,), torch.int32, "routed_counts")
    _check(counts, (cfg.E,), torch.int32, "counts")
    if y is None:
        y = _empty((cfg.T, cfg.d), dt, dev, stream)
    _check(y, (cfg.T, cfg.d), dt, "y")
    if ws is None:
        ws = workspace(cfg, MOE_OP_LAYER, dev, stream)
    args = (ctypes.byref(cfg), _ptr(h), _ptr(w_router), _ptr(bias), _ptr(w13_packed), _ptr(w_down), _ptr(y),
            _ptr(topk_idx), _ptr(topk_gate), _ptr(routed_counts), _ptr(counts), _ptr(ws), ws.numel(), _ptr(status),
            _stream(stream))
    if stage_events is None:
        _rc("moe_layer_forward", lib().moe_layer_forward(*args))
        return y
    if len(stage_events) != 5:
        raise ValueError("stage_events needs 5 entries")
    handles = (ctypes.c_void_p * 5)(*[None if e is None else _event_handle(e) for e in stage_events])
    _rc("moe_layer_forward_timed", lib().moe_layer_forward_timed(*args, handles))
    return y


def _event_handle(ev):
    """Raw cudaEvent_t of a torch.cuda.Event; torch creates the event on its
    first record, so an event that was never recorded is recorded once here."""
    if not ev.cuda_event:
        ev.record()
    return ctypes.c_void_p(ev.cuda_event)


def moe_permute_static_scratch(cfg, h, topk_idx, out=None, status=None, stream=None):
    """moe_permute without a workspace argument, for callers that cannot
    allocate device memory; the library keeps the scratch in a fixed 1 MiB
    device array shared by all calls (calls that overlap on the GPU race).
    Returns the same dict as moe_permute."""
    dt = cfg.torch_dtype
    dev = _dev(h)
    A = perm_rows(cfg)
    _check(h, (cfg.T, cfg.d), dt, "h")
    _check(topk_idx, (cfg.T, cfg.k), torch.int32, "topk_idx")
    if out is None:
        out = dict(routed_counts=_empty(cfg.E, torch.int32, dev, stream),
                   counts=_empty(cfg.E, torch.int32, dev, stream),
                   offsets=_empty(cfg.E + 1, torch.int32, dev, stream),
                   dest_row=_empty((cfg.T, cfg.k), torch.int32, dev, stream),
                   perm_src=_empty(max(A, 1), torch.int32, dev, stream),
                   x_perm=_empty((max(A, 1), cfg.d), dt, dev, stream))
    _rc("moe_permute_static_scratch", lib().moe_permute_static_scratch(
        ctypes.byref(cfg), _ptr(h), _ptr(topk_idx), _ptr(out["routed_counts"]), _ptr(out["counts"]),
        _ptr(out["offsets"]), _ptr(out["dest_row"]), _ptr(out["perm_src"]), _ptr(out["x_perm"]), _ptr(status),
        _stream(stream)))
    return out


def moe_pack_weights_backward(cfg, w13_packed, w_down, stream=None):
    """Per-expert transposes for the backward dgrad GEMMs: returns
    (w13_t [E, d, 2F], w_down_t [E, F, d])."""
    dt = cfg.torch_dtype
    dev = _dev(w13_packed)
    _check(w13_packed, (cfg.E, 2 * cfg.d_ff, cfg.d), dt, "w13_packed")
    _check(w_down, (cfg.E, cfg.d, cfg.d_ff), dt, "w_down")
    w13_t = _empty((cfg.E, cfg.d, 2 * cfg.d_ff), dt, dev, stream)
    w_down_t = _empty((cfg.E, cfg.d_ff, cfg.d), dt, dev, stream)
    _rc("moe_pack_weights_backward", lib().moe_pack_weights_backward(
        ctypes.byref(cfg), _ptr(w13_packed), _ptr(w_down), _ptr(w13_t), _ptr(w_down_t), _stream(stream)))
    return w13_t, w_down_t


def moe_layer_backward(cfg, h, w_router, w13_packed, w13_t, w_down_t, dy, fwd_ws, with_bias=True, ws=None,
                       status=None, stream=None):
    """Gradients of <dy, y> for the moe_layer_forward call that last used
    fwd_ws. Returns dict dh [T,d] (bf16), dw_router [E,d], dbias [E] (or None),
    dw13 [E,2F,d] (packed row order), dw_down [E,d,F] (fp32)."""
    dt = cfg.torch_dtype
    dev = _dev(h)
    _check(h, (cfg.T, cfg.d), dt, "h")
    _check(w_router, (cfg.E, cfg.d), dt, "w_router")
    _check(w13_packed, (cfg.E, 2 * cfg.d_ff, cfg.d), dt, "w13_packed")
    _check(w13_t, (cfg.E, cfg.d, 2 * cfg.d_ff), dt, "w13_t")
    _check(w_down_t, (cfg.E, cfg.d_ff, cfg.d), dt, "w_down_t")
    _check(dy, (cfg.T, cfg.d), dt, "dy")
    out = dict(dh=_empty((cfg.T, cfg.d), dt, dev, stream),
               dw_router=_empty((cfg.E, cfg.d), torch.float32, dev, stream),
               dbias=_empty(cfg.E, torch.float32, dev, stream) if with_bias else None,
               dw13=_empty((cfg.E, 2 * cfg.d_ff, cfg.d), torch.float32, dev, stream),
               dw_down=_empty((cfg.E, cfg.d, cfg.d_ff), torch.float32, dev, stream))
    if ws is None:
        ws = workspace(cfg, MOE_OP_BACKWARD, dev, stream)
    _rc("moe_layer_backward", lib().moe_layer_backward(
        ctypes.byref(cfg), _ptr(h), _ptr(w_router), _ptr(w13_packed), _ptr(w13_t), _ptr(w_down_t), _ptr(dy),
        _ptr(out["dh"]), _ptr(out["dw_router"]), _ptr(out["dbias"]), _ptr(out["dw13"]), _ptr(out["dw_down"]),
        _ptr(fwd_ws), fwd_ws.numel(), _ptr(ws), ws.numel(), _ptr(status), _stream(stream)))
    return out


def moe_mxfp8_weights_size(cfg, which: int) -> int:
    """Bytes of the MXFP8 weight blob: which 0 = w13, 1 = w_down."""
    return int(lib().moe_mxfp8_weights_size(ctypes.byref(cfg), which))


def mxfp8_scale_bytes(rows, cols) -> int:
    """Bytes of the scale atoms moe_mxfp8_quantize writes for [rows, cols]."""
    return (cols // 128) * ((rows + 127) // 128) * 512


def moe_mxfp8_quantize(x, q=None, sf=None, counts=None, status=None, stream=None):
    """MXFP8 quantisation of a bf16 matrix [rows, cols] along its rows.
    Returns (q [rows, cols] uint8 E4M3 bytes, sf uint8 scale atoms);
    counts (uint32 [2], may be None) receives the saturated and underflowed
    element counts added."""
    if x.dim() != 2 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bf16 tensor")
    rows, cols = x.shape
    dev = _dev(x)
    if q is None:
        q = _empty((rows, cols), torch.uint8, dev, stream)
    if sf is None:
        sf = _empty(max(mxfp8_scale_bytes(rows, cols), 1), torch.uint8, dev, stream)
        with torch.cuda.stream(stream):
            sf.zero_()
    _check(q, (rows, cols), torch.uint8, "q")
    if sf.numel() < mxfp8_scale_bytes(rows, cols) or sf.dtype != torch.uint8:
        raise ValueError("sf too small")
    if counts is not None and (counts.dtype != torch.int32 or counts.numel() < 2):
        raise ValueError("counts must be int32 with 2 entries (read as uint32)")
    _rc("moe_mxfp8_quantize", lib().moe_mxfp8_quantize(_ptr(x), rows, cols, _ptr(q), _ptr(sf), _ptr(counts),
                                                       _ptr(status), _stream(stream)))
    return q, sf


def moe_pack_weights_mxfp8(cfg, w13_packed, w_down, counts=None, stream=None):
    """Quantise the expert weights for MOE_PRECISION_MXFP8. Returns the two
    uint8 blobs (w13_mx, w_down_mx)."""
    _check(w13_packed, (cfg.E, 2 * cfg.d_ff, cfg.d), torch.bfloat16, "w13_packed")
    _check(w_down, (cfg.E, cfg.d, cfg.d_ff), torch.bfloat16, "w_down")
    dev = _dev(w13_packed)
    a = _empty(moe_mxfp8_weights_size(cfg, 0), torch.uint8, dev, stream)
    b = _empty(moe_mxfp8_weights_size(cfg, 1), torch.uint8, dev, stream)
    _rc("moe_pack_weights_mxfp8", lib().moe_pack_weights_mxfp8(ctypes.byref(cfg), _ptr(w13_packed), _ptr(w_down),
                                                               _ptr(a), _ptr(b), _ptr(counts), _stream(stream)))
    return a, b


def mx_counters(ws):
    """The four uint32 counters an MXFP8 call leaves at the start of its
    workspace: x saturated, x underflowed, h_mid saturated, h_mid underflowed."""
    return ws[:16].view(torch.int32).cpu().tolist()


# ------------------------------------------------------------------ free products and dropout

_ACTS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "gelu": MOE_ACT_GELU, "gelu_tanh": MOE_ACT_GELU_TANH,
         "silu": MOE_ACT_SILU}
_GEMM_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_F32}


def _act(act) -> int:
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"act: {act!r} is none of {', '.join(_ACTS)}") from None


def _refuse(t, shape, dtype, index, name):
    """The error of a tensor that is not `shape` of `dtype` on device `index`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    raise ValueError(f"{name}: on {t.device}, not on {torch.device('cuda', index) if index >= 0 else 'cpu'}")


def _strided(t, shape, dtype, index, name):
    """Checks a matrix whose rows may lie apart (unit stride along the last
    axis) and returns its address and row stride; (None, 0) for None."""
    if t is None:
        return None, 0
    try:
        wrong = t.shape != shape or t.dtype is not dtype or t.get_device() != index
    except AttributeError:  # no tensor
        wrong = True
    if wrong:
        _refuse(t, shape, dtype, index, name)
    st = t.stride()
    width = shape[-1]
    ld = st[-2] if shape[-2] > 1 else (width + 7) // 8 * 8  # a single row's stride leads nowhere
    if (st[-1] != 1 and width > 1) or ld < width:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap (strides {st})")
    return t.data_ptr(), ld


def _matrix(rows, width, dtype, device, stream):
    """A new matrix whose rows start on 16 bytes (odd widths get padded rows)."""
    wide = (width + 7) // 8 * 8
    t = _empty((rows, wide), dtype, device, stream)
    return t if wide == width else t[:, :width]


def _plain(t, shape, dtype, index, name):
    """Address of a contiguous tensor of this shape; None for None."""
    if t is None:
        return None
    try:
        wrong = t.shape != shape or t.dtype is not dtype or t.get_device() != index
    except AttributeError:  # no tensor
        wrong = True
    if wrong:
        _refuse(t, shape, dtype, index, name)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _axes(t, dims, name):
    try:
        have = t.dim()
    except AttributeError:
        raise TypeError(f"{name}: expected a torch.Tensor") from None
    if have != dims:
        raise ValueError(f"{name}: {have} axes, not {dims}")


def _first(t, dims, name):
    """Device index and MOE_DTYPE_* of a call's leading operand."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name}: must be on a CUDA device")
    _axes(t, dims, name)
    try:
        return index, _GEMM_DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{name}: dtype {t.dtype} is neither bfloat16 nor float32") from None


def _enqueue(fn, index, stream, *args):
    """Calls the entry point on `stream` (default: the device's current one),
    with the tensors' device current."""
    f = getattr(_lib or lib(), fn)
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        code = f(*args, raw)
    else:
        with torch.cuda.device(index):
            code = f(*args, raw)
    if code != MOE_OK:
        _rc(fn, code)


def _weights(w, groups, n, k, dtype, index):
    """Address, row stride and group stride of w [groups, n, k] (or [n, k])."""
    p, ld = _strided(w, (groups, n, k) if w.dim() == 3 else (n, k), dtype, index, "w")
    if groups <= 1:
        return p, ld, n * ld
    between = w.stride(0)
    if between < (n - 1) * ld + k:
        raise ValueError(f"w: groups must not overlap (strides {w.stride()})")
    return p, ld, between


def _forward(fn, dims, x, offsets, w, bias, act, residual, preact, y, status, stream):
    dev, dt = _first(x, 2, "x")
    _axes(w, dims, "w")
    rows, k = x.shape
    shape = w.shape
    n = shape[-2]
    groups = shape[0] if dims == 3 else 1
    tdt = x.dtype
    out = (rows, n)
    px, ldx = _strided(x, x.shape, tdt, dev, "x")
    pw, ldw, ws = _weights(w, groups, n, k, tdt, dev)
    pb = _plain(bias, shape[:-1], torch.float32, dev, "bias") if bias is not None else None
    pr, ldr = _strided(residual, out, tdt, dev, "residual")
    pz, ldz = _strided(preact, out, tdt, dev, "preact")
    if y is None:
        y = _matrix(rows, n, tdt, x.device, stream)
    py, ldy = _strided(y, out, tdt, dev, "y")
    cfg = MoeGemmConfig(rows, n, k, groups, dt, _act(act), ldx, ldw, ws, ldy, ldr, ldz)
    ps = _plain(status, (1,), torch.int32, dev, "status")
    if dims == 2:
        _enqueue(fn, dev, stream, cfg, px, pw, pb, pr, pz, py, ps)
    else:
        _enqueue(fn, dev, stream, cfg, px, _plain(offsets, (groups + 1,), torch.int32, dev, "offsets"), pw, pb, pr, pz,
                 py, ps)
    return y


def _dgrad(fn, dims, dy, offsets, w, z, act, residual, dx, status, stream):
    dev, dt = _first(dy, 2, "dy")
    _axes(w, dims, "w")
    rows, n = dy.shape
    k = w.shape[-1]
    groups = w.shape[0] if dims == 3 else 1
    tdt = dy.dtype
    out = (rows, k)
    pdy, ldy = _strided(dy, dy.shape, tdt, dev, "dy")
    pw, ldw, ws = _weights(w, groups, n, k, tdt, dev)
    pz, ldz = _strided(z, out, tdt, dev, "z")
    pr, ldr = _strided(residual, out, tdt, dev, "residual")
    if dx is None:
        dx = _matrix(rows, k, tdt, dy.device, stream)
    pdx, ldx = _strided(dx, out, tdt, dev, "dx")
    cfg = MoeGemmConfig(rows, n, k, groups, dt, _act(act), ldx, ldw, ws, ldy, ldr, ldz)
    ps = _plain(status, (1,), torch.int32, dev, "status")
    if dims == 2:
        _enqueue(fn, dev, stream, cfg, pdy, pw, pz, pr, pdx, ps)
    else:
        _enqueue(fn, dev, stream, cfg, pdy, _plain(offsets, (groups + 1,), torch.int32, dev, "offsets"), pw, pz, pr,
                 pdx, ps)
    return dx


def _wgrad(fn, dims, dy, offsets, x, groups, dw, dbias, status, stream):
    dev, dt = _first(dy, 2, "dy")
    _first(x, 2, "x")
    rows, n = dy.shape
    k = x.shape[1]
    pdy, ldy = _strided(dy, dy.shape, dy.dtype, dev, "dy")
    px, ldx = _strided(x, (rows, k), dy.dtype, dev, "x")
    shape = (n, k) if dims == 2 else (groups, n, k)
    if dw is None:
        dw = _empty(shape, torch.float32, dy.device, stream)
    pdw = _plain(dw, shape, torch.float32, dev, "dw")
    pdb = _plain(dbias, shape[:-1], torch.float32, dev, "dbias")
    cfg = MoeGemmConfig(rows, n, k, groups, dt, MOE_ACT_NONE, ldx, 0, 0, ldy, 0, 0)
    ps = _plain(status, (1,), torch.int32, dev, "status")
    if dims == 2:
        _enqueue(fn, dev, stream, cfg, pdy, px, pdw, pdb, ps)
    else:
        _enqueue(fn, dev, stream, cfg, pdy, _plain(offsets, (groups + 1,), torch.int32, dev, "offsets"), px, pdw, pdb,
                 ps)
    return dw


def moe_grouped_gemm(x, offsets, w, bias=None, act="none", residual=None, preact=None, y=None, status=None,
                     stream=None):
    """y[r] = act(x[r] w[e]^T + bias[e]) + residual[r] for the rows r in
    [offsets[e], offsets[e+1]) of each expert e. x [rows, k], offsets [E+1]
    int32 on the device (as moe_permute writes them), w [E, n, k], bias [E, n]
    fp32; act "none", "relu", "gelu", "gelu_tanh" or "silu"; preact [rows, n]
    receives the argument of act. Rows of matrices may lie apart (bf16 row
    strides: multiples of 8). Rows outside every group are left as they were
    (uninitialised in a y made here). residual may be y; no other argument may
    share memory with an output. stream: where the call runs (default: the
    device's current one), after whatever made its arguments; other streams
    wait for it before they read its outputs. Returns y."""
    return _forward("moe_grouped_gemm", 3, x, _required(offsets, "offsets"), w, bias, act, residual, preact, y, status,
                    stream)


def moe_grouped_gemm_dgrad(dy, offsets, w, z=None, act="none", residual=None, dx=None, status=None, stream=None):
    """dx[r] = act'(z[r]) * (dy[r] w[e]) + residual[r]: the input gradient,
    through the activation x = act(z) that made the input when z [rows, k] is
    given. Returns dx [rows, k]."""
    return _dgrad("moe_grouped_gemm_dgrad", 3, dy, _required(offsets, "offsets"), w, z, act, residual, dx, status,
                  stream)


def moe_grouped_gemm_wgrad(dy, offsets, x, dw=None, dbias=None, status=None, stream=None):
    """dw[e] = dy_e^T x_e (fp32 [E, n, k], E from offsets); dbias [E, n] fp32,
    when given, receives the column sums of dy_e. Returns dw."""
    _axes(offsets, 1, "offsets")
    groups = offsets.numel() - 1
    if groups < 1:
        raise ValueError("offsets: needs E + 1 entries")
    return _wgrad("moe_grouped_gemm_wgrad", 3, dy, offsets, x, groups, dw, dbias, status, stream)


def moe_linear(x, w, bias=None, act="none", residual=None, preact=None, y=None, status=None, stream=None):
    """y = act(x w^T + bias) + residual for one dense weight w [n, k]; the
    arguments are moe_grouped_gemm's. Returns y [rows, n]."""
    return _forward("moe_linear", 2, x, None, w, bias, act, residual, preact, y, status, stream)


def moe_linear_dgrad(dy, w, z=None, act="none", residual=None, dx=None, status=None, stream=None):
    """dx = act'(z) * (dy w) + residual, see moe_grouped_gemm_dgrad."""
    return _dgrad("moe_linear_dgrad", 2, dy, None, w, z, act, residual, dx, status, stream)


def moe_linear_wgrad(dy, x, dw=None, dbias=None, status=None, stream=None):
    """dw = dy^T x (fp32 [n, k]) and, when dbias [n] is given, the column sums
    of dy. Returns dw."""
    return _wgrad("moe_linear_wgrad", 2, dy, None, x, 1, dw, dbias, status, stream)


def _required(t, name):
    if t is None:
        raise TypeError(f"{name}: expected a torch.Tensor")
    return t


_PRODUCTS = {"forward": MOE_PRODUCT_FORWARD, "dgrad": MOE_PRODUCT_DGRAD, "wgrad": MOE_PRODUCT_WGRAD}


def moe_product_form_used(product, rows, n, k, groups=1, dtype=torch.bfloat16, sms=148):
    """How a product ("forward", "dgrad" or "wgrad") of these sizes is cut up on
    a device of `sms` SMs: (MOE_FORM_*, columns of a tile, CTAs that share a
    reduction). Host only."""
    if product not in _PRODUCTS:
        raise ValueError(f"product: {product!r} is none of {', '.join(_PRODUCTS)}")
    wide = [(v + 7) // 8 * 8 for v in (k, n)]  # rows on 16 bytes, as bf16 operands have them
    cfg = MoeGemmConfig(rows, n, k, groups, _GEMM_DTYPES[dtype], MOE_ACT_NONE, wide[0], wide[0], 0, wide[1], 0, 0)
    form = (ctypes.c_int32 * 3)()
    _rc("moe_product_form_used", lib().moe_product_form_used(ctypes.byref(cfg), _PRODUCTS[product], sms, form))
    return tuple(form)


def moe_act_backward(dy, z, act, dz=None, stream=None):
    """dz = dy * act'(z) over [rows, n], for an activation that no further
    product consumes. Returns dz (which may be dy)."""
    dev, dt = _first(dy, 2, "dy")
    shape = dy.shape
    pdy, ldy = _strided(dy, shape, dy.dtype, dev, "dy")
    pz, ldz = _strided(_required(z, "z"), shape, dy.dtype, dev, "z")
    if dz is None:
        dz = _matrix(*shape, dy.dtype, dy.device, stream)
    pdz, ldr = _strided(dz, shape, dy.dtype, dev, "dz")
    cfg = MoeGemmConfig(shape[0], shape[1], 1, 1, dt, _act(act), 0, 0, 0, ldy, ldr, ldz)
    _enqueue("moe_act_backward", dev, stream, cfg, pdy, pz, pdz)
    return dz


def moe_dropout(x, p, rng=None, offset=0, residual=None, y=None, stream=None):
    """y = residual + dropout(x) over a matrix [rows, cols], bf16 or fp32. rng:
    int64 [2] on the device (seed, counter offset), added to the host's
    `offset`; the mask is a function of them and of the element's place, so
    moe_dropout(dy, p, rng, offset) is the backward. Returns y (which may be x
    or residual)."""
    dev, dt = _first(x, 2, "x")
    shape = x.shape
    px, ldx = _strided(x, shape, x.dtype, dev, "x")
    pr, ldr = _strided(residual, shape, x.dtype, dev, "residual")
    if y is None:
        y = _empty(shape, x.dtype, x.device, stream)
    py, ldy = _strided(y, shape, x.dtype, dev, "y")
    _enqueue("moe_dropout", dev, stream, shape[0], shape[1], dt, px, ldx, pr, ldr, py, ldy, p,
             _plain(rng, (2,), torch.int64, dev, "rng"), offset)
    return y


def moe_unpermute_combine_dropout(cfg, y_perm, dest_row, topk_gate, p, rng=None, offset=0, residual=None, y=None,
                                  stream=None):
    """y[t] = residual[t] + dropout(sum_j topk_gate[t, j] y_perm[dest_row[t, j]]):
    moe_unpermute_combine and moe_dropout in one pass, the sum not rounded in
    between. Returns y [T, d] (which may be residual)."""
    dev, _ = _first(y_perm, 2, "y_perm")
    dt = cfg.torch_dtype
    rows = max(perm_rows(cfg), 1)
    if y_perm.shape[0] < perm_rows(cfg) or y_perm.shape[1] != cfg.d:
        raise ValueError(f"y_perm: shape {tuple(y_perm.shape)}, needs {rows} rows of {cfg.d}")
    pp = _plain(y_perm, y_perm.shape, dt, dev, "y_perm")
    pd = _plain(_required(dest_row, "dest_row"), (cfg.T, cfg.k), torch.int32, dev, "dest_row")
    pg = _plain(_required(topk_gate, "topk_gate"), (cfg.T, cfg.k), torch.float32, dev, "topk_gate")
    pr = _plain(residual, (cfg.T, cfg.d), dt, dev, "residual")
    if y is None:
        y = _empty((cfg.T, cfg.d), dt, y_perm.device, stream)
    py = _plain(y, (cfg.T, cfg.d), dt, dev, "y")
    _enqueue("moe_unpermute_combine_dropout", dev, stream, cfg, pp, pd, pg, pr, p,
             _plain(rng, (2,), torch.int64, dev, "rng"), offset, py)
    return y

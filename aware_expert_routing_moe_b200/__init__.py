"""Python binding of libmoe_decode.so: the decode-time MoE layer with
batch-aware expert re-routing on one B200.

This module only marshals arguments: torch tensors supply device memory and
the current CUDA stream; every step of the layer runs in the library's CUDA
kernels.  There is no fallback: if the shared library is missing or was not
built for this machine, importing the binding's functions raises.

Entry points mirror the C ABI in include/moe_decode.h:
``moe_route``, ``moe_reselect``, ``moe_expert_ffn``, ``moe_layer_decode``,
``moe_workspace_bytes``, ``moe_check_error``, ``moe_status_string``; the
general router ``moe_route_scored``; the block-scaled 8-bit operators
``moe_quantize_blocks``, ``moe_expert_gemm_blocks`` and
``moe_expert_ffn_blocks``.

A call runs on ``stream`` (a torch stream or a raw handle; default: the
current stream).  Workspaces, outputs and lists that the caller leaves out are
made on that stream, as under ``torch.cuda.stream(stream)``; a workspace that
is passed is used on one stream at a time.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

__all__ = [
    "MOE_RESELECT_NONE", "MOE_RESELECT_OEA", "MOE_RESELECT_XSHARE", "MOE_RESELECT_AFFINITY",
    "MOE_RESELECT_XSHARE_HIER", "MoeError",
    "Dims", "Rule", "Lists", "load_library", "library_path", "moe_workspace_bytes",
    "moe_status_string", "moe_route", "moe_reselect", "moe_expert_ffn", "moe_layer_decode",
    "moe_check_error", "moe_expert_ffn_noalloc", "new_workspace", "alloc_lists", "ABI_SYMBOLS",
    "NOALLOC_SCRATCH_BYTES", "moe_set_wait_limit_ns", "moe_decode_stack", "LayerWeights",
    "MOE_PHASE_DECODE", "MOE_PHASE_PREFILL", "moe_down_channel_major", "moe_expert_ffn_channels",
    "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "Scoring", "BlockWeights", "moe_route_scored", "new_route_workspace",
    "moe_quantize_blocks", "moe_expert_gemm_blocks", "new_gemm_workspace", "moe_expert_ffn_blocks",
    "new_blocks_workspace", "GEMM_WORKSPACE_BYTES",
]

MOE_RESELECT_NONE, MOE_RESELECT_OEA, MOE_RESELECT_XSHARE = 0, 1, 2
MOE_RESELECT_AFFINITY, MOE_RESELECT_XSHARE_HIER = 3, 4
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_MISALIGNED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_UNSUPPORTED", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_INTERNAL"}
ABI_SYMBOLS = ("moe_workspace_bytes", "moe_route", "moe_reselect", "moe_expert_ffn",
               "moe_layer_decode", "moe_expert_ffn_noalloc", "moe_check_error", "moe_status_string",
               "moe_set_wait_limit_ns", "moe_decode_stack", "moe_down_channel_major",
               "moe_channels_workspace_bytes", "moe_expert_ffn_channels", "moe_route_workspace_bytes",
               "moe_route_scored", "moe_quantize_blocks", "moe_expert_gemm_blocks", "moe_blocks_workspace_bytes",
               "moe_expert_ffn_blocks")
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
GEMM_WORKSPACE_BYTES = 4096
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}  # moe_dtype_t

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmoe_decode.so")
_lib = None


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({moe_status_string(status)})")


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("d_ff", ctypes.c_int32)]


class Rule(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("k0", ctypes.c_int32), ("budget", ctypes.c_int32),
                ("group", ctypes.c_int32)]


class LayerWeights(ctypes.Structure):
    _fields_ = [("Wg", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("Wgate", ctypes.c_void_p),
                ("Wup", ctypes.c_void_p), ("Wdown", ctypes.c_void_p)]


class Lists(ctypes.Structure):
    _fields_ = [("n_active", ctypes.c_void_p), ("active", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("tok", ctypes.c_void_p), ("w", ctypes.c_void_p)]


class Scoring(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class BlockWeights(ctypes.Structure):
    _fields_ = [("Wgate", ctypes.c_void_p), ("Sgate", ctypes.c_void_p), ("Wup", ctypes.c_void_p),
                ("Sup", ctypes.c_void_p), ("Wdown", ctypes.c_void_p), ("Sdown", ctypes.c_void_p)]


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libmoe_decode.so (raises OSError if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise OSError(f"{_LIB_PATH} not built: run `python -m aware_expert_routing_moe_b200.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P, S = ctypes.c_void_p, ctypes.c_size_t
        lib.moe_workspace_bytes.restype = S
        lib.moe_workspace_bytes.argtypes = [Dims]
        lib.moe_status_string.restype = ctypes.c_char_p
        lib.moe_status_string.argtypes = [ctypes.c_int]
        lib.moe_route.restype = ctypes.c_int
        lib.moe_route.argtypes = [P, P, P, Dims, P, P, P, P, P]
        lib.moe_reselect.restype = ctypes.c_int
        lib.moe_reselect.argtypes = [P, P, Dims, Rule, P, P, Lists, P]
        lib.moe_expert_ffn.restype = ctypes.c_int
        lib.moe_expert_ffn.argtypes = [P, P, P, P, Dims, Lists, P, P, S, P]
        lib.moe_layer_decode.restype = ctypes.c_int
        lib.moe_layer_decode.argtypes = [P, P, P, P, P, P, Dims, Rule, P, P, P, P, P, S, P]
        lib.moe_expert_ffn_noalloc.restype = ctypes.c_int
        lib.moe_expert_ffn_noalloc.argtypes = [P, P, P, P, Dims, Lists, P, P]
        lib.moe_check_error.restype = ctypes.c_int
        lib.moe_check_error.argtypes = [P, S, P]
        lib.moe_decode_stack.restype = ctypes.c_int
        lib.moe_decode_stack.argtypes = [ctypes.POINTER(LayerWeights), ctypes.c_int32, Dims, Rule, ctypes.c_int32,
                                         P, P, P, P, S, P]
        lib.moe_down_channel_major.restype = ctypes.c_int
        lib.moe_down_channel_major.argtypes = [P, Dims, P, P]
        lib.moe_channels_workspace_bytes.restype = S
        lib.moe_channels_workspace_bytes.argtypes = [Dims]
        lib.moe_expert_ffn_channels.restype = ctypes.c_int
        lib.moe_expert_ffn_channels.argtypes = [P, P, P, P, Dims, P, P, P, ctypes.c_int32, P, P, P, S, P]
        lib.moe_route_workspace_bytes.restype = S
        lib.moe_route_workspace_bytes.argtypes = [Dims]
        lib.moe_route_scored.restype = ctypes.c_int
        lib.moe_route_scored.argtypes = [P, P, Dims, Scoring, P, P, Lists, P, S, P]
        lib.moe_quantize_blocks.restype = ctypes.c_int
        lib.moe_quantize_blocks.argtypes = [P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.c_int32, P, P, P]
        lib.moe_expert_gemm_blocks.restype = ctypes.c_int
        lib.moe_expert_gemm_blocks.argtypes = [P, P, P, P, Dims, Lists, P, ctypes.c_int32, P, S, P]
        lib.moe_blocks_workspace_bytes.restype = S
        lib.moe_blocks_workspace_bytes.argtypes = [Dims]
        lib.moe_expert_ffn_blocks.restype = ctypes.c_int
        lib.moe_expert_ffn_blocks.argtypes = [P, ctypes.c_int32, BlockWeights, Dims, Lists, P, ctypes.c_int32, P, S, P]
        lib.moe_set_wait_limit_ns.restype = None
        lib.moe_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        _lib = lib
    return _lib


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise MoeError(status, where)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)  # raw address, for boundary tests
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream, dev: int):
    """Context in which a call on `stream` makes its own tensors (workspace,
    outputs, lists).  They belong to that stream: a workspace is zero-filled
    in order with the kernels that use it, and memory that is freed while
    they run is handed to nothing but later work of the same stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)  # (ExternalStream takes 0 for a new stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def _made(stream, t, make, *args, **kwargs):
    """make(..., device=t's) for a call on `stream`."""
    if stream is None:
        return make(*args, device=t.device, **kwargs)
    with _on(stream, t.get_device()):
        return make(*args, device=t.device, **kwargs)


def _empty(stream, t, shape, dtype):
    """_made(torch.empty), short where the call is on the current stream."""
    if stream is None:
        return t.new_empty(shape, dtype=dtype)
    return _made(stream, t, torch.empty, shape, dtype=dtype)


def dims(B: int, d: int, E: int, k: int, d_ff: int) -> Dims:
    return Dims(B, d, E, k, d_ff)


def moe_workspace_bytes(B: int, d: int, E: int, k: int, d_ff: int) -> int:
    return int(load_library().moe_workspace_bytes(Dims(B, d, E, k, d_ff)))


def new_workspace(B: int, d: int, E: int, k: int, d_ff: int, device="cuda") -> torch.Tensor:
    """Zero-filled workspace (uint8) of moe_workspace_bytes() bytes."""
    n = moe_workspace_bytes(B, d, E, k, d_ff)
    if n == 0:
        raise MoeError(1, "moe_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_lists(B: int, E: int, k: int, device="cuda") -> dict:
    i32 = dict(dtype=torch.int32, device=device)
    return {"n_active": torch.empty(4, **i32), "active": torch.empty(E, **i32),
            "offsets": torch.empty(E + 1, **i32), "tok": torch.empty(B * k, **i32),
            "w": torch.empty(B * k, dtype=torch.float32, device=device)}


def _lists(l: dict) -> Lists:
    return Lists(_ptr(l["n_active"]), _ptr(l["active"]), _ptr(l["offsets"]), _ptr(l["tok"]), _ptr(l["w"]))


def moe_route(x, Wg, bias, k: int, out=None, stream=None):
    """-> (logits[B][E], probs[B][E], topk_idx[B][k], topk_w[B][k])."""
    B, d = x.shape
    E = Wg.shape[0]
    if out is None:
        out = (_made(stream, x, torch.empty, B, E, dtype=torch.float32),
               _made(stream, x, torch.empty, B, E, dtype=torch.float32),
               _made(stream, x, torch.empty, B, k, dtype=torch.int32),
               _made(stream, x, torch.empty, B, k, dtype=torch.float32))
    logits, probs, ti, tw = out
    st = load_library().moe_route(_ptr(x), _ptr(Wg), _ptr(bias), Dims(B, d, E, k, 0), _ptr(logits),
                                  _ptr(probs), _ptr(ti), _ptr(tw), _stream(stream))
    _check(st, "moe_route")
    return logits, probs, ti, tw


def moe_reselect(logits, probs, k: int, mode: int, k0: int = 0, budget: int = 0,
                 out=None, lists=None, stream=None, group: int = 1):
    """-> (sel_idx[B][k], sel_w[B][k], lists dict).  ``group``: tokens per
    request (hierarchical XShare)."""
    B, E = logits.shape
    if out is None:
        out = (_made(stream, logits, torch.empty, B, k, dtype=torch.int32),
               _made(stream, logits, torch.empty, B, k, dtype=torch.float32))
    if lists is None:
        lists = _made(stream, logits, alloc_lists, B, E, k)
    sel, w = out
    st = load_library().moe_reselect(_ptr(logits), _ptr(probs), Dims(B, 0, E, k, 0),
                                     Rule(mode, k0, budget, group),
                                     _ptr(sel), _ptr(w), _lists(lists), _stream(stream))
    _check(st, "moe_reselect")
    return sel, w, lists


def moe_expert_ffn(x, Wgate, Wup, Wdown, lists: dict, k: int, ws, y=None, stream=None):
    """-> y[B][d] fp32 (overwritten)."""
    B, d = x.shape
    E, F, _ = Wgate.shape
    if y is None:
        y = _made(stream, x, torch.empty, B, d, dtype=torch.float32)
    st = load_library().moe_expert_ffn(_ptr(x), _ptr(Wgate), _ptr(Wup), _ptr(Wdown), Dims(B, d, E, k, F),
                                       _lists(lists), _ptr(y), _ptr(ws), ws.numel() * ws.element_size()
                                       if isinstance(ws, torch.Tensor) else 0, _stream(stream))
    _check(st, "moe_expert_ffn")
    return y


def moe_layer_decode(x, Wg, bias, Wgate, Wup, Wdown, k: int, mode: int, k0: int = 0, budget: int = 0,
                     ws=None, y=None, sel_idx=None, sel_w=None, n_active=None, stream=None, group: int = 1):
    """Whole layer; -> y[B][d] fp32.  Optional device outputs sel_idx[B][k],
    sel_w[B][k], n_active[1] are filled when given."""
    B, d = x.shape
    E, F, _ = Wgate.shape
    if ws is None:
        ws = _made(stream, x, new_workspace, B, d, E, k, F)
    if y is None:
        y = _made(stream, x, torch.empty, B, d, dtype=torch.float32)
    st = load_library().moe_layer_decode(
        _ptr(x), _ptr(Wg), _ptr(bias), _ptr(Wgate), _ptr(Wup), _ptr(Wdown), Dims(B, d, E, k, F),
        Rule(mode, k0, budget, group), _ptr(y), _ptr(sel_idx), _ptr(sel_w), _ptr(n_active), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_layer_decode")
    return y


MOE_PHASE_DECODE, MOE_PHASE_PREFILL = 0, 1


def moe_decode_stack(xs, layers, k: int, mode: int, k0: int = 0, budget: int = 0, phase: int = MOE_PHASE_DECODE,
                     ws=None, sel_idx=None, n_active=None, stream=None, group: int = 1):
    """n_layers residual MoE layers: xs[l + 1] = xs[l] + layer_l(xs[l]).
    ``xs``: [n_layers + 1][B][d] fp32 device tensor, xs[0] the input;
    ``layers``: list of (Wg, bias, Wgate, Wup, Wdown) device tensors.
    Optional device outputs sel_idx[n_layers][B][k], n_active[n_layers].
    -> xs."""
    n = len(layers)
    _, B, d = xs.shape
    E, F, _ = layers[0][2].shape
    if ws is None:
        ws = _made(stream, xs, new_workspace, B, d, E, k, F)
    arr = (LayerWeights * n)(*[LayerWeights(_ptr(Wg), _ptr(bias), _ptr(g), _ptr(u), _ptr(dn))
                               for (Wg, bias, g, u, dn) in layers])
    st = load_library().moe_decode_stack(arr, n, Dims(B, d, E, k, F), Rule(mode, k0, budget, group), int(phase),
                                         _ptr(xs), _ptr(sel_idx), _ptr(n_active), _ptr(ws),
                                         ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_decode_stack")
    return xs


def moe_down_channel_major(Wdown, out=None, stream=None):
    """Channel-major copy of the down weights: out[E][d_ff][d] = Wdown[E][d][d_ff]
    transposed per expert (bf16 bits as int16/uint16 tensors)."""
    E, d, F = Wdown.shape
    if out is None:
        out = _made(stream, Wdown, torch.empty, E, F, d, dtype=Wdown.dtype)
    st = load_library().moe_down_channel_major(_ptr(Wdown), Dims(1, d, E, 1, F), _ptr(out), _stream(stream))
    _check(st, "moe_down_channel_major")
    return out


def moe_expert_ffn_channels(x, Wgate, Wup, WdownT, sel_idx, sel_w, score, c: int, y=None, keep=None, ws=None,
                            stream=None):
    """Expert FFN where each (token, slot) keeps its c highest-scoring
    channels (score[B][k][d_ff]); WdownT from moe_down_channel_major.
    -> y[B][d] fp32.  ``keep``: optional [B][k][d_ff/32] int32 output."""
    B, d = x.shape
    E, F, _ = Wgate.shape
    k = sel_idx.shape[1]
    lib = load_library()
    dims = Dims(B, d, E, k, F)
    n = int(lib.moe_channels_workspace_bytes(dims))
    if n == 0:
        raise MoeError(4, "moe_channels_workspace_bytes")
    if ws is None:
        ws = _made(stream, x, torch.zeros, n, dtype=torch.uint8)
    if y is None:
        y = _made(stream, x, torch.empty, B, d, dtype=torch.float32)
    st = lib.moe_expert_ffn_channels(_ptr(x), _ptr(Wgate), _ptr(Wup), _ptr(WdownT), dims, _ptr(sel_idx),
                                     _ptr(sel_w), _ptr(score), int(c), _ptr(y), _ptr(keep), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "moe_expert_ffn_channels")
    return y


# The calls below are short on the GPU, so the binding keeps its own part
# short: structures of the same numbers are built once, and the current
# stream is read as a raw handle.
@functools.lru_cache(maxsize=1024)
def _dims(B: int, d: int, E: int, k: int, d_ff: int) -> Dims:
    return Dims(B, d, E, k, d_ff)


@functools.lru_cache(maxsize=256)
def _scoring(score: int, groups: int, top_groups: int, group_best: int, renorm: int, scale: float) -> Scoring:
    return Scoring(score, groups, top_groups, group_best, renorm, scale)


def _device_of(t) -> int:
    """The current CUDA device, which t (and every tensor of its call) must
    be on: a kernel of another device cannot read it."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError("tensors must be on the current CUDA device")
    return dev


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# Element types by what the library reads: it sees addresses only.  e4m3
# values may come as their bits.
_I32, _F32, _E4M3 = (torch.int32,), (torch.float32,), (torch.float8_e4m3fn, torch.uint8, torch.int8)


def _buf(t, n: int, types, dev: int):
    """Address of a contiguous tensor of at least n elements of one of the
    types, on device dev (raw addresses pass, for boundary tests)."""
    if (isinstance(t, torch.Tensor) and t.dtype in types and t.numel() >= n and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if isinstance(t, torch.Tensor):
        if t.dtype not in types:
            raise TypeError(f"expected a tensor of {types[0]}, got {t.dtype}")
        if t.numel() < n:
            raise ValueError(f"tensor of {t.numel()} elements where the call's sizes need {n}")
        if t.get_device() != dev:
            raise ValueError("tensors must be on the current CUDA device")
    return _ptr(t)


def _weight(w, scale, E: int, rows: int, cols: int, dev: int):
    """Addresses of e4m3 matrices [E][rows][cols] and their block scales
    (of that shape, or flat)."""
    rb, cb = (rows + 127) // 128, (cols + 127) // 128
    if (w.dtype in _E4M3 and w.numel() == E * rows * cols and w.size(-1) == cols and w.get_device() == dev
            and w.is_contiguous() and scale.dtype in _F32 and scale.numel() >= E * rb * cb
            and (scale.size(-1) == cb or scale.ndim != 3) and scale.get_device() == dev and scale.is_contiguous()):
        return w.data_ptr(), scale.data_ptr()
    if w.shape != (E, rows, cols):
        raise ValueError(f"weights of shape {tuple(w.shape)} where the call's sizes need {(E, rows, cols)}")
    if scale.ndim == 3 and scale.shape != (E, rb, cb):
        raise ValueError(f"weight scales of shape {tuple(scale.shape)} where the call's sizes need {(E, rb, cb)}")
    return _buf(w, E * rows * cols, _E4M3, dev), _buf(scale, E * rb * cb, _F32, dev)


def _list_bufs(l: dict, B: int, E: int, k: int, dev: int) -> Lists:
    return Lists(_buf(l["n_active"], 1, _I32, dev), _buf(l["active"], E, _I32, dev), _buf(l["offsets"], E + 1, _I32, dev),
                 _buf(l["tok"], B * k, _I32, dev), _buf(l["w"], B * k, _F32, dev))


def _workspace(ws, dev: int):
    """Address and bytes of a workspace."""
    if ws.get_device() != dev:
        raise ValueError("tensors must be on the current CUDA device")
    return _ptr(ws), ws.nbytes


def _dtype(t) -> int:
    code = _DTYPES.get(t if isinstance(t, torch.dtype) else t.dtype)
    if code is None:
        raise TypeError("expected a float32 or bfloat16 tensor")
    return code


def _new_bytes(n: int, where: str, device) -> torch.Tensor:
    if n == 0:
        raise MoeError(1, where)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def new_route_workspace(B: int, E: int, k: int, device="cuda") -> torch.Tensor:
    """Workspace of moe_route_scored."""
    n = int(load_library().moe_route_workspace_bytes(Dims(B, 0, E, k, 0)))
    return _new_bytes(n, "moe_route_workspace_bytes", device)


def new_gemm_workspace(device="cuda") -> torch.Tensor:
    """Workspace of moe_expert_gemm_blocks."""
    return torch.zeros(GEMM_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def new_blocks_workspace(B: int, d: int, E: int, k: int, d_ff: int, device="cuda") -> torch.Tensor:
    """Workspace of moe_expert_ffn_blocks."""
    n = int(load_library().moe_blocks_workspace_bytes(Dims(B, d, E, k, d_ff)))
    return _new_bytes(n, "moe_blocks_workspace_bytes", device)


def moe_route_scored(logits, k: int, score: int = MOE_SCORE_SOFTMAX, bias=None, groups: int = 1, top_groups: int = 1,
                     group_best: int = 1, renorm: bool = True, scale: float = 1.0, out=None, lists=None, ws=None,
                     stream=None):
    """-> (sel_idx[B][k], sel_w[B][k], lists dict) from router logits[B][E]
    fp32: softmax or sigmoid scores, a bias that steers the choice, expert
    groups, top-k, weights."""
    B, E = logits.shape
    dev = _device_of(logits)
    if out is None:
        out = _empty(stream, logits, (B, k), torch.int32), _empty(stream, logits, (B, k), torch.float32)
    if lists is None:
        lists = _made(stream, logits, alloc_lists, B, E, k)
    if ws is None:
        ws = _made(stream, logits, new_route_workspace, B, E, k)
    sel, w = out
    st = (_lib or load_library()).moe_route_scored(
        _buf(logits, B * E, _F32, dev), None if bias is None else _buf(bias, E, _F32, dev), _dims(B, 0, E, k, 0),
        _scoring(score, groups, top_groups, group_best, int(renorm), float(scale)), _buf(sel, B * k, _I32, dev),
        _buf(w, B * k, _F32, dev), _list_bufs(lists, B, E, k, dev), *_workspace(ws, dev), _raw_stream(dev) if stream is None else _stream(stream))
    _check(st, "moe_route_scored")
    return sel, w, lists


def moe_quantize_blocks(x, block_rows: int = 1, q=None, scale=None, stream=None):
    """-> (q e4m3, scale fp32) of x[..., rows, cols] (fp32 or bf16): a
    power-of-two scale per 128 columns of a row (block_rows 1: scale[...,
    rows, ceil(cols / 128)]) or per 128 x 128 block (block_rows 128)."""
    shape = x.shape
    rows, cols = shape[-2:]
    batch = x.numel() // (rows * cols) if rows * cols else 0
    code = _dtype(x)
    dev = _device_of(x)
    if q is None:
        q = (torch.empty_like(x, dtype=torch.float8_e4m3fn) if stream is None  # (the shortest)
             else _empty(stream, x, shape, torch.float8_e4m3fn))
    rb, cb = rows if block_rows == 1 else -(-rows // 128), -(-cols // 128)
    if scale is None:
        scale = _empty(stream, x, (*shape[:-2], rb, cb), torch.float32)
    st = (_lib or load_library()).moe_quantize_blocks(_ptr(x), code, batch, rows, cols, block_rows,
                                                      _buf(q, batch * rows * cols, _E4M3, dev),
                                                      _buf(scale, batch * rb * cb, _F32, dev), _raw_stream(dev) if stream is None else _stream(stream))
    _check(st, "moe_quantize_blocks")
    return q, scale


def moe_expert_gemm_blocks(q, scale, W, Wscale, lists: dict, k: int, ws=None, y=None, y_dtype=torch.bfloat16,
                           stream=None):
    """-> y[B * k][rows] = W[e] x of every list entry; q[B][d] e4m3 with
    scale[B][ceil(d / 128)], W[E][rows][d] e4m3 with Wscale[E][ceil(rows /
    128)][ceil(d / 128)].  Rows past the last list entry keep what y held."""
    B, d = q.shape
    E, F, _ = W.shape
    dev = _device_of(q)
    if ws is None:
        ws = _made(stream, q, new_gemm_workspace)
    if y is None:
        y = _empty(stream, q, (B * k, F), y_dtype)
    code = _dtype(y)
    st = (_lib or load_library()).moe_expert_gemm_blocks(
        _buf(q, B * d, _E4M3, dev), _buf(scale, B * -(-d // 128), _F32, dev), *_weight(W, Wscale, E, F, d, dev),
        _dims(B, d, E, k, F), _list_bufs(lists, B, E, k, dev), _buf(y, B * k * F, (y.dtype,), dev), code,
        *_workspace(ws, dev), _raw_stream(dev) if stream is None else _stream(stream))
    _check(st, "moe_expert_gemm_blocks")
    return y


def moe_expert_ffn_blocks(x, Wgate, Sgate, Wup, Sup, Wdown, Sdown, lists: dict, k: int, ws=None, y=None,
                          y_dtype=None, stream=None):
    """-> y[B][d] (y_dtype: fp32 or bf16, x's type by default): the expert
    FFN of moe_expert_ffn on block-scaled e4m3 weights; x fp32 or bf16."""
    B, d = x.shape
    E, F, _ = Wgate.shape
    x_code = _dtype(x)
    dev = _device_of(x)
    if ws is None:
        ws = _made(stream, x, new_blocks_workspace, B, d, E, k, F)
    if y is None:
        y = _empty(stream, x, (B, d), y_dtype or x.dtype)
    code = _dtype(y)
    st = (_lib or load_library()).moe_expert_ffn_blocks(
        _ptr(x), x_code,
        BlockWeights(*_weight(Wgate, Sgate, E, F, d, dev), *_weight(Wup, Sup, E, F, d, dev),
                     *_weight(Wdown, Sdown, E, d, F, dev)),
        _dims(B, d, E, k, F), _list_bufs(lists, B, E, k, dev), _buf(y, B * d, (y.dtype,), dev), code,
        *_workspace(ws, dev), _raw_stream(dev) if stream is None else _stream(stream))
    _check(st, "moe_expert_ffn_blocks")
    return y


def moe_expert_ffn_noalloc(x, Wgate, Wup, Wdown, lists: dict, k: int, y=None, stream=None):
    """moe_expert_ffn without a workspace, for callers that cannot allocate
    device memory: the library's static 32 MiB device scratch is used instead
    (shared by all calls on a device; overlapping calls race).  -> y[B][d]."""
    B, d = x.shape
    E, F, _ = Wgate.shape
    if y is None:
        y = _made(stream, x, torch.empty, B, d, dtype=torch.float32)
    st = load_library().moe_expert_ffn_noalloc(_ptr(x), _ptr(Wgate), _ptr(Wup), _ptr(Wdown),
                                               Dims(B, d, E, k, F), _lists(lists), _ptr(y), _stream(stream))
    _check(st, "moe_expert_ffn_noalloc")
    return y


def moe_set_wait_limit_ns(ns: int) -> None:
    """Limit of the kernels' bounded waits for later launches (0 = 1 s)."""
    load_library().moe_set_wait_limit_ns(int(ns))


def moe_check_error(ws, stream=None) -> int:
    """Synchronise and return the status of kernels' error word (0 = ok)."""
    return int(load_library().moe_check_error(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))

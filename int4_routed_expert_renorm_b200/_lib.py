"""ctypes binding of libcolimoe (include/coli_moe.h): argument marshalling only.

Every function here has the name of the C entry point it calls, takes torch
tensors that already live on the device (or None where the C call accepts
NULL), passes their data pointers and the current CUDA stream, and raises
``ColiError`` on a non-OK status.  No step of the layer runs in Python; if the
library is missing the import fails loudly.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libcolimoe.so")

# COLI_* constants of include/coli_moe.h
COLI_OK, COLI_ERR_INVALID_ARG, COLI_ERR_UNSUPPORTED, COLI_ERR_WORKSPACE = 0, 1, 2, 3
COLI_ERR_CUDA, COLI_ERR_NONFINITE, COLI_ERR_DEVICE = 4, 5, 6
COLI_FLAG_NONFINITE, COLI_FLAG_BAD_ID, COLI_FLAG_TIMEOUT, COLI_FLAG_RANGE = 0x1, 0x2, 0x4, 0x8
COLI_LAYER_PRENORM, COLI_PATH_DECODE, COLI_PATH_PREFILL = 0x1, 0x10, 0x20
COLI_LAYER_HOST_X, COLI_LAYER_HOST_OUT = 0x2, 0x4
COLI_FORM_DECODE_SPLITK, COLI_FORM_DECODE_TWOPHASE, COLI_FORM_PREFILL = 1, 2, 3

EXPORTS = ("coli_moe_route", "coli_moe_union", "coli_moe_expert_ffn", "coli_moe_layer",
           "coli_moe_workspace_bytes", "coli_moe_get_status", "coli_status_str", "coli_moe_version",
           "coli_moe_launch_count", "coli_moe_set_stage_events", "coli_moe_layer_noalloc", "coli_moe_ffn_form",
           "coli_moe_union_offsets", "coli_moe_test_wait_timeout", "coli_moe_layer_ep", "coli_moe_partial_to_bf16",
           "coli_moe_tier_state_bytes", "coli_moe_tier_reset", "coli_moe_layer_tiered", "coli_moe_tier_prefetch",
           "coli_moe_tier_lookahead", "coli_moe_balance", "coli_moe_balance_backward",
           "coli_moe_balance_workspace_bytes", "coli_add_rmsnorm_fp8", "coli_fp8_matmul", "coli_moe_expert_ffn_fp8",
           "coli_moe_fp8_workspace_bytes")
COLI_FP8_OUT_F32 = 0x1
COLI_NOALLOC_SCRATCH_BYTES = 32 << 20


class ColiError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_str(status)} (status {status})")
        self.status = status


class coli_moe_dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_shared", ctypes.c_int32), ("group", ctypes.c_int32),
                ("code_bits", ctypes.c_int32)]


class coli_moe_weights(ctypes.Structure):
    _fields_ = [("gate_q", ctypes.c_void_p), ("up_q", ctypes.c_void_p), ("down_q", ctypes.c_void_p),
                ("gate_s", ctypes.c_void_p), ("up_s", ctypes.c_void_p), ("down_s", ctypes.c_void_p),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p)]


class coli_moe_tier(ctypes.Structure):
    _fields_ = [("gate_q", ctypes.c_void_p), ("up_q", ctypes.c_void_p), ("down_q", ctypes.c_void_p),
                ("gate_s", ctypes.c_void_p), ("up_s", ctypes.c_void_p), ("down_s", ctypes.c_void_p),
                ("n_slots", ctypes.c_int32), ("state", ctypes.c_void_p)]


class coli_moe_weights_fp8(ctypes.Structure):
    _fields_ = [("gate_q", ctypes.c_void_p), ("up_q", ctypes.c_void_p), ("down_q", ctypes.c_void_p),
                ("gate_s", ctypes.c_void_p), ("up_s", ctypes.c_void_p), ("down_s", ctypes.c_void_p)]


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m int4_routed_expert_renorm_b200.build`")
    lib = ctypes.CDLL(path)
    P, I, Z, U32, U64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_uint64
    D, W = ctypes.POINTER(coli_moe_dims), ctypes.POINTER(coli_moe_weights)
    TR, W8, F = ctypes.POINTER(coli_moe_tier), ctypes.POINTER(coli_moe_weights_fp8), ctypes.c_float
    sig = {
        "coli_moe_route": (I, [P, P, I, I, I, P, P, P]),
        "coli_moe_union": (I, [P, I, I, I, P, P, P, P, P, P]),
        "coli_moe_expert_ffn": (I, [D, W, P, I, P, P, P, P, P, P, P, P, P, U32, P, Z, P]),
        "coli_moe_layer": (I, [D, W, P, I, P, P, U32, P, P, P, P, P, Z, P]),
        "coli_moe_workspace_bytes": (Z, [D, I]),
        "coli_moe_get_status": (I, [P, ctypes.POINTER(U32)]),
        "coli_status_str": (ctypes.c_char_p, [I]),
        "coli_moe_version": (I, []),
        "coli_moe_launch_count": (U64, [I]),
        "coli_moe_set_stage_events": (I, [ctypes.POINTER(ctypes.c_void_p), I]),
        "coli_moe_layer_noalloc": (I, [D, W, P, I, P, P, U32, P, P, P, P, P]),
        "coli_moe_ffn_form": (I, [D, I, U32, ctypes.POINTER(I)]),
        "coli_moe_union_offsets": (I, [D, I, ctypes.POINTER(Z)]),
        "coli_moe_test_wait_timeout": (I, [U64, P, P]),
        "coli_moe_layer_ep": (I, [D, W, I, I, I, P, I, P, P, U32, P, P, P, P, P, Z, P]),
        "coli_moe_partial_to_bf16": (I, [P, P, Z, P]),
        "coli_moe_tier_state_bytes": (Z, [D, I]),
        "coli_moe_tier_reset": (I, [D, TR, P]),
        "coli_moe_layer_tiered": (I, [D, W, TR, P, I, P, P, U32, P, P, P, P, P, Z, P]),
        "coli_moe_tier_prefetch": (I, [D, W, TR, P, I, P]),
        "coli_moe_tier_lookahead": (I, [D, W, TR, P, I, U32, P, Z, P]),
        "coli_moe_balance": (I, [P, P, P, P, I, I, I, P, P, P, P, P, Z, P]),
        "coli_moe_balance_backward": (I, [P, P, P, P, P, P, P, P, P, I, I, I, P, P, P, Z, P]),
        "coli_moe_balance_workspace_bytes": (Z, [I, I]),
        "coli_add_rmsnorm_fp8": (I, [P, P, P, F, I, I, P, P, P, P, P]),
        "coli_fp8_matmul": (I, [P, P, P, P, I, I, I, P, U32, P]),
        "coli_moe_expert_ffn_fp8": (I, [D, W8, P, P, I, P, P, P, P, P, P, P, P, P, P, Z, P]),
        "coli_moe_fp8_workspace_bytes": (Z, [D, I]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


_lib = load()


def status_str(s: int) -> str:
    return _lib.coli_status_str(s).decode()


def _ptr(t):
    """Device address of a tensor argument (None -> NULL).  The library reads and
    writes dense row-major device buffers, so only contiguous CUDA tensors pass:
    a strided view would be read as if it were dense, and a host pointer would
    reach a kernel."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (dense, row-major)")
    if t.device.type != "cuda":
        raise ValueError(f"tensor arguments must be in device memory, got a tensor on {t.device}")
    return ctypes.c_void_p(t.data_ptr())


def _host_ptr(t, name: str):
    """Host address of a page-locked CPU tensor (COLI_LAYER_HOST_X / _OUT);
    the library maps it to its device address and refuses any other."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (dense, row-major)")
    if t.device.type != "cpu" or not t.is_pinned():
        raise ValueError(f"{name}: the HOST flag needs a page-locked CPU tensor, got one on {t.device}")
    return ctypes.c_void_p(t.data_ptr())


def _need(t, n: int, esize: int, name: str, at_least: bool = False):
    """Refuse a tensor whose size does not match what the C call will read or
    write through its pointer (n elements of esize bytes; None passes)."""
    if t is None:
        return
    if t.element_size() != esize:
        raise ValueError(f"{name}: elements of {t.element_size()} bytes, the call needs {esize}")
    if (t.numel() < n) if at_least else (t.numel() != n):
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {'at least ' if at_least else ''}{n}")


def _tokens(x, H: int) -> int:
    if x.dim() != 2 or x.shape[1] != H:
        raise ValueError(f"x: shape {tuple(x.shape)}, the call needs [T, {H}]")
    _need(x, x.shape[0] * H, 2, "x")
    return x.shape[0]


def _layer_sizes(dims, T: int, out, residual, logits_in, logits_out, topk_ids_out, topk_w_out):
    H, E, k = dims.hidden, dims.n_experts, dims.top_k
    _need(out, T * H, 2, "out")
    _need(residual, T * H, 2, "residual")
    _need(logits_in, T * E, 4, "logits_in")
    _need(logits_out, T * E, 4, "logits_out")
    _need(topk_ids_out, T * k, 4, "topk_ids_out")
    _need(topk_w_out, T * k, 4, "topk_w_out")


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _stream_scope(stream, device):
    """The scope in which a holder makes the tensors that it hands to calls on
    `stream` (None: the current one): memory that the allocator ties to that
    stream, so that it is handed out again only behind the kernels that use it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream),
                                           device=device)
    return torch.cuda.stream(stream)


def _check(st: int, where: str):
    if st != COLI_OK:
        raise ColiError(st, where)


def coli_moe_version() -> int:
    return _lib.coli_moe_version()


def coli_moe_launch_count(reset: bool = False) -> int:
    return _lib.coli_moe_launch_count(1 if reset else 0)


def coli_moe_workspace_bytes(dims: coli_moe_dims, t_max: int) -> int:
    return _lib.coli_moe_workspace_bytes(ctypes.byref(dims), t_max)


def coli_moe_ffn_form(dims: coli_moe_dims, T: int, flags: int = 0) -> int:
    """The COLI_FORM_* value a layer call with these dims, T and flags takes
    (0 for T == 0); raises ColiError where the call would fail on them."""
    form = ctypes.c_int(0)
    _check(_lib.coli_moe_ffn_form(ctypes.byref(dims), T, flags, ctypes.byref(form)), "coli_moe_ffn_form")
    return form.value


def coli_moe_route(logits, bias, topk_ids, topk_w, stream=None):
    T, E = logits.shape
    k = topk_ids.shape[1]
    _need(logits, T * E, 4, "logits")
    _need(bias, E, 4, "bias")
    _need(topk_ids, T * k, 4, "topk_ids")
    _need(topk_w, T * k, 4, "topk_w")
    _check(_lib.coli_moe_route(_ptr(logits), _ptr(bias), T, E, k, _ptr(topk_ids), _ptr(topk_w), _stream(stream)),
           "coli_moe_route")


def coli_moe_union(topk_ids, n_experts, unique_ids, n_unique, seg_off, perm, pair_pos, stream=None):
    T, k = topk_ids.shape
    P = T * k
    _need(topk_ids, P, 4, "topk_ids")
    _need(unique_ids, min(n_experts, P), 4, "unique_ids", at_least=True)
    _need(n_unique, 1, 4, "n_unique", at_least=True)
    _need(seg_off, min(n_experts, P) + 1, 4, "seg_off", at_least=True)
    _need(perm, P, 4, "perm", at_least=True)
    _need(pair_pos, P, 4, "pair_pos", at_least=True)
    _check(_lib.coli_moe_union(_ptr(topk_ids), T, k, n_experts, _ptr(unique_ids), _ptr(n_unique), _ptr(seg_off),
                               _ptr(perm), _ptr(pair_pos), _stream(stream)), "coli_moe_union")


def coli_moe_expert_ffn(dims, weights, x, topk_ids, topk_w, unique_ids, n_unique, seg_off, perm, pair_pos,
                        residual, out, ws, flags=0, stream=None):
    T = _tokens(x, dims.hidden)
    P, E = T * dims.top_k, dims.n_experts
    _layer_sizes(dims, T, out, residual, None, None, topk_ids, topk_w)
    _need(unique_ids, min(E, P), 4, "unique_ids", at_least=True)
    _need(n_unique, 1, 4, "n_unique", at_least=True)
    _need(seg_off, min(E, P) + 1, 4, "seg_off", at_least=True)
    _need(perm, P, 4, "perm", at_least=True)
    _need(pair_pos, P, 4, "pair_pos", at_least=True)
    _check(_lib.coli_moe_expert_ffn(ctypes.byref(dims), ctypes.byref(weights), _ptr(x), T, _ptr(topk_ids),
                                    _ptr(topk_w), _ptr(unique_ids), _ptr(n_unique), _ptr(seg_off), _ptr(perm),
                                    _ptr(pair_pos), _ptr(residual), _ptr(out), flags, _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)), "coli_moe_expert_ffn")


def _io_ptrs(flags, x, residual, out):
    """x, residual, out: device tensors, or page-locked CPU tensors under the
    COLI_LAYER_HOST_X (x, residual) and COLI_LAYER_HOST_OUT (out) flags."""
    hx, ho = flags & COLI_LAYER_HOST_X, flags & COLI_LAYER_HOST_OUT
    return ((_host_ptr(x, "x") if hx else _ptr(x)), (_host_ptr(residual, "residual") if hx else _ptr(residual)),
            (_host_ptr(out, "out") if ho else _ptr(out)))


def coli_moe_layer(dims, weights, x, out, ws, logits_in=None, residual=None, flags=0, logits_out=None,
                   topk_ids_out=None, topk_w_out=None, stream=None):
    T = _tokens(x, dims.hidden)
    _layer_sizes(dims, T, out, residual, logits_in, logits_out, topk_ids_out, topk_w_out)
    px, pr, po = _io_ptrs(flags, x, residual, out)
    _check(_lib.coli_moe_layer(ctypes.byref(dims), ctypes.byref(weights), px, T, _ptr(logits_in), pr, flags, po,
                               _ptr(logits_out), _ptr(topk_ids_out), _ptr(topk_w_out), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)), "coli_moe_layer")


def coli_moe_layer_noalloc(dims, weights, x, out, logits_in=None, residual=None, flags=0, logits_out=None,
                           topk_ids_out=None, topk_w_out=None, stream=None):
    """coli_moe_layer with the library's own scratch instead of a workspace
    tensor, for callers that cannot allocate device memory (see the header)."""
    T = _tokens(x, dims.hidden)
    _layer_sizes(dims, T, out, residual, logits_in, logits_out, topk_ids_out, topk_w_out)
    px, pr, po = _io_ptrs(flags, x, residual, out)
    _check(_lib.coli_moe_layer_noalloc(ctypes.byref(dims), ctypes.byref(weights), px, T, _ptr(logits_in), pr, flags,
                                       po, _ptr(logits_out), _ptr(topk_ids_out), _ptr(topk_w_out),
                                       _stream(stream)), "coli_moe_layer_noalloc")


def coli_moe_layer_ep(dims, weights, expert_begin: int, expert_end: int, with_shared: bool, x, out_partial, ws,
                      logits_in=None, residual=None, flags=0, logits_out=None, topk_ids_out=None, topk_w_out=None,
                      stream=None):
    """One expert-parallel rank's fp32 partial output (see the header)."""
    T = _tokens(x, dims.hidden)
    _layer_sizes(dims, T, None, residual, logits_in, logits_out, topk_ids_out, topk_w_out)
    _need(out_partial, T * dims.hidden, 4, "out_partial")
    _check(_lib.coli_moe_layer_ep(ctypes.byref(dims), ctypes.byref(weights), expert_begin, expert_end,
                                  1 if with_shared else 0, _ptr(x), T, _ptr(logits_in), _ptr(residual), flags,
                                  _ptr(out_partial), _ptr(logits_out), _ptr(topk_ids_out), _ptr(topk_w_out), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)), "coli_moe_layer_ep")


def coli_moe_tier_state_bytes(dims, n_slots: int) -> int:
    return _lib.coli_moe_tier_state_bytes(ctypes.byref(dims), n_slots)


def coli_moe_tier_reset(dims, tier, stream=None):
    _check(_lib.coli_moe_tier_reset(ctypes.byref(dims), ctypes.byref(tier), _stream(stream)), "coli_moe_tier_reset")


def coli_moe_layer_tiered(dims, slots, tier, x, out, ws, logits_in=None, residual=None, flags=0, logits_out=None,
                          topk_ids_out=None, topk_w_out=None, stream=None):
    """coli_moe_layer through a host-RAM expert tier (see the header)."""
    T = _tokens(x, dims.hidden)
    _layer_sizes(dims, T, out, residual, logits_in, logits_out, topk_ids_out, topk_w_out)
    px, pr, po = _io_ptrs(flags, x, residual, out)
    _check(_lib.coli_moe_layer_tiered(ctypes.byref(dims), ctypes.byref(slots), ctypes.byref(tier), px, T,
                                      _ptr(logits_in), pr, flags, po, _ptr(logits_out), _ptr(topk_ids_out),
                                      _ptr(topk_w_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "coli_moe_layer_tiered")


def coli_moe_tier_prefetch(dims, slots, tier, ids, stream=None):
    """Places experts ids (device int32, at most n_slots of them) in the tier."""
    if ids.dtype.itemsize != 4:
        raise ValueError("ids: int32 expert ids")
    _check(_lib.coli_moe_tier_prefetch(ctypes.byref(dims), ctypes.byref(slots), ctypes.byref(tier), _ptr(ids),
                                       ids.numel(), _stream(stream)), "coli_moe_tier_prefetch")


def coli_moe_tier_lookahead(dims, next_slots, next_tier, x, ws, flags=0, stream=None):
    """Routes x with the next layer's router and places its experts in that
    layer's tier (see the header)."""
    T = _tokens(x, dims.hidden)
    _check(_lib.coli_moe_tier_lookahead(ctypes.byref(dims), ctypes.byref(next_slots), ctypes.byref(next_tier),
                                        _ptr(x), T, flags, _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)), "coli_moe_tier_lookahead")


def coli_moe_partial_to_bf16(partial, out, stream=None):
    """out = bf16(partial), elementwise (out: bf16 bits, int16 tensor)."""
    n = partial.numel()
    _need(out, n, 2, "out")
    _check(_lib.coli_moe_partial_to_bf16(_ptr(partial), _ptr(out), n, _stream(stream)), "coli_moe_partial_to_bf16")


def coli_moe_union_offsets(dims, T: int) -> list[int]:
    """Byte offsets of unique_ids, n_unique, seg_off, perm and pair_pos inside
    the workspace of a coli_moe_layer call with these dims and T."""
    off = (ctypes.c_size_t * 5)()
    _check(_lib.coli_moe_union_offsets(ctypes.byref(dims), T, off), "coli_moe_union_offsets")
    return list(off)


def coli_moe_test_wait_timeout(limit_ns: int, elapsed=None, stream=None):
    """Test hook of the bounded device waits (see the header); elapsed: None or
    a device int64 tensor of 2 elements receiving each wait's duration in ns."""
    _need(elapsed, 2, 8, "elapsed")
    _check(_lib.coli_moe_test_wait_timeout(limit_ns, _ptr(elapsed), _stream(stream)), "coli_moe_test_wait_timeout")


def coli_moe_set_stage_events(events):
    """events: list of torch.cuda.Event (already recorded once, so they exist) or []."""
    n = len(events)
    arr = (ctypes.c_void_p * max(n, 1))(*[e.cuda_event for e in events])
    _check(_lib.coli_moe_set_stage_events(arr if n else None, n), "coli_moe_set_stage_events")


def coli_moe_get_status(stream=None):
    """Returns (status, flags); synchronises the stream and clears the device word."""
    f = ctypes.c_uint32(0)
    st = _lib.coli_moe_get_status(_stream(stream), ctypes.byref(f))
    return st, f.value


# ---- balance loss, 8-bit floating point ------------------------------------
#
# These calls are short (a few microseconds on the GPU for single tokens), so
# their checks are written for few interpreter steps: one pass per tensor over
# type, size, layout and device.

_F32, _I32 = (torch.float32,), (torch.int32,)
_U8 = (torch.uint8, torch.bool)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_E4M3 = (torch.float8_e4m3fn, torch.uint8, torch.int8)
_ANY = None


# The quick forms of torch.cuda.current_device and current_stream, where this torch has them.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _refuse(specs):
    """Why _args refused its arguments: types and sizes first, then layout and device."""
    given = [x for x in specs if x[1] is not None]
    for name, t, types, n, at_least in given:
        if types is not None and t.dtype not in types:
            names = " or ".join(str(x).replace("torch.", "") for x in types)
            raise ValueError(f"{name}: {t.dtype}, the call needs {names}")
        if n is not None and (t.numel() < n if at_least else t.numel() != n):
            raise ValueError(f"{name}: {t.numel()} elements, the call needs {'at least ' if at_least else ''}{n}")
    for name, t, *_ in given:
        _ptr(t)
    for name, t, *_ in given:
        if t.get_device() != _current_device():
            raise ValueError(f"{name}: a tensor on {t.device}, but the current device is cuda:{_current_device()}")
    raise ValueError("arguments refused")


def _args(*specs):
    """Data pointers of (name, tensor, types, elements, at_least) arguments (None
    -> NULL) and their device: dense tensors of these types and sizes on the
    current device, where the call launches."""
    dev = None
    out = []
    for _, t, types, n, at_least in specs:
        if t is None:
            out.append(None)
            continue
        d = t.get_device()
        if dev is None:
            dev = d
        if (d != dev or d < 0 or not t.is_contiguous() or (types is not None and t.dtype not in types)
                or (n is not None and (t.numel() < n if at_least else t.numel() != n))):
            _refuse(specs)
        out.append(t.data_ptr())
    if dev != _current_device():
        _refuse(specs)
    out.append(dev)
    return out


def _raw_stream(stream, dev):
    if stream is None:
        return _current_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _rows(t, name: str):
    """The shape of a 2-D tensor."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: shape {tuple(shape)}, the call needs two dimensions")
    return shape


def coli_moe_balance_workspace_bytes(t_max: int, n_experts: int) -> int:
    return _lib.coli_moe_balance_workspace_bytes(t_max, n_experts)


def coli_moe_balance(logits, bias, topk_ids, mask, counts, n_live, prob_mean, loss, ws, stream=None):
    """Per-expert counts, mean probabilities and the balance loss of a routed
    batch (see the header).  mask: None, or uint8/bool [T], 0 for padding."""
    T, E = _rows(logits, "logits")
    k = _rows(topk_ids, "topk_ids")[1]
    p = _args(("logits", logits, _F32, None, False), ("bias", bias, _F32, E, False),
              ("topk_ids", topk_ids, _I32, T * k, False), ("mask", mask, _U8, T, False),
              ("counts", counts, _I32, E, False), ("n_live", n_live, _I32, 1, False),
              ("prob_mean", prob_mean, _F32, E, False), ("loss", loss, _F32, 1, False), ("ws", ws, _ANY, None, False))
    st = _lib.coli_moe_balance(p[0], p[1], p[2], p[3], T, E, k, p[4], p[5], p[6], p[7], p[8], ws.nbytes,
                               _raw_stream(stream, p[-1]))
    if st:
        _check(st, "coli_moe_balance")


def coli_moe_balance_backward(logits, bias, mask, counts, n_live, grad_loss, topk_ids, topk_w, d_topk_w, d_logits,
                              d_bias, ws, stream=None):
    """Gradient of the router logits from the balance loss and from the
    renormalised weights (see the header).  grad_loss: a device tensor of one
    fp32 value, or None; d_topk_w: the weights' gradient, or None."""
    T, E = _rows(logits, "logits")
    if d_topk_w is not None and (topk_ids is None or topk_w is None):
        raise ValueError("d_topk_w needs topk_ids and topk_w")
    given = topk_ids if topk_ids is not None else topk_w
    if given is None:
        raise ValueError("topk_ids: the call needs the routing's shape [T, k]")
    k = _rows(given, "topk_ids")[1]
    p = _args(("logits", logits, _F32, None, False), ("bias", bias, _F32, E, False), ("mask", mask, _U8, T, False),
              ("counts", counts, _I32, E, False), ("n_live", n_live, _I32, 1, False),
              ("grad_loss", grad_loss, _F32, 1, False), ("topk_ids", topk_ids, _I32, T * k, False),
              ("topk_w", topk_w, _F32, T * k, False), ("d_topk_w", d_topk_w, _F32, T * k, False),
              ("d_logits", d_logits, _F32, T * E, False), ("d_bias", d_bias, _F32, E, False),
              ("ws", ws, _ANY, None, False))
    st = _lib.coli_moe_balance_backward(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], T, E, k, p[9], p[10], p[11],
                                        ws.nbytes, _raw_stream(stream, p[-1]))
    if st:
        _check(st, "coli_moe_balance_backward")


def coli_add_rmsnorm_fp8(x, residual, weight, eps: float, sum_out, norm_out, q, q_scale, stream=None):
    """Residual addition, root-mean-square norm and e4m3 rows with a scale per
    128 columns (see the header)."""
    T, H = _rows(x, "x")
    n = T * H
    p = _args(("x", x, _BF16, None, False), ("residual", residual, _BF16, n, False), ("weight", weight, _BF16, H, False),
              ("sum_out", sum_out, _BF16, n, False), ("norm_out", norm_out, _BF16, n, False), ("q", q, _E4M3, n, False),
              ("q_scale", q_scale, _F32, T * (H // 128), False))
    st = _lib.coli_add_rmsnorm_fp8(p[0], p[1], p[2], eps, T, H, p[3], p[4], p[5], p[6], _raw_stream(stream, p[-1]))
    if st:
        _check(st, "coli_add_rmsnorm_fp8")


def coli_fp8_matmul(a, a_scale, w, w_scale, out, stream=None):
    """out = (a * a_scale) @ (w * w_scale).T for e4m3 codes with a scale per row
    and 128 columns (a) and per 128 x 128 block (w); out: bf16 (2-byte elements)
    or fp32 [M, N] (see the header)."""
    M, K = _rows(a, "a")
    N = _rows(w, "w")[0]
    nk = -(-K // 128)
    f32 = out.dtype == torch.float32
    p = _args(("a", a, _E4M3, None, False), ("a_scale", a_scale, _F32, M * nk, False), ("w", w, _E4M3, N * K, False),
              ("w_scale", w_scale, _F32, -(-N // 128) * nk, False), ("out", out, _F32 if f32 else _BF16, M * N, False))
    st = _lib.coli_fp8_matmul(p[0], p[1], p[2], p[3], M, N, K, p[4], COLI_FP8_OUT_F32 if f32 else 0,
                              _raw_stream(stream, p[-1]))
    if st:
        _check(st, "coli_fp8_matmul")


def coli_moe_fp8_workspace_bytes(dims: coli_moe_dims, t_max: int) -> int:
    return _lib.coli_moe_fp8_workspace_bytes(ctypes.byref(dims), t_max)


def coli_moe_expert_ffn_fp8(dims, weights, x, x_scale, topk_ids, topk_w, unique_ids, n_unique, seg_off, perm, pair_pos,
                            residual, out, ws, stream=None):
    """Expert FFN + combine over e4m3 experts for a routed and unioned batch (see
    the header); weights: ``fp8_weights(...)``."""
    T, H = _rows(x, "x")
    if H != dims.hidden:
        raise ValueError(f"x: shape {tuple(x.shape)}, the call needs [T, {dims.hidden}]")
    made = getattr(weights, "made_of", None)        # None: a struct filled in by hand
    if made is not None and made[:3] != (dims.n_experts + dims.n_shared, dims.inter, dims.hidden):
        raise ValueError(f"weights: {made[0]} experts of {made[1]} x {made[2]}, the dims need "
                         f"{dims.n_experts + dims.n_shared} of {dims.inter} x {dims.hidden}")
    P = T * dims.top_k
    U = min(dims.n_experts, P)
    p = _args(("x", x, _E4M3, None, False), ("x_scale", x_scale, _F32, T * (H // 128), False),
              ("topk_ids", topk_ids, _I32, P, False), ("topk_w", topk_w, _F32, P, False),
              ("unique_ids", unique_ids, _I32, U, True), ("n_unique", n_unique, _I32, 1, True),
              ("seg_off", seg_off, _I32, U + 1, True), ("perm", perm, _I32, P, True),
              ("pair_pos", pair_pos, _I32, P, True), ("residual", residual, _BF16, T * H, False),
              ("out", out, _BF16, T * H, False), ("ws", ws, _ANY, None, False))
    if made is not None and made[3] != p[-1]:
        raise ValueError(f"weights: tensors on cuda:{made[3]}, but the call runs on cuda:{p[-1]}")
    st = _lib.coli_moe_expert_ffn_fp8(ctypes.byref(dims), ctypes.byref(weights), p[0], p[1], T, p[2], p[3], p[4], p[5],
                                      p[6], p[7], p[8], p[9], p[10], p[11], ws.nbytes, _raw_stream(stream, p[-1]))
    if st:
        _check(st, "coli_moe_expert_ffn_fp8")

"""Python binding of the MI355X MoE layer-forward library (libmoe_mi355x.so).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI declared in ``include/moe_mi355x.h``.  torch supplies device
memory and the current stream; nothing here computes any part of the layer,
and there is no CPU fallback -- if the library is missing, importing the
binding works but every call raises.

Function names match the C ABI: moe_route, moe_align,
moe_grouped_gemm_w13_act, moe_grouped_gemm_w2_combine, moe_forward,
moe_forward_quantized, moe_forward_mxfp8, moe_mx_quantize, plus
moe_workspace_size, moe_mx_workspace_size, moe_pick_block_m,
moe_forward_list_offsets and moe_strerror; and, with a :class:`Routing` rule,
moe_select, moe_select_backward, moe_route_scored, moe_forward_scored,
moe_forward_quantized_scored and moe_forward_mxfp8_scored; and
moe_linear_quantized.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libmoe_mi355x.so")

MOE_VARIANT_TILED = 0
MOE_VARIANT_STREAM = 1
MOE_VARIANT_PAIR_GEMV = 2
MOE_VARIANT_PAIR_GEMV_QUANT = 3
MOE_VARIANT_TILED_MXFP8 = 4
MOE_VARIANT_STREAM_MXFP8 = 5
MOE_VARIANT_PAIR_GEMV_MXFP8 = 6
MOE_VARIANT_STREAM_QUANT = 7
MOE_VARIANT_TILED_QUANT = 8

_c_void_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_size_t = ctypes.c_size_t


class MoeError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} failed: {moe_strerror(status)} (status {status})")
        self.status = status


class DispatchInfo(ctypes.Structure):
    _fields_ = [("variant", _c_int), ("block_m", _c_int), ("block_n", _c_int),
                ("block_k", _c_int), ("k_tail", _c_int), ("launches", _c_int),
                ("sorted", _c_int)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class ForwardLists(ctypes.Structure):
    """moe_forward_lists: where moe_forward leaves its index lists."""
    _fields_ = [("block_m", _c_int), ("sorted", _c_int), ("sorted_token_ids", _c_size_t),
                ("expert_ids", _c_size_t), ("expert_block_offsets", _c_size_t),
                ("expert_counts", _c_size_t)]


class MxWeights(ctypes.Structure):
    """moe_mx_weights: four device pointers (E4M3 codes and E8M0 scales)."""
    _fields_ = [("w13_codes", _c_void_p), ("w13_scales", _c_void_p),
                ("w2_codes", _c_void_p), ("w2_scales", _c_void_p)]


class QuantizedWeights(ctypes.Structure):
    """moe_quantized_weights: bits, group size and six device pointers."""
    _fields_ = [("bits", _c_int), ("group_size", _c_int),
                ("w13_q", _c_void_p), ("w13_scales", _c_void_p), ("w13_biases", _c_void_p),
                ("w2_q", _c_void_p), ("w2_scales", _c_void_p), ("w2_biases", _c_void_p)]


class RoutingRule(ctypes.Structure):
    """moe_routing: score, sizes, flags, scale and the device pointer of the bias."""
    _fields_ = [("score", _c_int), ("top_k", _c_int), ("renormalize", _c_int),
                ("n_group", _c_int), ("topk_group", _c_int), ("group_top", _c_int),
                ("scale", ctypes.c_float), ("select_bias", _c_void_p)]


class QuantizedMatrix(ctypes.Structure):
    """moe_quantized_matrix: bits, group size and three device pointers."""
    _fields_ = [("bits", _c_int), ("group_size", _c_int), ("q", _c_void_p),
                ("scales", _c_void_p), ("biases", _c_void_p)]


# the same struct as bytes, which a call takes in a third of the time
_pack_matrix = struct.Struct("@iiPPP").pack


_SIGNATURES = {
    "moe_workspace_size": (_c_size_t, [_c_int] * 5),
    "moe_strerror": (ctypes.c_char_p, [_c_int]),
    "moe_pick_block_m": (_c_int, [_c_int] * 3),
    "moe_route": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                           _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                           _c_void_p]),
    "moe_align_workspace_size": (_c_size_t, [_c_int] * 3),
    "moe_align": (_c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_void_p,
                           _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    "moe_grouped_gemm_w13_act": (_c_int, [_c_void_p] * 5 + [_c_int] * 6 +
                                 [_c_void_p, ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_grouped_gemm_w2_combine": (_c_int, [_c_void_p] * 6 + [_c_int] * 6 +
                                    [_c_void_p, _c_void_p, _c_size_t,
                                     ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_forward": (_c_int, [_c_void_p] * 5 + [_c_int] * 6 +
                    [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                     ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_forward_noalloc": (_c_int, [_c_void_p] * 5 + [_c_int] * 6 +
                            [_c_void_p, _c_void_p, _c_void_p, ctypes.POINTER(DispatchInfo),
                             _c_void_p]),
    "moe_forward_list_offsets": (_c_int, [_c_int] * 5 + [ctypes.POINTER(ForwardLists)]),
    "moe_mx_quantize": (_c_int, [_c_void_p, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    "moe_mx_workspace_size": (_c_size_t, [_c_int] * 5),
    "moe_forward_mxfp8": (_c_int, [_c_void_p] * 3 + [ctypes.POINTER(MxWeights)] + [_c_int] * 6 +
                          [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                           ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_forward_quantized": (_c_int, [_c_void_p] * 3 + [ctypes.POINTER(QuantizedWeights)] +
                              [_c_int] * 6 +
                              [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                               ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_select": (_c_int, [_c_void_p, _c_void_p, _c_int, _c_int] + [_c_void_p] * 3),
    "moe_select_backward": (_c_int, [_c_void_p] * 4 + [_c_int] * 2 + [_c_void_p] * 2),
    "moe_route_scored": (_c_int, [_c_void_p] * 4 + [_c_int] * 3 + [_c_void_p] * 4 +
                         [_c_size_t, _c_void_p]),
    "moe_forward_scored": (_c_int, [_c_void_p] * 6 + [_c_int] * 4 + [_c_void_p] * 4 +
                           [_c_size_t, ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_forward_quantized_scored": (_c_int, [_c_void_p] * 4 + [ctypes.POINTER(QuantizedWeights)] +
                                     [_c_int] * 4 + [_c_void_p] * 4 +
                                     [_c_size_t, ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_forward_mxfp8_scored": (_c_int, [_c_void_p] * 4 + [ctypes.POINTER(MxWeights)] +
                                 [_c_int] * 4 + [_c_void_p] * 4 +
                                 [_c_size_t, ctypes.POINTER(DispatchInfo), _c_void_p]),
    "moe_linear_quantized": (_c_int, [_c_void_p] * 2 + [_c_int] * 4 + [_c_void_p] * 4),
}

_lib: Optional[ctypes.CDLL] = None


def library() -> ctypes.CDLL:
    """Load libmoe_mi355x.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first (python -c "
                "'import __graft_entry__ as g; g.build()'); there is no fallback path")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def moe_workspace_size(M_max: int, E: int, top_k: int, H: int, I: int) -> int:
    return int(library().moe_workspace_size(M_max, E, top_k, H, I))


def moe_strerror(status: int) -> str:
    return library().moe_strerror(status).decode()


def moe_pick_block_m(M: int, E: int, top_k: int) -> int:
    return int(library().moe_pick_block_m(M, E, top_k))


# ---------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t, name, dtypes, shape=None):
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.data_ptr() % 16 != 0:
        raise ValueError(f"{name} must be 16-byte aligned")
    del torch


def _bf16_types():
    torch = _torch()
    return (torch.bfloat16, torch.int16, torch.uint16)


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _raise(call: str, st: int):
    if st != 0:
        raise MoeError(call, st)


def workspace(M_max: int, E: int, top_k: int, H: int, I: int, device=None):
    """Allocate a workspace tensor (uint8) large enough for every call with
    M <= M_max and these layer sizes."""
    torch = _torch()
    n = moe_workspace_size(M_max, E, top_k, H, I)
    if n == 0:
        raise MoeError("moe_workspace_size", -2)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_route(x, w_router, top_k: int, renormalize: bool = True, logit_bias=None,
              topk_ids=None, topk_weights=None, logits_out=None, ws=None, stream=None):
    torch = _torch()
    M, H = x.shape
    E = w_router.shape[0]
    _check(x, "x", _bf16_types())
    _check(w_router, "w_router", _bf16_types(), (E, H))
    if logit_bias is not None:
        _check(logit_bias, "logit_bias", (torch.float32,), (E,))
    if topk_ids is None:
        topk_ids = torch.empty((M, top_k), dtype=torch.int32, device=x.device)
    if topk_weights is None:
        topk_weights = torch.empty((M, top_k), dtype=torch.float32, device=x.device)
    _check(topk_ids, "topk_ids", (torch.int32,), (M, top_k))
    _check(topk_weights, "topk_weights", (torch.float32,), (M, top_k))
    if logits_out is not None:
        _check(logits_out, "logits_out", (torch.float32,), (M, E))
    elif ws is None:
        ws = torch.empty(max(M * E * 4, 16), dtype=torch.uint8, device=x.device)
    st = library().moe_route(_ptr(x), _ptr(w_router), _ptr(logit_bias), M, H, E, top_k,
                             int(bool(renormalize)), _ptr(topk_ids), _ptr(topk_weights),
                             _ptr(logits_out), _ptr(ws), 0 if ws is None else ws.numel(),
                             _stream(stream))
    _raise("moe_route", st)
    return topk_ids, topk_weights


def align_capacity(P: int, E: int, block_m: int) -> tuple:
    """(sorted_token_ids length, expert_ids length) that moe_align needs."""
    nz = min(E, P)
    return P + nz * (block_m - 1), -(-P // block_m) + nz


def moe_align_workspace_size(M: int, top_k: int, E: int) -> int:
    return int(library().moe_align_workspace_size(M, top_k, E))


def moe_align(topk_ids, E: int, block_m: int, sorted_token_ids=None, expert_ids=None,
              expert_block_offsets=None, expert_counts=None, ws=None, stream=None):
    torch = _torch()
    M, top_k = topk_ids.shape
    _check(topk_ids, "topk_ids", (torch.int32,))
    P = M * top_k
    cap, nbl = align_capacity(P, E, block_m)
    dev = topk_ids.device
    if sorted_token_ids is None:
        sorted_token_ids = torch.empty(max(cap, 4), dtype=torch.int32, device=dev)
    if expert_ids is None:
        expert_ids = torch.empty(max(nbl, 4), dtype=torch.int32, device=dev)
    if expert_block_offsets is None:
        expert_block_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    if expert_counts is None:
        expert_counts = torch.empty(E, dtype=torch.int32, device=dev)
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (expert_block_offsets, "expert_block_offsets"),
                 (expert_counts, "expert_counts")):
        _check(t, n, (torch.int32,))
    if sorted_token_ids.numel() < cap or expert_ids.numel() < nbl or \
            expert_block_offsets.numel() < E + 1 or expert_counts.numel() < E:
        raise ValueError("moe_align output buffers are too small")
    need = moe_align_workspace_size(M, top_k, E)
    if ws is None and need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    st = library().moe_align(_ptr(topk_ids), M, top_k, E, block_m, _ptr(sorted_token_ids),
                             _ptr(expert_ids), _ptr(expert_block_offsets),
                             _ptr(expert_counts), _ptr(ws), 0 if ws is None else ws.numel(),
                             _stream(stream))
    _raise("moe_align", st)
    return sorted_token_ids, expert_ids, expert_block_offsets, expert_counts


def moe_grouped_gemm_w13_act(x, w13, sorted_token_ids, expert_ids, expert_block_offsets,
                             top_k: int, block_m: int, act=None, stream=None):
    torch = _torch()
    M, H = x.shape
    E, two_i, H2 = w13.shape
    I = two_i // 2
    _check(x, "x", _bf16_types())
    _check(w13, "w13", _bf16_types(), (E, 2 * I, H))
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (expert_block_offsets, "expert_block_offsets")):
        _check(t, n, (torch.int32,))
    if act is None:
        act = torch.empty((M * top_k, I), dtype=torch.bfloat16, device=x.device)
    _check(act, "act", _bf16_types(), (M * top_k, I))
    info = DispatchInfo()
    st = library().moe_grouped_gemm_w13_act(
        _ptr(x), _ptr(w13), _ptr(sorted_token_ids), _ptr(expert_ids),
        _ptr(expert_block_offsets), M, top_k, E, H, I, block_m, _ptr(act),
        ctypes.byref(info), _stream(stream))
    _raise("moe_grouped_gemm_w13_act", st)
    return act, info.as_dict()


def moe_grouped_gemm_w2_combine(act, w2, topk_weights, sorted_token_ids, expert_ids,
                                expert_block_offsets, M: int, top_k: int, block_m: int,
                                out=None, ws=None, stream=None):
    torch = _torch()
    E, H, I = w2.shape
    _check(act, "act", _bf16_types(), (M * top_k, I))
    _check(w2, "w2", _bf16_types())
    _check(topk_weights, "topk_weights", (torch.float32,))
    if topk_weights.numel() != M * top_k:
        raise ValueError("topk_weights must hold M*top_k values")
    for t, n in ((sorted_token_ids, "sorted_token_ids"), (expert_ids, "expert_ids"),
                 (expert_block_offsets, "expert_block_offsets")):
        _check(t, n, (torch.int32,))
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=act.device)
    _check(out, "out", _bf16_types(), (M, H))
    if ws is None:
        ws = workspace(M, E, top_k, H, I, act.device)
    info = DispatchInfo()
    st = library().moe_grouped_gemm_w2_combine(
        _ptr(act), _ptr(w2), _ptr(topk_weights), _ptr(sorted_token_ids), _ptr(expert_ids),
        _ptr(expert_block_offsets), M, top_k, E, H, I, block_m, _ptr(out), _ptr(ws),
        ws.numel(), ctypes.byref(info), _stream(stream))
    _raise("moe_grouped_gemm_w2_combine", st)
    return out, info.as_dict()


def moe_forward(x, w_router, w13, w2, top_k: int, renormalize: bool = True,
                logit_bias=None, out=None, topk_ids_out=None, topk_weights_out=None,
                ws=None, stream=None):
    """The whole layer.  Returns (out [M, H] bf16, dispatch info dict)."""
    torch = _torch()
    M, H = x.shape
    E, two_i, _ = w13.shape
    I = two_i // 2
    _check(x, "x", _bf16_types())
    _check(w_router, "w_router", _bf16_types(), (E, H))
    _check(w13, "w13", _bf16_types(), (E, 2 * I, H))
    _check(w2, "w2", _bf16_types(), (E, H, I))
    if logit_bias is not None:
        _check(logit_bias, "logit_bias", (torch.float32,), (E,))
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", _bf16_types(), (M, H))
    if topk_ids_out is not None:
        _check(topk_ids_out, "topk_ids_out", (torch.int32,), (M, top_k))
    if topk_weights_out is not None:
        _check(topk_weights_out, "topk_weights_out", (torch.float32,), (M, top_k))
    if ws is None:
        ws = workspace(M, E, top_k, H, I, x.device)
    info = DispatchInfo()
    st = library().moe_forward(
        _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(w13), _ptr(w2), M, E, top_k, H, I,
        int(bool(renormalize)), _ptr(out), _ptr(topk_ids_out), _ptr(topk_weights_out),
        _ptr(ws), ws.numel(), ctypes.byref(info), _stream(stream))
    _raise("moe_forward", st)
    return out, info.as_dict()


MOE_NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_forward_noalloc(x, w_router, w13, w2, top_k: int, renormalize: bool = True,
                        logit_bias=None, out=None, topk_ids_out=None, topk_weights_out=None,
                        stream=None):
    """moe_forward with the library's own device scratch array (no workspace
    argument; allocates no device memory when ``out`` is given).  Returns
    (out [M, H] bf16, dispatch info dict)."""
    torch = _torch()
    M, H = x.shape
    E, two_i, _ = w13.shape
    I = two_i // 2
    _check(x, "x", _bf16_types())
    _check(w_router, "w_router", _bf16_types(), (E, H))
    _check(w13, "w13", _bf16_types(), (E, 2 * I, H))
    _check(w2, "w2", _bf16_types(), (E, H, I))
    if logit_bias is not None:
        _check(logit_bias, "logit_bias", (torch.float32,), (E,))
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", _bf16_types(), (M, H))
    if topk_ids_out is not None:
        _check(topk_ids_out, "topk_ids_out", (torch.int32,), (M, top_k))
    if topk_weights_out is not None:
        _check(topk_weights_out, "topk_weights_out", (torch.float32,), (M, top_k))
    info = DispatchInfo()
    st = library().moe_forward_noalloc(
        _ptr(x), _ptr(w_router), _ptr(logit_bias), _ptr(w13), _ptr(w2), M, E, top_k, H, I,
        int(bool(renormalize)), _ptr(out), _ptr(topk_ids_out), _ptr(topk_weights_out),
        ctypes.byref(info), _stream(stream))
    _raise("moe_forward_noalloc", st)
    return out, info.as_dict()


def moe_forward_list_offsets(M: int, E: int, top_k: int, H: int, I: int) -> dict:
    """Byte offsets in moe_forward's workspace of the index lists it builds
    for a batch of M tokens, with their block size (``sorted`` 0: none)."""
    lists = ForwardLists()
    _raise("moe_forward_list_offsets",
           library().moe_forward_list_offsets(M, E, top_k, H, I, ctypes.byref(lists)))
    return {f: getattr(lists, f) for f, _ in lists._fields_}


def forward_lists(ws, M: int, E: int, top_k: int, H: int, I: int):
    """The index lists moe_forward left in workspace tensor ``ws`` (after a
    completed call with these sizes), as int32 views: (sorted_token_ids,
    expert_ids, expert_block_offsets, expert_counts, block_m).  Only the
    first num_blocks*block_m / num_blocks entries of the first two hold
    data (num_blocks = expert_block_offsets[E])."""
    torch = _torch()
    o = moe_forward_list_offsets(M, E, top_k, H, I)
    if not o["sorted"]:
        raise ValueError("moe_forward builds no index lists for this batch size")
    cap, nbl = align_capacity(M * top_k, E, o["block_m"])

    def view(off, n):
        return ws[off:off + 4 * n].view(torch.int32)

    return (view(o["sorted_token_ids"], cap), view(o["expert_ids"], nbl),
            view(o["expert_block_offsets"], E + 1), view(o["expert_counts"], E), o["block_m"])


def moe_forward_quantized(x, w_router, qweights: dict, top_k: int, renormalize: bool = True,
                          logit_bias=None, out=None, topk_ids_out=None, topk_weights_out=None,
                          ws=None, stream=None):
    """The layer with group-quantized expert weights.  ``qweights`` holds
    ``bits`` (4 or 8), ``w13_q`` [E, 2I, H*bits/32] and ``w2_q``
    [E, H, I*bits/32] (int32 or uint32 words of packed codes), and
    ``w13_scales``, ``w13_biases`` [E, 2I, H/64], ``w2_scales``,
    ``w2_biases`` [E, H, I/64] (bf16).  Returns (out [M, H] bf16, dispatch
    info dict)."""
    torch = _torch()
    M, H = x.shape
    E = w_router.shape[0]
    bits = int(qweights["bits"])
    I = qweights["w2_q"].shape[2] * 32 // bits if bits in (4, 8) else 0
    words = (torch.int32, getattr(torch, "uint32", torch.int32))
    _check(x, "x", _bf16_types())
    _check(w_router, "w_router", _bf16_types(), (E, H))
    if bits in (4, 8):
        for name, shape, types in (("w13_q", (E, 2 * I, H * bits // 32), words),
                                   ("w13_scales", (E, 2 * I, H // 64), _bf16_types()),
                                   ("w13_biases", (E, 2 * I, H // 64), _bf16_types()),
                                   ("w2_q", (E, H, I * bits // 32), words),
                                   ("w2_scales", (E, H, I // 64), _bf16_types()),
                                   ("w2_biases", (E, H, I // 64), _bf16_types())):
            _check(qweights[name], name, types, shape)
    if logit_bias is not None:
        _check(logit_bias, "logit_bias", (torch.float32,), (E,))
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", _bf16_types(), (M, H))
    if topk_ids_out is not None:
        _check(topk_ids_out, "topk_ids_out", (torch.int32,), (M, top_k))
    if topk_weights_out is not None:
        _check(topk_weights_out, "topk_weights_out", (torch.float32,), (M, top_k))
    if ws is None:
        ws = workspace(M, E, top_k, H, max(I, 1), x.device)
    qw = QuantizedWeights(bits, int(qweights.get("group_size", 64)),
                          *(_ptr(qweights.get(n)) for n in ("w13_q", "w13_scales", "w13_biases",
                                                            "w2_q", "w2_scales", "w2_biases")))
    info = DispatchInfo()
    st = library().moe_forward_quantized(
        _ptr(x), _ptr(w_router), _ptr(logit_bias), ctypes.byref(qw), M, E, top_k, H, I,
        int(bool(renormalize)), _ptr(out), _ptr(topk_ids_out), _ptr(topk_weights_out),
        _ptr(ws), ws.numel(), ctypes.byref(info), _stream(stream))
    _raise("moe_forward_quantized", st)
    return out, info.as_dict()


def moe_mx_workspace_size(M_max: int, E: int, top_k: int, H: int, I: int) -> int:
    return int(library().moe_mx_workspace_size(M_max, E, top_k, H, I))


def mx_workspace(M_max: int, E: int, top_k: int, H: int, I: int, device=None):
    """Workspace tensor (uint8) for every moe_forward_mxfp8 call with M <= M_max."""
    torch = _torch()
    n = moe_mx_workspace_size(M_max, E, top_k, H, I)
    if n == 0:
        raise MoeError("moe_mx_workspace_size", -2)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_mx_quantize(src, codes=None, scales=None, stream=None):
    """MXFP8 codes [rows, K] (uint8 E4M3) and scales [rows, K/32] (uint8
    E8M0) of bf16 rows src [rows, K]."""
    torch = _torch()
    rows, K = src.shape
    _check(src, "src", _bf16_types())
    if codes is None:
        codes = torch.empty((rows, K), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=src.device)
    _check(codes, "codes", (torch.uint8,), (rows, K))
    _check(scales, "scales", (torch.uint8,), (rows, K // 32))
    st = library().moe_mx_quantize(_ptr(src), rows, K, _ptr(codes), _ptr(scales), _stream(stream))
    _raise("moe_mx_quantize", st)
    return codes, scales


def moe_forward_mxfp8(x, w_router, mxw: dict, top_k: int, renormalize: bool = True,
                      logit_bias=None, out=None, topk_ids_out=None, topk_weights_out=None,
                      ws=None, stream=None):
    """The layer with MXFP8 experts and GEMM inputs.  ``mxw`` holds
    ``w13_codes`` [E, 2I, H], ``w13_scales`` [E, 2I, H/32], ``w2_codes``
    [E, H, I] and ``w2_scales`` [E, H, I/32] (uint8).  Returns (out [M, H]
    bf16, dispatch info dict)."""
    torch = _torch()
    M, H = x.shape
    E = w_router.shape[0]
    I = mxw["w2_codes"].shape[2]
    _check(x, "x", _bf16_types())
    _check(w_router, "w_router", _bf16_types(), (E, H))
    for name, shape in (("w13_codes", (E, 2 * I, H)), ("w13_scales", (E, 2 * I, H // 32)),
                        ("w2_codes", (E, H, I)), ("w2_scales", (E, H, I // 32))):
        _check(mxw[name], name, (torch.uint8,), shape)
    if logit_bias is not None:
        _check(logit_bias, "logit_bias", (torch.float32,), (E,))
    if out is None:
        out = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
    _check(out, "out", _bf16_types(), (M, H))
    if topk_ids_out is not None:
        _check(topk_ids_out, "topk_ids_out", (torch.int32,), (M, top_k))
    if topk_weights_out is not None:
        _check(topk_weights_out, "topk_weights_out", (torch.float32,), (M, top_k))
    if ws is None:
        ws = mx_workspace(M, E, top_k, H, I, x.device)
    w = MxWeights(*(_ptr(mxw[n]) for n in ("w13_codes", "w13_scales", "w2_codes", "w2_scales")))
    info = DispatchInfo()
    st = library().moe_forward_mxfp8(
        _ptr(x), _ptr(w_router), _ptr(logit_bias), ctypes.byref(w), M, E, top_k, H, I,
        int(bool(renormalize)), _ptr(out), _ptr(topk_ids_out), _ptr(topk_weights_out),
        _ptr(ws), ws.numel(), ctypes.byref(info), _stream(stream))
    _raise("moe_forward_mxfp8", st)
    return out, info.as_dict()


# ---------------------------------------------------------------------------
# scored routing and dense 4-bit products
# ---------------------------------------------------------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}

# ctypes keeps the low 32 bits of a larger number without a word, so the calls
# below refuse sizes from here on (a tensor of 2^32 + 5 rows fits the memory)
_INT_END = 1 << 31


class Routing:
    """A routing rule (moe_routing in the header): how a token's experts are
    chosen from its logits and weighted.  Built once and given to every call
    of a layer.

    ``score``: "softmax" or "sigmoid"; ``select_bias``: [E] fp32 device tensor
    added to the scores for the choice alone, or None (read at every call, so
    it may be updated in place between calls); ``n_group`` groups of
    consecutive experts, of which the ``topk_group`` best stay (default: all),
    scored by their best expert (``group_top`` 1) or the sum of their best two
    (2); ``scale``: a factor of every weight."""

    __slots__ = ("_c", "_address", "top_k", "select_bias")

    def __init__(self, top_k: int, score: str = "softmax", renormalize: bool = True,
                 select_bias=None, n_group: int = 1, topk_group: Optional[int] = None,
                 group_top: int = 1, scale: float = 1.0):
        if score not in _SCORES:
            raise ValueError(f"score must be one of {tuple(_SCORES)}, got {score!r}")
        if select_bias is not None:
            _check(select_bias, "select_bias", (_torch().float32,))
        numbers = [int(v) for v in (top_k, n_group, n_group if topk_group is None else topk_group,
                                    group_top)]
        for name, v in zip(("top_k", "n_group", "topk_group", "group_top"), numbers):
            if not -_INT_END <= v < _INT_END:   # the struct would keep its low bits
                raise ValueError(f"{name} {v} is not a C int")
        set_ = object.__setattr__
        set_(self, "select_bias", select_bias)
        set_(self, "top_k", numbers[0])
        set_(self, "_c", RoutingRule(
            _SCORES[score], numbers[0], int(bool(renormalize)), *numbers[1:], float(scale),
            None if select_bias is None else select_bias.data_ptr()))
        set_(self, "_address", ctypes.addressof(self._c))

    def __setattr__(self, name, value):
        raise AttributeError("a Routing does not change; build another one")

    @property
    def score(self) -> str:
        return "sigmoid" if self._c.score else "softmax"

    @property
    def renormalize(self) -> bool:
        return bool(self._c.renormalize)

    @property
    def n_group(self) -> int:
        return self._c.n_group

    @property
    def topk_group(self) -> int:
        return self._c.topk_group

    @property
    def group_top(self) -> int:
        return self._c.group_top

    @property
    def scale(self) -> float:
        return self._c.scale

    def _arg(self, E: int, device: int) -> int:
        """Address of the C struct for a layer of E experts on a device."""
        b = self.select_bias
        if b is not None:
            _need(b, "select_bias", b.dtype, (E,), device)
            if b.data_ptr() != self._c.select_bias:   # its storage was replaced
                _check(b, "select_bias", (_torch().float32,))
                self._c.select_bias = b.data_ptr()
        return self._address


def _need(t, name, dtype, shape, device: int):
    """Raise unless t is a dense aligned tensor of that kind on that device."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == device and
            t.is_contiguous() and not t.data_ptr() & 15):
        _refuse(t, name, dtype, shape, device)


def _refuse(t, name, dtype, shape, device: int):
    torch = _torch()
    _check(t, name, _bf16_types() if dtype is torch.bfloat16 else (dtype,), shape)
    if t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, expected {device}")


def _current(device: int) -> bool:
    """Whether the call's device is the current one (False too for a host
    tensor's -1, which the argument checks then refuse)."""
    return device >= 0 and _torch()._C._cuda_getDevice() == device


def _elsewhere(device: int, call, *args):
    """The call with its tensors' device made current."""
    torch = _torch()
    if device < 0:
        raise ValueError(f"{call.__name__} needs device tensors")
    with torch.cuda.device(device):
        return call(*args)


def _raw_stream(device: int, stream) -> int:
    """The hipStream_t of a call: ``stream``, or the device's current one."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is on device {stream.device_index}, the tensors on {device}")
    return stream.cuda_stream


def _empty(shape, dtype, device: int, stream):
    """A new tensor that the call's stream may write at once (memory of the
    current stream may still be in use there) and the current one may read."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def moe_select(logits, routing: Routing, topk_ids=None, topk_weights=None, stream=None):
    """Expert ids [M, top_k] int32 and weights [M, top_k] fp32 of logits
    [M, E] fp32 under a routing rule.  The outputs overlap neither each other
    nor an operand."""
    torch = _torch()
    M, E = logits.shape
    if M >= _INT_END or E >= _INT_END:
        raise MoeError("moe_select", -2)
    dev = logits.get_device()
    if not _current(dev):
        return _elsewhere(dev, moe_select, logits, routing, topk_ids, topk_weights, stream)
    out = (M, routing.top_k)
    _need(logits, "logits", torch.float32, (M, E), dev)
    if topk_ids is None:
        topk_ids = _empty(out, torch.int32, dev, stream)
    else:
        _need(topk_ids, "topk_ids", torch.int32, out, dev)
    if topk_weights is None:
        topk_weights = _empty(out, torch.float32, dev, stream)
    else:
        _need(topk_weights, "topk_weights", torch.float32, out, dev)
    st = library().moe_select(logits.data_ptr(), routing._arg(E, dev), M, E, topk_ids.data_ptr(),
                              topk_weights.data_ptr(), _raw_stream(dev, stream))
    if st:
        _raise("moe_select", st)
    return topk_ids, topk_weights


def moe_select_backward(logits, topk_ids, grad_weights, routing: Routing, grad_logits=None,
                        stream=None):
    """Gradient [M, E] fp32 of moe_select's weights with respect to its
    logits, for the ids it gave and the weights' gradient [M, top_k] fp32.
    ``grad_logits`` overlaps no operand."""
    torch = _torch()
    M, E = logits.shape
    if M >= _INT_END or E >= _INT_END:
        raise MoeError("moe_select_backward", -2)
    dev = logits.get_device()
    if not _current(dev):
        return _elsewhere(dev, moe_select_backward, logits, topk_ids, grad_weights, routing,
                          grad_logits, stream)
    pairs = (M, routing.top_k)
    _need(logits, "logits", torch.float32, (M, E), dev)
    _need(topk_ids, "topk_ids", torch.int32, pairs, dev)
    _need(grad_weights, "grad_weights", torch.float32, pairs, dev)
    if grad_logits is None:
        grad_logits = _empty((M, E), torch.float32, dev, stream)
    else:
        _need(grad_logits, "grad_logits", torch.float32, (M, E), dev)
    st = library().moe_select_backward(logits.data_ptr(), topk_ids.data_ptr(),
                                       grad_weights.data_ptr(), routing._arg(E, dev), M, E,
                                       grad_logits.data_ptr(), _raw_stream(dev, stream))
    if st:
        _raise("moe_select_backward", st)
    return grad_logits


def moe_route_scored(x, w_router, routing: Routing, logit_bias=None, topk_ids=None,
                     topk_weights=None, logits_out=None, ws=None, stream=None):
    """moe_route with a routing rule: (topk_ids, topk_weights)."""
    torch = _torch()
    M, H = x.shape
    E = w_router.shape[0]
    if M >= _INT_END or H >= _INT_END or E >= _INT_END:
        raise MoeError("moe_route_scored", -2)
    dev = x.get_device()
    if not _current(dev):
        return _elsewhere(dev, moe_route_scored, x, w_router, routing, logit_bias, topk_ids,
                          topk_weights, logits_out, ws, stream)
    out = (M, routing.top_k)
    _need(x, "x", torch.bfloat16, (M, H), dev)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    if logit_bias is not None:
        _need(logit_bias, "logit_bias", torch.float32, (E,), dev)
    if topk_ids is None:
        topk_ids = _empty(out, torch.int32, dev, stream)
    else:
        _need(topk_ids, "topk_ids", torch.int32, out, dev)
    if topk_weights is None:
        topk_weights = _empty(out, torch.float32, dev, stream)
    else:
        _need(topk_weights, "topk_weights", torch.float32, out, dev)
    if logits_out is not None:
        _need(logits_out, "logits_out", torch.float32, (M, E), dev)
    elif ws is None:
        ws = _empty((max(M * E * 4, 16),), torch.uint8, dev, stream)
    if ws is not None:
        _need(ws, "ws", torch.uint8, (ws.numel(),), dev)
    st = library().moe_route_scored(
        x.data_ptr(), w_router.data_ptr(), _ptr(logit_bias), routing._arg(E, dev), M, H, E,
        topk_ids.data_ptr(), topk_weights.data_ptr(), _ptr(logits_out), _ptr(ws),
        0 if ws is None else ws.numel(), _raw_stream(dev, stream))
    if st:
        _raise("moe_route_scored", st)
    return topk_ids, topk_weights


def _layer_scored(call: str, x, w_router, routing: Routing, weights, weight_args, I: int, ws_size,
                  logit_bias, out, topk_ids_out, topk_weights_out, ws, stream):
    """A layer call with a routing rule: ``weights`` are (name, tensor, dtype,
    shape) to check, ``weight_args`` what the C call takes for them."""
    torch = _torch()
    M, H = x.shape
    E = w_router.shape[0]
    k = routing.top_k
    if max(M, E, H, I) >= _INT_END:
        raise MoeError(call, -2)
    dev = x.get_device()
    if not _current(dev):
        return _elsewhere(dev, _layer_scored, call, x, w_router, routing, weights, weight_args, I,
                          ws_size, logit_bias, out, topk_ids_out, topk_weights_out, ws, stream)
    _need(x, "x", torch.bfloat16, (M, H), dev)
    _need(w_router, "w_router", torch.bfloat16, (E, H), dev)
    for name, t, dtype, shape in weights:
        _need(t, name, dtype, shape, dev)
    if logit_bias is not None:
        _need(logit_bias, "logit_bias", torch.float32, (E,), dev)
    if out is None:
        out = _empty((M, H), torch.bfloat16, dev, stream)
    else:
        _need(out, "out", torch.bfloat16, (M, H), dev)
    if topk_ids_out is not None:
        _need(topk_ids_out, "topk_ids_out", torch.int32, (M, k), dev)
    if topk_weights_out is not None:
        _need(topk_weights_out, "topk_weights_out", torch.float32, (M, k), dev)
    if ws is None:
        n = ws_size(M, E, k, H, I)
        if n == 0:
            raise MoeError(call, -2)
        ws = _empty((n,), torch.uint8, dev, stream)
    else:
        _need(ws, "ws", torch.uint8, (ws.numel(),), dev)
    info = DispatchInfo()
    st = getattr(library(), call)(
        x.data_ptr(), w_router.data_ptr(), _ptr(logit_bias), routing._arg(E, dev), *weight_args, M,
        E, H, I, out.data_ptr(), _ptr(topk_ids_out), _ptr(topk_weights_out), ws.data_ptr(),
        ws.numel(), ctypes.byref(info), _raw_stream(dev, stream))
    _raise(call, st)
    return out, info.as_dict()


def _word_type(t):
    """The type that a tensor of packed code words has to have: int32, or
    uint32 where it has that."""
    torch = _torch()
    return t.dtype if t.dtype is getattr(torch, "uint32", None) else torch.int32


def moe_forward_scored(x, w_router, w13, w2, routing: Routing, logit_bias=None, out=None,
                       topk_ids_out=None, topk_weights_out=None, ws=None, stream=None):
    """moe_forward with a routing rule.  Returns (out [M, H] bf16, dispatch
    info dict)."""
    bf16 = _torch().bfloat16
    E, H = w_router.shape
    I = w2.shape[2]
    return _layer_scored(
        "moe_forward_scored", x, w_router, routing,
        (("w13", w13, bf16, (E, 2 * I, H)), ("w2", w2, bf16, (E, H, I))),
        (w13.data_ptr(), w2.data_ptr()), I, moe_workspace_size, logit_bias, out, topk_ids_out,
        topk_weights_out, ws, stream)


def moe_forward_quantized_scored(x, w_router, qweights: dict, routing: Routing, logit_bias=None,
                                 out=None, topk_ids_out=None, topk_weights_out=None, ws=None,
                                 stream=None):
    """moe_forward_quantized with a routing rule; ``qweights`` as there."""
    bf16 = _torch().bfloat16
    E, H = w_router.shape
    bits = int(qweights["bits"])
    if bits not in (4, 8):
        raise MoeError("moe_forward_quantized_scored", -2)
    I = qweights["w2_q"].shape[2] * 32 // bits
    names = ("w13_q", "w13_scales", "w13_biases", "w2_q", "w2_scales", "w2_biases")
    shapes = ((E, 2 * I, H * bits // 32), (E, 2 * I, H // 64), (E, 2 * I, H // 64),
              (E, H, I * bits // 32), (E, H, I // 64), (E, H, I // 64))
    qw = QuantizedWeights(bits, int(qweights.get("group_size", 64)),
                          *(qweights[n].data_ptr() for n in names))
    return _layer_scored(
        "moe_forward_quantized_scored", x, w_router, routing,
        tuple((n, qweights[n], _word_type(qweights[n]) if n.endswith("_q") else bf16, s)
              for n, s in zip(names, shapes)),
        (ctypes.byref(qw),), I, moe_workspace_size, logit_bias, out, topk_ids_out,
        topk_weights_out, ws, stream)


def moe_forward_mxfp8_scored(x, w_router, mxw: dict, routing: Routing, logit_bias=None, out=None,
                             topk_ids_out=None, topk_weights_out=None, ws=None, stream=None):
    """moe_forward_mxfp8 with a routing rule; ``mxw`` as there."""
    u8 = _torch().uint8
    E, H = w_router.shape
    I = mxw["w2_codes"].shape[2]
    names = ("w13_codes", "w13_scales", "w2_codes", "w2_scales")
    shapes = ((E, 2 * I, H), (E, 2 * I, H // 32), (E, H, I), (E, H, I // 32))
    w = MxWeights(*(mxw[n].data_ptr() for n in names))
    return _layer_scored(
        "moe_forward_mxfp8_scored", x, w_router, routing,
        tuple((n, mxw[n], u8, s) for n, s in zip(names, shapes)), (ctypes.byref(w),), I,
        moe_mx_workspace_size, logit_bias, out, topk_ids_out, topk_weights_out, ws, stream)


def moe_linear_quantized(x, weight: dict, gated: bool = False, row_scale=None, addend=None,
                         out=None, stream=None):
    """out [M, n_out] bf16 = addend + row_scale * f(x W^T) for one dense
    matrix with 4-bit affine weights: ``weight`` holds ``bits`` (4),
    ``group_size`` (32, 64 or 128; default 64), ``q`` [N, K/8] (int32 or
    uint32 words of packed codes), ``scales`` and ``biases``
    [N, K/group_size] (bf16).  ``gated``: the first N/2 rows are gates and
    f = SiLU(gate) * up, n_out = N/2; else f is the identity, n_out = N.
    ``row_scale`` [M] fp32 and ``addend`` [M, n_out] bf16 (``out`` itself, to
    add in place) are optional; ``out`` overlaps no other operand.  |x| is
    below 2^112, and |x| (271 |scale| + |bias|) summed over K within fp32's
    range."""
    torch = _torch()
    M, K = x.shape
    bits, group = int(weight["bits"]), int(weight.get("group_size", 64))
    q, scales, biases = weight["q"], weight["scales"], weight["biases"]
    N = q.shape[0]
    if bits != 4 or group not in (32, 64, 128) or K % group != 0 or M >= _INT_END or \
            N >= _INT_END or K >= _INT_END:
        raise MoeError("moe_linear_quantized", -2)
    dev = x.get_device()
    if not _current(dev):
        return _elsewhere(dev, moe_linear_quantized, x, weight, gated, row_scale, addend, out,
                          stream)
    bf16 = torch.bfloat16
    shape = (M, N // 2 if gated else N)
    _need(x, "x", bf16, (M, K), dev)
    _need(q, "q", _word_type(q), (N, K // 8), dev)
    _need(scales, "scales", bf16, (N, K // group), dev)
    _need(biases, "biases", bf16, (N, K // group), dev)
    if row_scale is not None:
        _need(row_scale, "row_scale", torch.float32, (M,), dev)
    if addend is not None:
        _need(addend, "addend", bf16, shape, dev)
    if out is None:
        out = _empty(shape, bf16, dev, stream)
    else:
        _need(out, "out", bf16, shape, dev)
    w = _pack_matrix(bits, group, q.data_ptr(), scales.data_ptr(), biases.data_ptr())
    st = library().moe_linear_quantized(x.data_ptr(), w, M, N, K, 1 if gated else 0,
                                        _ptr(row_scale), _ptr(addend), out.data_ptr(),
                                        _raw_stream(dev, stream))
    if st:
        _raise("moe_linear_quantized", st)
    return out

"""Thin ctypes binding of the C ABI in include/mm.h.

Argument marshalling only: torch tensors supply device pointers and the
current CUDA stream; every step of the MoE layer runs in libmm.so's kernels.
There is no fallback: if the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmm.so")

MM_OK = 0
MM_ERR_INVALID_ARG = 1
MM_ERR_UNSUPPORTED = 2
MM_ERR_CUDA = 3
MM_ERR_NO_MEMORY = 4
MM_ERR_DEVICE = 5
MM_ERR_TIMEOUT = 6
MM_DTYPE_FP32, MM_DTYPE_BF16, MM_DTYPE_FP16 = 0, 1, 2
MM_GEMM_GATE_UP = 0
MM_GEMM_DOWN = 1
FORWARD_BLOCK_M = 16  # expert segments are padded to this multiple by mm_moe_forward

# Every entry point include/mm.h declares, with its ctypes signature.
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "mm_status_string": (ctypes.c_char_p, [_I]),
    "mm_route": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "mm_align_capacity": (_I64, [_I, _I, _I, _I]),
    "mm_align": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "mm_align_noalloc": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, _P]),
    "mm_grouped_gemm": (_I, [_I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "mm_moe_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "mm_moe_workspace_size": (_I64, [_I, _I, _I, _I, _I]),
    "mm_moe_workspace_layout": (_I, [_I, _I, _I, _I, _I, _P]),
    "mm_moe_forward_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "mm_moe_forward_profiled": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P,
                                     _P]),
    "mm_moe_forward_partial": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "mm_moe_forward_single_launch": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ,
                                          _P]),
    "mm_round_bf16": (_I, [_P, _P, _I64, _P]),
    "mm_gated_mlp": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "mm_gated_mlp_workspace_size": (_I64, [_I, _I, _I]),
    "mm_add_rmsnorm": (_I, [_P, _P, _P, ctypes.c_float, _I, _I, _P, _P]),
    "mm_moe_forward_add_norm": (_I, [_P, _P, _P, ctypes.c_float, _P, _P, _P, _I, _I, _I, _I, _I,
                                     _I, _P, _P]),
    "mm_moe_forward_add_norm_residual": (_I, [_P, _P, _P, ctypes.c_float, _P, _P, _P, _I, _I, _I,
                                              _I, _I, _I, _P, _P, _P]),
    "mm_poll_device_status": (_I, [_P]),
    "mm_selftest_wait_timeout": (_I, [_P]),
    "mm_selftest_layer_barrier_timeout": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                                               _P]),
    "mm_route_logits": (_I, [_P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "mm_route_logits_workspace_size": (_I64, [_I, _I]),
    "mm_route_logits_backward": (_I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "mm_mxfp4_quantize": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "mm_mxfp4_scales_size": (_I64, [_I, _I, _I]),
    "mm_mxfp4_dequantize": (_I, [_P, _P, _I, _I, _I, _P, _I, _P]),
    "mm_mxfp4_gemm": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _I, _P]),
    "mm_moe_experts_mxfp4": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ,
                                  _P]),
    "mm_moe_experts_mxfp4_workspace_size": (_I64, [_I, _I, _I, _I, _I]),
    "mm_shutdown": (None, []),
}

_lib: Optional[ctypes.CDLL] = None

# The marshalling of the short calls as an extension (csrc/marshal.cpp), loaded
# with the library. Its functions return None for a call that is not an ordinary
# one, and everything is marshalled here where it has not been built from these
# sources for this torch.
_fast = None


def _load_fast():
    from . import buildlib
    try:
        from . import _marshal
        return _marshal if getattr(_marshal, "tag", None) == buildlib.marshal_tag() else None
    except (ImportError, OSError):
        return None


class MMError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} (code {code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libmm.so (built by __graft_entry__.build()); raises if absent."""
    global _lib, _fast
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run __graft_entry__.build())")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
        _fast = _load_fast()
    return _lib


def status_string(code: int) -> str:
    return lib().mm_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != MM_OK:
        raise MMError(code, where)


def _ptr(t: Optional[torch.Tensor], dtype: torch.dtype, name: str) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _given(stream, di: int):
    """The caller's stream as torch's (a handle is one of device `di`)."""
    return (stream if isinstance(stream, torch.cuda.Stream)
            else torch.cuda.ExternalStream(int(stream), device=di))


def _empty(shape, dtype, like, stream, result: bool = True) -> torch.Tensor:
    """A result (or a workspace) on the device of `like` for a call on `stream`:
    of that stream's memory, since a block of the current one's may still be in
    use there by work that a given stream does not wait for."""
    if stream is None or not like.is_cuda:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(_given(stream, like.get_device())):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    if result and t.numel():  # read on the caller's stream, once that waits for this one
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def mm_align_capacity(T: int, top_k: int, E: int, block_m: int) -> int:
    return int(lib().mm_align_capacity(T, top_k, E, block_m))


def mm_moe_workspace_size(T: int, H: int, E: int, I: int, top_k: int) -> int:
    return int(lib().mm_moe_workspace_size(T, H, E, I, top_k))


# Fields of mm_moe_workspace_layout, in the order of its MM_WS_* indices.
WS_LAYOUT_FIELDS = ("topk_ids", "topk_w", "sorted_token_ids", "expert_offsets", "expert_counts",
                    "capacity", "block_m", "total")


def mm_moe_workspace_layout(T: int, H: int, E: int, I: int, top_k: int) -> dict:
    """Byte offsets of the routing and grouping inside a caller workspace of
    mm_moe_forward_ex, plus capacity, block_m and the total size."""
    buf = (ctypes.c_int64 * len(WS_LAYOUT_FIELDS))()
    _check(lib().mm_moe_workspace_layout(T, H, E, I, top_k, ctypes.cast(buf, ctypes.c_void_p)),
           "mm_moe_workspace_layout")
    return dict(zip(WS_LAYOUT_FIELDS, (int(v) for v in buf)))


def forward_routing(workspace, T: int, H: int, E: int, I: int, top_k: int) -> dict:
    """Views into a caller workspace that mm_moe_forward_ex just used: its
    own topk_ids, topk_w, sorted_token_ids, expert_offsets and expert_counts
    (valid once the call's kernels have completed)."""
    lay = mm_moe_workspace_layout(T, H, E, I, top_k)
    if workspace.dtype != torch.uint8 or workspace.numel() < lay["total"]:
        raise ValueError("workspace is not a caller workspace of these sizes")

    def view(name, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return workspace[lay[name]:lay[name] + nbytes].view(dtype)

    return {"topk_ids": view("topk_ids", T * top_k, torch.int32).view(T, top_k),
            "topk_w": view("topk_w", T * top_k, torch.float32).view(T, top_k),
            "sorted_token_ids": view("sorted_token_ids", lay["capacity"], torch.int32),
            "expert_offsets": view("expert_offsets", E + 1, torch.int32),
            "expert_counts": view("expert_counts", E, torch.int32),
            "block_m": lay["block_m"]}


def mm_route(hidden, router_w, top_k: int, renorm: bool, router_bias=None,
             topk_ids=None, topk_w=None, stream=None):
    """Router + softmax + top-k. Returns (topk_ids int32 [T,k], topk_w fp32 [T,k])."""
    T, H = hidden.shape
    E = router_w.shape[0]
    if topk_ids is None:
        topk_ids = _empty((T, top_k), torch.int32, hidden, stream)
    if topk_w is None:
        topk_w = _empty((T, top_k), torch.float32, hidden, stream)
    _check(lib().mm_route(_ptr(hidden, torch.bfloat16, "hidden"),
                          _ptr(router_w, torch.bfloat16, "router_w"),
                          _ptr(router_bias, torch.float32, "router_bias"),
                          T, H, E, top_k, int(bool(renorm)),
                          _ptr(topk_ids, torch.int32, "topk_ids"),
                          _ptr(topk_w, torch.float32, "topk_w"), _stream(stream)), "mm_route")
    return topk_ids, topk_w


def mm_align(topk_ids, E: int, block_m: int, sorted_token_ids=None, expert_offsets=None,
             expert_counts=None, stream=None):
    """Block-padded grouping by expert. Returns (sorted_token_ids, expert_offsets, expert_counts)."""
    T, k = topk_ids.shape
    cap = mm_align_capacity(T, k, E, block_m)
    if cap < 0:
        raise MMError(MM_ERR_INVALID_ARG, "mm_align_capacity")
    if sorted_token_ids is None:
        sorted_token_ids = _empty(cap, torch.int32, topk_ids, stream)
    if expert_offsets is None:
        expert_offsets = _empty(E + 1, torch.int32, topk_ids, stream)
    if expert_counts is None:
        expert_counts = _empty(E, torch.int32, topk_ids, stream)
    _check(lib().mm_align(_ptr(topk_ids, torch.int32, "topk_ids"), T, k, E, block_m,
                          _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
                          _ptr(expert_offsets, torch.int32, "expert_offsets"),
                          _ptr(expert_counts, torch.int32, "expert_counts"),
                          _stream(stream)), "mm_align")
    return sorted_token_ids, expert_offsets, expert_counts


def mm_align_noalloc(topk_ids, E: int, block_m: int, sorted_token_ids, expert_offsets,
                     expert_counts=None, stream=None):
    """mm_align with caller-owned outputs and no device allocation (see include/mm.h)."""
    T, k = topk_ids.shape
    _check(lib().mm_align_noalloc(_ptr(topk_ids, torch.int32, "topk_ids"), T, k, E, block_m,
                                  _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
                                  _ptr(expert_offsets, torch.int32, "expert_offsets"),
                                  _ptr(expert_counts, torch.int32, "expert_counts"),
                                  _stream(stream)), "mm_align_noalloc")
    return sorted_token_ids, expert_offsets, expert_counts


def mm_grouped_gemm(mode: int, A, B, C, sorted_token_ids, expert_offsets, topk_w,
                    T: int, top_k: int, block_m: int, stream=None):
    """One grouped GEMM (MM_GEMM_GATE_UP or MM_GEMM_DOWN); C is written in place."""
    E = B.shape[0]
    if mode == MM_GEMM_GATE_UP:
        N, K = B.shape[1] // 2, B.shape[2]
        cdt = torch.bfloat16
    else:
        N, K = B.shape[1], B.shape[2]
        cdt = torch.float32
    _check(lib().mm_grouped_gemm(mode, _ptr(A, torch.bfloat16, "A"), _ptr(B, torch.bfloat16, "B"),
                                 _ptr(C, cdt, "C"),
                                 _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
                                 _ptr(expert_offsets, torch.int32, "expert_offsets"),
                                 _ptr(topk_w, torch.float32, "topk_w"),
                                 T, top_k, E, N, K, block_m, _stream(stream)), "mm_grouped_gemm")
    return C


def mm_moe_forward(hidden, router_w, w_gate_up, w_down, top_k: int, renorm: bool,
                   out=None, router_bias=None, workspace=None, stream=None):
    """The whole MoE layer; returns out [T, H] bf16."""
    T, H = hidden.shape
    E = router_w.shape[0]
    I = w_down.shape[2]
    if out is None:
        out = _empty((T, H), torch.bfloat16, hidden, stream)
    if router_bias is None and workspace is None:
        _check(lib().mm_moe_forward(_ptr(hidden, torch.bfloat16, "hidden"),
                                    _ptr(router_w, torch.bfloat16, "router_w"),
                                    _ptr(w_gate_up, torch.bfloat16, "w_gate_up"),
                                    _ptr(w_down, torch.bfloat16, "w_down"),
                                    T, H, E, I, top_k, int(bool(renorm)),
                                    _ptr(out, torch.bfloat16, "out"), _stream(stream)),
               "mm_moe_forward")
        return out
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace, torch.uint8, "workspace"), workspace.numel()
    _check(lib().mm_moe_forward_ex(_ptr(hidden, torch.bfloat16, "hidden"),
                                   _ptr(router_w, torch.bfloat16, "router_w"),
                                   _ptr(router_bias, torch.float32, "router_bias"),
                                   _ptr(w_gate_up, torch.bfloat16, "w_gate_up"),
                                   _ptr(w_down, torch.bfloat16, "w_down"),
                                   T, H, E, I, top_k, int(bool(renorm)),
                                   _ptr(out, torch.bfloat16, "out"), ws_ptr, ws_bytes,
                                   _stream(stream)), "mm_moe_forward_ex")
    return out


def mm_moe_forward_single_launch(hidden, router_w, w_gate_up, w_down, top_k: int, renorm: bool,
                                 out=None, router_bias=None, workspace=None, stream=None):
    """The whole MoE layer in one cooperative launch (small batches; see
    include/mm.h for the shapes it takes); returns out [T, H] bf16."""
    T, H = hidden.shape
    E = router_w.shape[0]
    I = w_down.shape[2]
    if out is None:
        out = _empty((T, H), torch.bfloat16, hidden, stream)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace, torch.uint8, "workspace"), workspace.numel()
    _check(lib().mm_moe_forward_single_launch(
        _ptr(hidden, torch.bfloat16, "hidden"), _ptr(router_w, torch.bfloat16, "router_w"),
        _ptr(router_bias, torch.float32, "router_bias"),
        _ptr(w_gate_up, torch.bfloat16, "w_gate_up"), _ptr(w_down, torch.bfloat16, "w_down"),
        T, H, E, I, top_k, int(bool(renorm)), _ptr(out, torch.bfloat16, "out"), ws_ptr, ws_bytes,
        _stream(stream)), "mm_moe_forward_single_launch")
    return out


def tp_slice(w_gate_up, w_down, rank: int, world: int):
    """The expert weights rank `rank` of `world` holds under tensor
    parallelism: gate rows [i0, i0 + I/world) and the same up rows of every
    expert, as one [E, 2*I/world, H] tensor (gate slice first), and the same
    columns of w_down, [E, H, I/world]. Weight preparation (done once, like
    the loader's sharding), for torch tensors or numpy arrays."""
    E, twoI, H = w_gate_up.shape
    I = twoI // 2
    if world < 1 or I % world != 0:
        raise ValueError(f"I={I} does not split into {world} equal slices")
    il = I // world
    i0 = rank * il
    gate, up = w_gate_up[:, i0:i0 + il, :], w_gate_up[:, I + i0:I + i0 + il, :]
    if isinstance(w_gate_up, torch.Tensor):
        return torch.cat([gate, up], dim=1).contiguous(), w_down[:, :, i0:i0 + il].contiguous()
    import numpy as np
    return (np.ascontiguousarray(np.concatenate([gate, up], axis=1)),
            np.ascontiguousarray(w_down[:, :, i0:i0 + il]))


def mm_moe_forward_partial(hidden, router_w, w_gate_up_slice, w_down_slice, top_k: int,
                           renorm: bool, partial=None, router_bias=None, workspace=None,
                           stream=None):
    """The layer on one tensor-parallel slice of the experts' intermediates
    (see tp_slice): returns this rank's unrounded fp32 contribution [T, H]."""
    T, H = hidden.shape
    E = router_w.shape[0]
    I = w_down_slice.shape[2]
    if partial is None:
        partial = _empty((T, H), torch.float32, hidden, stream)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace, torch.uint8, "workspace"), workspace.numel()
    _check(lib().mm_moe_forward_partial(_ptr(hidden, torch.bfloat16, "hidden"),
                                        _ptr(router_w, torch.bfloat16, "router_w"),
                                        _ptr(router_bias, torch.float32, "router_bias"),
                                        _ptr(w_gate_up_slice, torch.bfloat16, "w_gate_up_slice"),
                                        _ptr(w_down_slice, torch.bfloat16, "w_down_slice"),
                                        T, H, E, I, top_k, int(bool(renorm)),
                                        _ptr(partial, torch.float32, "partial"), ws_ptr, ws_bytes,
                                        _stream(stream)), "mm_moe_forward_partial")
    return partial


def mm_round_bf16(x, out=None, stream=None):
    """bf16 rounding (to nearest even) of an fp32 tensor, on the GPU."""
    if out is None:
        out = _empty(x.shape, torch.bfloat16, x, stream)
    _check(lib().mm_round_bf16(_ptr(x, torch.float32, "x"), _ptr(out, torch.bfloat16, "out"),
                               x.numel(), _stream(stream)), "mm_round_bf16")
    return out


def mm_gated_mlp_workspace_size(T: int, H: int, I: int) -> int:
    return int(lib().mm_gated_mlp_workspace_size(T, H, I))


def mm_gated_mlp(hidden, w_gate_up, w_down, out=None, stream=None):
    """Dense SwiGLU MLP through the grouped-GEMM kernels; returns out [T, H] bf16."""
    T, H = hidden.shape
    I = w_down.shape[1]
    if out is None:
        out = _empty((T, H), torch.bfloat16, hidden, stream)
    _check(lib().mm_gated_mlp(_ptr(hidden, torch.bfloat16, "hidden"),
                              _ptr(w_gate_up, torch.bfloat16, "w_gate_up"),
                              _ptr(w_down, torch.bfloat16, "w_down"), T, H, I,
                              _ptr(out, torch.bfloat16, "out"), _stream(stream)), "mm_gated_mlp")
    return out


def mm_add_rmsnorm(x, norm_w, eps: float, residual=None, normed=None, stream=None):
    """residual <- bf16(x + residual) in place (residual None: x is the
    residual); returns normed = rmsnorm(residual, norm_w, eps) [T, H] bf16."""
    T, H = x.shape
    if normed is None:
        normed = _empty((T, H), torch.bfloat16, x, stream)
    _check(lib().mm_add_rmsnorm(_ptr(x, torch.bfloat16, "x"),
                                _ptr(residual, torch.bfloat16, "residual"),
                                _ptr(norm_w, torch.bfloat16, "norm_w"), float(eps), T, H,
                                _ptr(normed, torch.bfloat16, "normed"), _stream(stream)),
           "mm_add_rmsnorm")
    return normed


def mm_moe_forward_add_norm(x, norm_w, eps: float, router_w, w_gate_up, w_down, top_k: int,
                            renorm: bool, residual=None, out=None, stream=None):
    """The MoE layer on rmsnorm(x + residual) (residual updated in place, or
    x itself when residual is None); returns out [T, H] bf16."""
    T, H = x.shape
    E = router_w.shape[0]
    I = w_down.shape[2]
    if out is None:
        out = _empty((T, H), torch.bfloat16, x, stream)
    _check(lib().mm_moe_forward_add_norm(_ptr(x, torch.bfloat16, "x"),
                                         _ptr(residual, torch.bfloat16, "residual"),
                                         _ptr(norm_w, torch.bfloat16, "norm_w"), float(eps),
                                         _ptr(router_w, torch.bfloat16, "router_w"),
                                         _ptr(w_gate_up, torch.bfloat16, "w_gate_up"),
                                         _ptr(w_down, torch.bfloat16, "w_down"), T, H, E, I,
                                         top_k, int(bool(renorm)),
                                         _ptr(out, torch.bfloat16, "out"), _stream(stream)),
           "mm_moe_forward_add_norm")
    return out


def mm_moe_forward_add_norm_residual(x, norm_w, eps: float, router_w, w_gate_up, w_down,
                                     top_k: int, renorm: bool, residual=None, residual_out=None,
                                     out=None, stream=None):
    """The MoE half of a decoder layer: residual' = bf16(x + residual) (in
    place; x when residual is None), out = layer(rmsnorm(residual')), and
    residual_out = bf16(out + residual') (default: residual itself, updated
    in place; a new tensor when residual is None). Returns (out, residual_out)."""
    T, H = x.shape
    E = router_w.shape[0]
    I = w_down.shape[2]
    if out is None:
        out = _empty((T, H), torch.bfloat16, x, stream)
    if residual_out is None:
        residual_out = (residual if residual is not None
                        else _empty(x.shape, x.dtype, x, stream))
    _check(lib().mm_moe_forward_add_norm_residual(
        _ptr(x, torch.bfloat16, "x"), _ptr(residual, torch.bfloat16, "residual"),
        _ptr(norm_w, torch.bfloat16, "norm_w"), float(eps),
        _ptr(router_w, torch.bfloat16, "router_w"), _ptr(w_gate_up, torch.bfloat16, "w_gate_up"),
        _ptr(w_down, torch.bfloat16, "w_down"), T, H, E, I, top_k, int(bool(renorm)),
        _ptr(out, torch.bfloat16, "out"), _ptr(residual_out, torch.bfloat16, "residual_out"),
        _stream(stream)), "mm_moe_forward_add_norm_residual")
    return out, residual_out


PROFILE_STAGES = ("route", "align", "gate_up", "down", "finalize")


def mm_moe_forward_profiled(hidden, router_w, w_gate_up, w_down, top_k: int, renorm: bool,
                            events, out=None, router_bias=None, workspace=None, stream=None):
    """mm_moe_forward that records len(PROFILE_STAGES)+1 torch.cuda.Event
    (timing enabled) around its stages on the stream; returns out."""
    T, H = hidden.shape
    E = router_w.shape[0]
    I = w_down.shape[2]
    if len(events) != len(PROFILE_STAGES) + 1:
        raise ValueError(f"need {len(PROFILE_STAGES) + 1} events")
    if out is None:
        out = _empty((T, H), torch.bfloat16, hidden, stream)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = _ptr(workspace, torch.uint8, "workspace"), workspace.numel()
    for e in events:  # torch creates the CUDA event on its first record
        if e.cuda_event == 0:
            e.record()
    ev = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().mm_moe_forward_profiled(_ptr(hidden, torch.bfloat16, "hidden"),
                                         _ptr(router_w, torch.bfloat16, "router_w"),
                                         _ptr(router_bias, torch.float32, "router_bias"),
                                         _ptr(w_gate_up, torch.bfloat16, "w_gate_up"),
                                         _ptr(w_down, torch.bfloat16, "w_down"),
                                         T, H, E, I, top_k, int(bool(renorm)),
                                         _ptr(out, torch.bfloat16, "out"), ws_ptr, ws_bytes,
                                         _stream(stream), ev), "mm_moe_forward_profiled")
    return out


def mm_poll_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status code."""
    return int(lib().mm_poll_device_status(_stream(stream)))


def mm_selftest_wait_timeout(stream=None) -> None:
    """Launches the kernel whose bounded wait must time out (see include/mm.h)."""
    _check(lib().mm_selftest_wait_timeout(_stream(stream)), "mm_selftest_wait_timeout")


def mm_selftest_layer_barrier_timeout(hidden, router_w, w_gate_up, w_down, top_k: int,
                                      renorm: bool, barrier: int, out=None, stream=None):
    """Runs the single-launch small-batch layer with CTA 0 absent from grid
    barrier `barrier` (see include/mm.h); every CTA's wait there runs out.
    Returns out (undefined contents)."""
    T, H = hidden.shape
    E = router_w.shape[0]
    I = w_down.shape[2]
    if out is None:
        out = _empty((T, H), torch.bfloat16, hidden, stream)
    _check(lib().mm_selftest_layer_barrier_timeout(
        _ptr(hidden, torch.bfloat16, "hidden"), _ptr(router_w, torch.bfloat16, "router_w"),
        _ptr(w_gate_up, torch.bfloat16, "w_gate_up"), _ptr(w_down, torch.bfloat16, "w_down"),
        T, H, E, I, top_k, int(bool(renorm)), barrier, _ptr(out, torch.bfloat16, "out"),
        _stream(stream)), "mm_selftest_layer_barrier_timeout")
    return out


_DTYPES = {torch.float32: MM_DTYPE_FP32, torch.bfloat16: MM_DTYPE_BF16,
           torch.float16: MM_DTYPE_FP16}


def _dtype(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return dt


def _shape(t, shape, name: str) -> None:
    if t is not None and t.shape != shape:  # torch.Size compares as a tuple
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _mask_ptr(mask, T: int):
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"token_mask must be bool or uint8, got {mask.dtype}")
    _shape(mask, (T,), "token_mask")
    return _ptr(mask, mask.dtype, "token_mask")


def _device(name: str, *tensors) -> None:
    """All tensors (None: absent) have to be on the first one's device."""
    di = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != di:
            raise ValueError(f"{name}: all tensors must be on {tensors[0].device}, got {t.device}")


class _On:
    """Where a call runs: the device of `like`, and `stream` (the caller's, else
    that device's current one)."""

    def __init__(self, name: str, like: torch.Tensor, stream):
        self.name, self.like, self.di, self.stream = name, like, like.get_device(), None
        if stream is not None:
            s = _given(stream, self.di)
            if s.device_index != self.di:
                raise ValueError(f"{name}: the stream is on another device than the tensors")
            if s.cuda_stream != torch._C._cuda_getCurrentRawStream(self.di):
                self.stream = s

    def empty(self, shape, dtype, result: bool = True) -> torch.Tensor:
        return _empty(shape, dtype, self.like, self.stream, result)

    def parts(self, *parts) -> list:
        """Tensors (shape, dtype) of one allocation, 256-byte aligned each, as
        the extension makes them."""
        sizes = [math.prod(shape) * dtype.itemsize for shape, dtype in parts]
        at = [0]
        for n in sizes:
            at.append(at[-1] + (n + 255) // 256 * 256)
        whole = self.empty(at[-1], torch.uint8)
        return [torch.empty(0, dtype=dtype, device=whole.device).set_(
                    whole.untyped_storage(), o // dtype.itemsize, shape)
                for (shape, dtype), o in zip(parts, at)]

    def launch(self, fn, *args) -> None:
        """fn(*args, stream handle)."""
        st = (torch._C._cuda_getCurrentRawStream(self.di) if self.stream is None
              else self.stream.cuda_stream)
        if torch._C._cuda_getDevice() == self.di:
            rc = fn(*args, st)
        else:
            with torch.cuda.device(self.di):
                rc = fn(*args, st)
        if rc != MM_OK:
            raise MMError(rc, self.name)


def mm_route_logits(logits, top_k: int, renorm: bool, token_mask=None, stream=None):
    """Top-k routing of given router logits [T, E] (float32 or bfloat16) with
    the statistics of the balance loss. Returns (topk_ids int32 [T, k],
    topk_w fp32 [T, k], expert_counts int32 [E], prob_sums fp32 [E],
    loss fp32 [1]). token_mask [T] (bool or uint8): zero for padding tokens.
    Ids and weights share one allocation, and so do the other three: clone()
    what is to be stored on its own. Results carry no autograd graph:
    mm_route_logits_backward is the gradient."""
    if _fast is not None and stream is None:
        r = _fast.route_logits(logits, top_k, renorm, token_mask)
        if r is not None:
            return r
    dt = _dtype(logits, "logits")
    T, E = logits.shape
    x = _ptr(logits, logits.dtype, "logits")
    mask = _mask_ptr(token_mask, T)
    _device("mm_route_logits", logits, token_mask)
    l = lib()
    need = l.mm_route_logits_workspace_size(T, E)
    # Refused here already: results of such a size are not to be allocated.
    if E == 0 or top_k <= 0:
        raise MMError(MM_ERR_INVALID_ARG, "mm_route_logits")
    if need < 0 or top_k > E or T * top_k >= 1 << 31:
        raise MMError(MM_ERR_UNSUPPORTED, "mm_route_logits")
    on = _On("mm_route_logits", logits, stream)
    ids, w = on.parts(((T, top_k), torch.int32), ((T, top_k), torch.float32))
    counts, sums, loss = on.parts(((E,), torch.int32), ((E,), torch.float32),
                                  ((1,), torch.float32))
    ws = on.empty(need, torch.uint8, result=False) if need > 0 else None
    on.launch(l.mm_route_logits, x, dt, mask, T, E, top_k, 1 if renorm else 0, ids.data_ptr(),
              w.data_ptr(), counts.data_ptr(), sums.data_ptr(), loss.data_ptr(),
              None if ws is None else ws.data_ptr(), need)
    return ids, w, counts, sums, loss


def mm_route_logits_backward(logits, topk_ids, expert_counts, renorm: bool, d_topk_w=None,
                             d_loss=None, token_mask=None, stream=None):
    """The gradient of mm_route_logits: d_logits [T, E] of the logits' dtype
    from d_topk_w [T, k] fp32 and / or d_loss [1] fp32. expert_counts may be
    the sum over several replicas (the loss is then the one over all of them)."""
    if _fast is not None and stream is None:
        r = _fast.route_logits_backward(logits, topk_ids, expert_counts, renorm, d_topk_w, d_loss,
                                        token_mask)
        if r is not None:
            return r
    dt = _dtype(logits, "logits")
    T, E = logits.shape
    k = topk_ids.shape[1]
    _shape(topk_ids, (T, k), "topk_ids")
    _shape(expert_counts, (E,), "expert_counts")
    _shape(d_topk_w, (T, k), "d_topk_w")
    if d_loss is not None and d_loss.numel() != 1:
        raise ValueError("d_loss must hold one value")
    x, mask = _ptr(logits, logits.dtype, "logits"), _mask_ptr(token_mask, T)
    ids, counts = (_ptr(topk_ids, torch.int32, "topk_ids"),
                   _ptr(expert_counts, torch.int32, "expert_counts"))
    dw, dl = _ptr(d_topk_w, torch.float32, "d_topk_w"), _ptr(d_loss, torch.float32, "d_loss")
    _device("mm_route_logits_backward", logits, token_mask, topk_ids, expert_counts, d_topk_w,
            d_loss)
    on = _On("mm_route_logits_backward", logits, stream)
    grad = on.empty((T, E), logits.dtype)
    on.launch(lib().mm_route_logits_backward, x, dt, mask, ids, counts, dw, dl, T, E, k,
              1 if renorm else 0, grad.data_ptr())
    return grad


def mm_mxfp4_scales_shape(rows: int, K: int) -> tuple:
    """Shape of the scale tiles of one [rows, K] matrix."""
    return ((rows + 127) // 128, (K + 127) // 128, 512)


def mxfp4_tile_scales(scales):
    """Scale bytes [..., rows, K/32] in plain row order -> the stored tiles
    [..., ceil(rows/128), ceil(K/128), 512] (weight preparation, done once)."""
    lead, (rows, cols) = scales.shape[:-2], scales.shape[-2:]
    rt, kt, _ = mm_mxfp4_scales_shape(rows, cols * 32)
    s = scales.new_zeros((*lead, rt * 128, kt * 4))
    s[..., :rows, :cols] = scales
    s = s.reshape(-1, rt, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5)
    return s.reshape(*lead, rt, kt, 512).contiguous()


def mm_mxfp4_quantize(x, stream=None):
    """x [rows, K] or [batch, rows, K] (float32, bfloat16, float16; K % 32 == 0)
    as microscaled 4-bit floats. Returns (codes uint8 [..., rows, K/2],
    scales uint8 [..., ceil(rows/128), ceil(K/128), 512])."""
    if _fast is not None and stream is None:
        r = _fast.mxfp4_quantize(x)
        if r is not None:
            return r
    dt = _dtype(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError("x must have 2 or 3 dimensions")
    lead, (rows, K) = x.shape[:-2], x.shape[-2:]
    batch = lead[0] if lead else 1
    xp = _ptr(x, x.dtype, "x")
    if K % 32 != 0 or K == 0:
        raise MMError(MM_ERR_UNSUPPORTED if K else MM_ERR_INVALID_ARG, "mm_mxfp4_quantize")
    on = _On("mm_mxfp4_quantize", x, stream)
    codes = on.empty((*lead, rows, K // 2), torch.uint8)
    scales = on.empty((*lead, *mm_mxfp4_scales_shape(rows, K)), torch.uint8)
    on.launch(lib().mm_mxfp4_quantize, xp, dt, batch, rows, K, codes.data_ptr(),
              scales.data_ptr())
    return codes, scales


def mm_mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, stream=None):
    """The values [..., rows, K] of codes [..., rows, K/2] and their scale tiles."""
    if _fast is not None and stream is None:
        r = _fast.mxfp4_dequantize(codes, scales, _DTYPES.get(dtype, -1))
        if r is not None:
            return r
    if codes.dim() not in (2, 3):
        raise ValueError("codes must have 2 or 3 dimensions")
    lead, (rows, half) = codes.shape[:-2], codes.shape[-2:]
    K, batch = 2 * half, (lead[0] if lead else 1)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    cp, sp = _ptr(codes, torch.uint8, "codes"), _ptr(scales, torch.uint8, "scales")
    _shape(scales, (*lead, *mm_mxfp4_scales_shape(rows, K)), "scales")
    _device("mm_mxfp4_dequantize", codes, scales)
    on = _On("mm_mxfp4_dequantize", codes, stream)
    out = on.empty((*lead, rows, K), dtype)
    on.launch(lib().mm_mxfp4_dequantize, cp, sp, batch, rows, K, out.data_ptr(), _DTYPES[dtype])
    return out


def _matrix(codes, scales, name: str):
    """(rows, K) and the pointers of one 4-bit matrix (a leading dimension of 1 allowed)."""
    shape = codes.shape
    if len(shape) == 3 and shape[0] == 1:
        shape = shape[1:]
    if len(shape) != 2:
        raise ValueError(f"{name} must be one matrix, got codes of shape {tuple(codes.shape)}")
    rows, half = shape
    tiles = ((rows + 127) // 128, (2 * half + 127) // 128, 512)
    if scales.shape != tiles and scales.shape != (1, *tiles):
        raise ValueError(f"{name} scales must have shape {tiles}, got {tuple(scales.shape)}")
    return (rows, 2 * half, _ptr(codes, torch.uint8, name),
            _ptr(scales, torch.uint8, "scales"))


def mm_mxfp4_gemm(a_codes, a_scales, b_codes, b_scales, out_dtype=torch.bfloat16, stream=None):
    """C [M, N] = A B^T of two 4-bit matrices [M, K] and [N, K]; bfloat16 or float32."""
    if _fast is not None and stream is None:
        r = _fast.mxfp4_gemm(a_codes, a_scales, b_codes, b_scales, _DTYPES.get(out_dtype, -1))
        if r is not None:
            return r
    M, K, a, sa = _matrix(a_codes, a_scales, "a")
    N, Kb, b, sb = _matrix(b_codes, b_scales, "b")
    if K != Kb:
        raise ValueError(f"a has {K} columns, b has {Kb}")
    if out_dtype not in _DTYPES:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    _device("mm_mxfp4_gemm", a_codes, a_scales, b_codes, b_scales)
    on = _On("mm_mxfp4_gemm", a_codes, stream)
    c = on.empty((M, N), out_dtype)
    on.launch(lib().mm_mxfp4_gemm, a, sa, b, sb, M, N, K, c.data_ptr(), _DTYPES[out_dtype])
    return c


def mm_moe_experts_mxfp4_workspace_size(T: int, H: int, E: int, I: int, top_k: int) -> int:
    return int(lib().mm_moe_experts_mxfp4_workspace_size(T, H, E, I, top_k))


def mm_moe_experts_mxfp4(hidden, topk_ids, topk_w, w_gate_up, w_gate_up_scales, w_down,
                         w_down_scales, out=None, workspace=None, stream=None):
    """The experts of the layer with 4-bit weights for a given routing; returns
    out [T, H] bf16. w_gate_up: codes [2E, I, H/2] (or [E, 2I, H/2]) with the
    scale tiles of 2E matrices [I, H]; w_down: codes [E, H, I/2]. workspace:
    uint8 of mm_moe_experts_mxfp4_workspace_size bytes (allocated per call if
    None)."""
    if _fast is not None and stream is None:
        r = _fast.experts_mxfp4(hidden, topk_ids, topk_w, w_gate_up, w_gate_up_scales, w_down,
                                w_down_scales, out, workspace)
        if r is not None:
            return r
    T, H = hidden.shape
    k = topk_ids.shape[1]
    E, _, half = w_down.shape
    I = 2 * half
    _shape(topk_ids, (T, k), "topk_ids")
    _shape(topk_w, (T, k), "topk_w")
    _shape(w_down, (E, H, half), "w_down")
    if tuple(w_gate_up.shape) != (E, 2 * I, H // 2):
        _shape(w_gate_up, (2 * E, I, H // 2), "w_gate_up")
    _shape(w_gate_up_scales, (2 * E, *mm_mxfp4_scales_shape(I, H)), "w_gate_up_scales")
    _shape(w_down_scales, (E, *mm_mxfp4_scales_shape(H, I)), "w_down_scales")
    x, ids, w = (_ptr(hidden, torch.bfloat16, "hidden"), _ptr(topk_ids, torch.int32, "topk_ids"),
                 _ptr(topk_w, torch.float32, "topk_w"))
    gu, sgu = (_ptr(w_gate_up, torch.uint8, "w_gate_up"),
               _ptr(w_gate_up_scales, torch.uint8, "w_gate_up_scales"))
    dn, sdn = (_ptr(w_down, torch.uint8, "w_down"),
               _ptr(w_down_scales, torch.uint8, "w_down_scales"))
    _shape(out, (T, H), "out")
    outp, ws = _ptr(out, torch.bfloat16, "out"), _ptr(workspace, torch.uint8, "workspace")
    _device("mm_moe_experts_mxfp4", hidden, topk_ids, topk_w, w_gate_up, w_gate_up_scales,
            w_down, w_down_scales, out, workspace)
    l, on = lib(), _On("mm_moe_experts_mxfp4", hidden, stream)
    if out is None:
        out = on.empty((T, H), torch.bfloat16)
        outp = out.data_ptr()
    if workspace is None:
        need = l.mm_moe_experts_mxfp4_workspace_size(T, H, E, I, k)
        workspace = on.empty(max(need, 0), torch.uint8, result=False)
        ws = workspace.data_ptr()
    on.launch(l.mm_moe_experts_mxfp4, x, ids, w, gu, sgu, dn, sdn, T, H, E, I, k, outp, ws,
              workspace.numel())
    return out


def mm_shutdown() -> None:
    lib().mm_shutdown()

"""Python binding of libmoe, the GB300 (sm_103a) forward pass of a
Mixture-of-Experts FFN layer:

    y = g(x) * shared(x) + sum_k route_weight_k * SwiGLU-expert_k(x)

Every function here marshals torch tensors into the C ABI declared in
``include/moe.h`` (same names, same argument order) and raises ``MoEError``
on a non-OK status.  All arithmetic runs in the library's CUDA kernels;
PyTorch only provides device memory and the current stream.  There is no
fallback: if ``libmoe.so`` is missing or fails to load, every call raises.
"""
from __future__ import annotations

import bisect
import ctypes
import os
from typing import NamedTuple, Optional

import torch

from . import workloads  # noqa: F401  (seeded input generators)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE = 0, 1, 2, 3
MOE_ERR_CUDA, MOE_ERR_DEVICE_ROUTE, MOE_ERR_TIMEOUT, MOE_ERR_ROWS = 4, 5, 6, 7
MOE_ERR_GATHER = 8
MOE_ERR_TARGET = 9
MOE_ERR_TOKEN = 10
MOE_F32, MOE_BF16 = 0, 1
STAGES = ("residual_setup", "route", "permute", "gate_up", "down", "shared", "combine")


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str, why: str = ""):
        self.status = status
        super().__init__("%s: %s%s" % (where, moe_status_string(status),
                                       (" (" + why + ")") if why else ""))


class MoEShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int32),
                ("moe_inter", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
                ("topk_shape", ctypes.c_uint32), ("shared_gate", ctypes.c_int32),
                ("norm_topk", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("input_norm", ctypes.c_int32), ("residual", ctypes.c_int32),
                ("norm_eps", ctypes.c_double), ("train", ctypes.c_int32),
                ("weight_format", ctypes.c_int32)]


class MoEWeights(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p),
                ("gate_up_stride", ctypes.c_int64), ("down", ctypes.c_void_p),
                ("down_stride", ctypes.c_int64), ("shared_gate_proj", ctypes.c_void_p),
                ("shared_up", ctypes.c_void_p), ("shared_down", ctypes.c_void_p),
                ("norm_weight", ctypes.c_void_p)]


class MoEExpertGrads(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p),
                ("gate_up_stride", ctypes.c_int64), ("down", ctypes.c_void_p),
                ("down_stride", ctypes.c_int64)]


class MoEBackwardInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("fc1", "grad_fc2", "d_fc1", "dx_perm")]


class MoECeShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
                ("ignore_index", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("w_stride", ctypes.c_int64)]


class MoEGradTensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("src_dtype", ctypes.c_int32), ("dst_dtype", ctypes.c_int32)]


class MoEGradPlan(ctypes.Structure):
    _fields_ = [("tensors", ctypes.c_int64), ("chunks", ctypes.c_int64),
                ("chunk_elems", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoEEmbedShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("padding_idx", ctypes.c_int32),
                ("scale", ctypes.c_double), ("w_stride", ctypes.c_int64)]


class MoEBlockNormShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("unit_offset", ctypes.c_int32),
                ("residual_scale", ctypes.c_double), ("eps", ctypes.c_double)]


MOE_ORTH_MAX_STEPS = 16


class MoEOrthCoefs(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("reserved", ctypes.c_int32), ("eps", ctypes.c_double),
                ("coef", (ctypes.c_double * 3) * MOE_ORTH_MAX_STEPS)]


class MoEOrthShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoEMuonTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class MoEMuonConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("momentum", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("nesterov", ctypes.c_int32),
                ("scale", ctypes.c_int32), ("coefs", MoEOrthCoefs)]


class MoERouteInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_idx", "topk_w", "gate", "counts", "offsets", "scatter_index", "row_token",
        "x_perm", "h", "y_perm", "shared_out")]


_lib = None


def lib():
    """The loaded libmoe (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libmoe.so is not built (run __graft_entry__.build() or "
                           "python -m mixture_experts_ffn_04_gb300.build)")
    L = ctypes.CDLL(LIB_PATH)
    P, S, i32, i64, u32, sz = (ctypes.c_void_p, ctypes.POINTER(MoEShape), ctypes.c_int32,
                               ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t)
    C = ctypes.POINTER(MoECeShape)
    M, N = ctypes.POINTER(MoEEmbedShape), ctypes.POINTER(MoEBlockNormShape)
    O, K = ctypes.POINTER(MoEOrthShape), ctypes.POINTER(MoEOrthCoefs)
    sig = {
        "moe_topk_pack": (u32, [i32, i32]),
        "moe_topk_unpack": (i32, [u32, ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "moe_scratch_bytes": (sz, [S]),
        "moe_workspace_bytes": (sz, [S]),
        "moe_workspace_views": (i32, [S, P, ctypes.POINTER(MoERouteInfo)]),
        "moe_workspace_init": (i32, [P, P]),
        "moe_quantize_mxfp8": (i32, [P, i32, i64, i64, i32, i64, i64, P, P]),
        "moe_route": (i32, [S, P, P, P, P, P, P, sz, P]),
        "moe_hash_route": (i32, [S, P, P, i64, P, P, P, sz, P]),
        "moe_permute": (i32, [S, P, P, P, P, P, P, P, P, sz, P]),
        "moe_permute_static": (i32, [S, P, P, P, P, P, P, P, P]),
        "moe_grouped_swiglu": (i32, [S, P, P, P, i64, P, i32, i64, i32, P, P, sz, P]),
        "moe_grouped_swiglu_gather": (i32, [S, P, P, P, P, i64, P, i32, i64, i32, P, P, sz, P]),
        "moe_grouped_down": (i32, [S, P, P, i64, P, i32, i64, i32, P, P, sz, P]),
        "moe_combine": (i32, [S, P, P, P, P, P, P, P, P]),
        "moe_residual_setup": (i32, [S, P, P, P, P]),
        "moe_layer_forward": (i32, [S, ctypes.POINTER(MoEWeights), P, P, P, P, P, sz, P]),
        "moe_layer_forward_traced": (i32, [S, ctypes.POINTER(MoEWeights), P, P, P, P, P, sz, P,
                                           ctypes.POINTER(ctypes.c_void_p)]),
        "moe_get_device_status": (i32, [P, P, ctypes.POINTER(u32)]),
        "moe_status_string": (ctypes.c_char_p, [i32]),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_stage_name": (ctypes.c_char_p, [i32]),
        "moe_last_launch_count": (i32, []),
        "moe_testing_set_gemm_engine": (i32, [i32]),
        "moe_testing_set_fork_sms": (i32, [i32]),
        "moe_testing_set_zero_pad": (i32, [i32]),
        "moe_testing_set_norm_wait": (i64, [i64]),
        "moe_get_route_stats": (i32, [P, P, ctypes.POINTER(u32)]),
        "moe_testing_router_logits": (i32, [S, P, P, P, P, sz, P]),
        "moe_testing_wait_probe": (i32, [P, i64, i32, P]),
        # backward (moe_backward.h)
        "moe_backward_views": (i32, [S, P, ctypes.POINTER(MoEBackwardInfo)]),
        "moe_grouped_swiglu_save": (i32, [S, P, P, P, i64, P, i32, i64, i32, P, P, P, sz, P]),
        "moe_scatter_grad": (i32, [S, P, P, P, P, P, P, P]),
        "moe_grouped_down_dgrad": (i32, [S, P, P, i64, P, P, i32, i64, i32, P, P, sz, P]),
        "moe_grouped_gate_up_dgrad": (i32, [S, P, P, P, i64, P, i32, i64, i32, P, P, sz, P]),
        "moe_grouped_wgrad": (i32, [S, P, i64, P, i64, P, i32, i64, i32, i32, P, i64, P, sz, P]),
        "moe_gather_grad": (i32, [S, P, P, P, P, P]),
        "moe_layer_backward": (i32, [S, ctypes.POINTER(MoEWeights), P, P, P,
                                     ctypes.POINTER(MoEExpertGrads), P, sz, P]),
        # training operators (moe_train.h)
        "moe_linear_ce_workspace_bytes": (sz, [C]),
        "moe_linear_ce_forward": (i32, [C, P, P, P, P, P, P, P, P, sz, P]),
        "moe_linear_ce_backward": (i32, [C, P, P, P, P, P, P, P, P, sz, P]),
        "moe_router_backward_workspace_bytes": (sz, [S]),
        "moe_router_backward": (i32, [S, P, P, P, P, P, ctypes.c_double, ctypes.c_double, P, P, P,
                                      P, P, sz, P]),
        "moe_grad_clip_workspace_bytes": (sz, [P, i64]),
        "moe_grad_clip_plan": (i32, [P, i64, ctypes.POINTER(MoEGradPlan), P, sz, P]),
        "moe_grad_clip": (i32, [ctypes.POINTER(MoEGradPlan), ctypes.c_double, P, P, sz, P]),
        # operators between the layer and the rest of a model (moe_model.h)
        "moe_embed_workspace_bytes": (sz, [M]),
        "moe_embed_forward": (i32, [M, P, P, P, P, sz, P]),
        "moe_embed_backward": (i32, [M, P, P, P, P, P, sz, P]),
        "moe_block_norm_workspace_bytes": (sz, [N]),
        "moe_block_norm_forward": (i32, [N] + [P] * 9),
        "moe_block_norm_backward": (i32, [N] + [P] * 14 + [sz, P]),
        "moe_orthogonalize_workspace_bytes": (sz, [O, K]),
        "moe_orthogonalize": (i32, [O, K, P, P, P, sz, P]),
        "moe_muon_workspace_bytes": (sz, [P, i64, ctypes.POINTER(MoEMuonConfig)]),
        "moe_muon_step": (i32, [P, i64, ctypes.POINTER(MoEMuonConfig), P, sz, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


# The current stream's handle without the Stream object that torch.cuda makes around
# it (3 us of a small call); not part of torch's public interface, so it may be absent.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def _check(st: int, where: str):
    if st != MOE_OK:
        why = lib().moe_last_error()
        raise MoEError(st, where, why.decode() if why else "")


def _dtype_code(dt: torch.dtype) -> int:
    return {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}[dt]


# ---------------------------------------------------------------------------
# the C ABI, name for name
# ---------------------------------------------------------------------------
def moe_topk_pack(num_experts: int, top_k: int) -> int:
    return int(lib().moe_topk_pack(num_experts, top_k))


def moe_topk_unpack(word: int):
    e, k = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_topk_unpack(word, ctypes.byref(e), ctypes.byref(k)), "moe_topk_unpack")
    return e.value, k.value


def moe_scratch_bytes(shape: MoEShape) -> int:
    return int(lib().moe_scratch_bytes(ctypes.byref(shape)))


def moe_workspace_bytes(shape: MoEShape) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(shape)))


def moe_quantize_mxfp8(w, batch, rows, K, src_stride, dst_stride, packed, stream=None):
    """Packed MXFP8 matrices from bf16 / fp32 ones (see include/moe.h)."""
    _check(lib().moe_quantize_mxfp8(_p(w), _dtype_code(w.dtype), batch, rows, K, src_stride,
                                    dst_stride, _p(packed), _stream(stream)),
           "moe_quantize_mxfp8")


def mxfp8_pack(w: torch.Tensor, stream=None) -> torch.Tensor:
    """[..., N, K] weights -> [..., N*K*9/8] uint8 packed MXFP8 matrices (the
    leading dimensions are the batch), on w's device."""
    N, K = w.shape[-2], w.shape[-1]
    batch = w.numel() // (N * K)
    out = torch.empty(tuple(w.shape[:-2]) + (N * K // 8 * 9,), dtype=torch.uint8, device=w.device)
    moe_quantize_mxfp8(w, batch, N, K, N * K, N * K // 8 * 9, out, stream)
    return out


MOE_WEIGHTS_ACT, MOE_WEIGHTS_MXFP8 = 0, 1


def moe_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().moe_workspace_init(_p(ws), _stream(stream)), "moe_workspace_init")


def moe_workspace_views(shape: MoEShape, ws: torch.Tensor) -> dict:
    """Tensor views of the routing and intermediates inside a layer workspace."""
    info = MoERouteInfo()
    _check(lib().moe_workspace_views(ctypes.byref(shape), _p(ws), ctypes.byref(info)),
           "moe_workspace_views")
    E, k = moe_topk_unpack(shape.topk_shape)
    T, H, I = shape.tokens, shape.hidden, shape.moe_inter
    act = torch.float32 if shape.dtype == MOE_F32 else torch.bfloat16
    base = ws.data_ptr()

    def view(ptr, dt, shp):
        if ptr is None:
            return None
        n = 1
        for d in shp:
            n *= d
        off = ptr - base
        return ws[off: off + n * torch.tensor([], dtype=dt).element_size()].view(dt).view(*shp)

    return dict(topk_idx=view(info.topk_idx, torch.int32, (T, k)),
                topk_w=view(info.topk_w, torch.float32, (T, k)),
                gate=view(info.gate, torch.float32, (T,)),
                counts=view(info.counts, torch.int32, (E,)),
                offsets=view(info.offsets, torch.int32, (E + 1,)),
                scatter_index=view(info.scatter_index, torch.int32, (T, k)),
                row_token=view(info.row_token, torch.int32, (T * k,)),
                x_perm=view(info.x_perm, act, (T * k, H)),
                h=view(info.h, act, (T * k, I)),
                y_perm=view(info.y_perm, act, (T * k, H)),
                shared_out=view(info.shared_out, act, (T, H)))


def moe_route(shape, x, w_router, topk_idx, topk_w, gate, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(shape), _p(x), _p(w_router), _p(topk_idx), _p(topk_w),
                           _p(gate), _p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "moe_route")


def moe_hash_route(shape, token_ids, table, vocab, topk_idx, topk_w, ws, stream=None):
    _check(lib().moe_hash_route(ctypes.byref(shape), _p(token_ids), _p(table), vocab,
                                _p(topk_idx), _p(topk_w), _p(ws), ws.numel() * ws.element_size(),
                                _stream(stream)), "moe_hash_route")


def moe_permute(shape, x, topk_idx, counts, offsets, scatter_index, row_token, x_perm, ws,
                stream=None):
    _check(lib().moe_permute(ctypes.byref(shape), _p(x), _p(topk_idx), _p(counts), _p(offsets),
                             _p(scatter_index), _p(row_token), _p(x_perm), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "moe_permute")


def moe_permute_static(shape, x, topk_idx, counts, offsets, scatter_index, row_token, x_perm,
                       stream=None):
    """moe_permute with the library's static scratch instead of a workspace."""
    _check(lib().moe_permute_static(ctypes.byref(shape), _p(x), _p(topk_idx), _p(counts),
                                    _p(offsets), _p(scatter_index), _p(row_token), _p(x_perm),
                                    _stream(stream)), "moe_permute_static")


def moe_grouped_swiglu(shape, x_perm, w_gate, w_up, expert_stride, offsets, num_groups,
                       rows_bound, inter, h, ws, stream=None, w_up_ptr=None):
    up = w_up_ptr if w_up_ptr is not None else _p(w_up)
    _check(lib().moe_grouped_swiglu(ctypes.byref(shape), _p(x_perm), _p(w_gate), up,
                                    expert_stride, _p(offsets), num_groups, rows_bound, inter,
                                    _p(h), _p(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)), "moe_grouped_swiglu")


def moe_grouped_swiglu_gather(shape, x, row_token, w_gate, w_up, expert_stride, offsets,
                              num_groups, rows_bound, inter, h, ws, stream=None, w_up_ptr=None):
    up = w_up_ptr if w_up_ptr is not None else _p(w_up)
    _check(lib().moe_grouped_swiglu_gather(ctypes.byref(shape), _p(x), _p(row_token), _p(w_gate),
                                           up, expert_stride, _p(offsets), num_groups,
                                           rows_bound, inter, _p(h), _p(ws),
                                           ws.numel() * ws.element_size(), _stream(stream)),
           "moe_grouped_swiglu_gather")


def moe_grouped_down(shape, h, w_down, expert_stride, offsets, num_groups, rows_bound, inter,
                     y_perm, ws, stream=None):
    _check(lib().moe_grouped_down(ctypes.byref(shape), _p(h), _p(w_down), expert_stride,
                                  _p(offsets), num_groups, rows_bound, inter, _p(y_perm), _p(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)),
           "moe_grouped_down")


def moe_combine(shape, y_perm, scatter_index, topk_w, shared_out, gate, y, stream=None,
                residual=None):
    _check(lib().moe_combine(ctypes.byref(shape), _p(y_perm), _p(scatter_index), _p(topk_w),
                             _p(shared_out), _p(gate), _p(residual), _p(y), _stream(stream)),
           "moe_combine")


def moe_residual_setup(shape, x, norm_weight, x_norm, stream=None):
    _check(lib().moe_residual_setup(ctypes.byref(shape), _p(x), _p(norm_weight), _p(x_norm),
                                    _stream(stream)), "moe_residual_setup")


def moe_layer_forward(shape, weights: MoEWeights, x, routes_idx, routes_w, y, ws, stream=None):
    _check(lib().moe_layer_forward(ctypes.byref(shape), ctypes.byref(weights), _p(x),
                                   _p(routes_idx), _p(routes_w), _p(y), _p(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)),
           "moe_layer_forward")


def moe_layer_forward_traced(shape, weights: MoEWeights, x, routes_idx, routes_w, y, ws,
                             stage_events, stream=None):
    """stage_events: MOE_NUM_STAGES + 1 torch.cuda.Event objects (recorded once
    beforehand so that their CUDA events exist)."""
    arr = (ctypes.c_void_p * len(stage_events))(*[e.cuda_event for e in stage_events])
    _check(lib().moe_layer_forward_traced(ctypes.byref(shape), ctypes.byref(weights), _p(x),
                                          _p(routes_idx), _p(routes_w), _p(y), _p(ws),
                                          ws.numel() * ws.element_size(), _stream(stream), arr),
           "moe_layer_forward_traced")


def moe_get_device_status(ws, stream=None):
    bits = ctypes.c_uint32(0)
    st = lib().moe_get_device_status(_p(ws), _stream(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


def moe_get_route_stats(ws, stream=None) -> int:
    """Read and clear the count of tokens whose top-k was re-decided exactly."""
    n = ctypes.c_uint32(0)
    _check(lib().moe_get_route_stats(_p(ws), _stream(stream), ctypes.byref(n)),
           "moe_get_route_stats")
    return int(n.value)


def moe_testing_router_logits(shape, x, w_router, logits, ws, stream=None):
    _check(lib().moe_testing_router_logits(ctypes.byref(shape), _p(x), _p(w_router), _p(logits),
                                           _p(ws), ws.numel() * ws.element_size(),
                                           _stream(stream)), "moe_testing_router_logits")


def moe_testing_wait_probe(ws, max_cycles: int, arrive: bool, stream=None):
    _check(lib().moe_testing_wait_probe(_p(ws), max_cycles, int(arrive), _stream(stream)),
           "moe_testing_wait_probe")


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def moe_stage_name(stage: int) -> str:
    return lib().moe_stage_name(stage).decode()


def moe_last_launch_count() -> int:
    return int(lib().moe_last_launch_count())


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def moe_testing_set_gemm_engine(engine: int) -> int:
    return int(lib().moe_testing_set_gemm_engine(engine))


def moe_testing_set_fork_sms(sms: int) -> int:
    return int(lib().moe_testing_set_fork_sms(sms))


def moe_testing_set_zero_pad(mode: int) -> int:
    return int(lib().moe_testing_set_zero_pad(mode))


def moe_testing_set_norm_wait(max_cycles: int) -> int:
    return int(lib().moe_testing_set_norm_wait(max_cycles))


# ---------------------------------------------------------------------------
# backward (moe_backward.h), name for name
# ---------------------------------------------------------------------------
def _nbytes(ws):
    return ws.numel() * ws.element_size()


def moe_backward_views(shape, ws) -> dict:
    """Tensor views of the backward's grouped buffers in a train-mode workspace."""
    info = MoEBackwardInfo()
    _check(lib().moe_backward_views(ctypes.byref(shape), _p(ws), ctypes.byref(info)),
           "moe_backward_views")
    _, k = moe_topk_unpack(shape.topk_shape)
    R, H, I = shape.tokens * k, shape.hidden, shape.moe_inter
    act = torch.float32 if shape.dtype == MOE_F32 else torch.bfloat16
    esz = 4 if shape.dtype == MOE_F32 else 2
    base = ws.data_ptr()

    def view(ptr, cols):
        off = ptr - base
        return ws[off: off + R * cols * esz].view(act).view(R, cols)

    return dict(fc1=view(info.fc1, 2 * I), grad_fc2=view(info.grad_fc2, H),
                d_fc1=view(info.d_fc1, 2 * I), dx_perm=view(info.dx_perm, H))


def moe_grouped_swiglu_save(shape, x_perm, w_gate, w_up, expert_stride, offsets, num_groups,
                            rows_bound, inter, h, fc1, ws, stream=None):
    _check(lib().moe_grouped_swiglu_save(ctypes.byref(shape), _p(x_perm), _p(w_gate), _p(w_up),
                                         expert_stride, _p(offsets), num_groups, rows_bound,
                                         inter, _p(h), _p(fc1), _p(ws), _nbytes(ws),
                                         _stream(stream)), "moe_grouped_swiglu_save")


def moe_scatter_grad(shape, dy, scatter_index, topk_w, y_perm, grad_fc2, d_topk_w, stream=None):
    _check(lib().moe_scatter_grad(ctypes.byref(shape), _p(dy), _p(scatter_index), _p(topk_w),
                                  _p(y_perm), _p(grad_fc2), _p(d_topk_w), _stream(stream)),
           "moe_scatter_grad")


def moe_grouped_down_dgrad(shape, grad_fc2, w_down, expert_stride, fc1, offsets, num_groups,
                           rows_bound, inter, d_fc1, ws, stream=None):
    _check(lib().moe_grouped_down_dgrad(ctypes.byref(shape), _p(grad_fc2), _p(w_down),
                                        expert_stride, _p(fc1), _p(offsets), num_groups,
                                        rows_bound, inter, _p(d_fc1), _p(ws), _nbytes(ws),
                                        _stream(stream)), "moe_grouped_down_dgrad")


def moe_grouped_gate_up_dgrad(shape, d_fc1, w_gate, w_up, expert_stride, offsets, num_groups,
                              rows_bound, inter, dx_perm, ws, stream=None):
    _check(lib().moe_grouped_gate_up_dgrad(ctypes.byref(shape), _p(d_fc1), _p(w_gate), _p(w_up),
                                           expert_stride, _p(offsets), num_groups, rows_bound,
                                           inter, _p(dx_perm), _p(ws), _nbytes(ws),
                                           _stream(stream)), "moe_grouped_gate_up_dgrad")


def moe_grouped_wgrad(shape, a, lda, b, ldb, offsets, num_groups, rows_bound, M, N, dw,
                      dw_stride, ws, stream=None, a_ptr=None):
    """a_ptr: a raw device address for a (a column offset into a wider matrix)."""
    ap = a_ptr if a_ptr is not None else _p(a)
    _check(lib().moe_grouped_wgrad(ctypes.byref(shape), ap, lda, _p(b), ldb, _p(offsets),
                                   num_groups, rows_bound, M, N, _p(dw), dw_stride, _p(ws),
                                   _nbytes(ws), _stream(stream)), "moe_grouped_wgrad")


def moe_gather_grad(shape, dx_perm, scatter_index, residual_grad, dx, stream=None):
    _check(lib().moe_gather_grad(ctypes.byref(shape), _p(dx_perm), _p(scatter_index),
                                 _p(residual_grad), _p(dx), _stream(stream)), "moe_gather_grad")


def moe_layer_backward(shape, weights: MoEWeights, dy, dx, d_topk_w, grads: MoEExpertGrads, ws,
                       stream=None):
    _check(lib().moe_layer_backward(ctypes.byref(shape), ctypes.byref(weights), _p(dy), _p(dx),
                                    _p(d_topk_w), ctypes.byref(grads), _p(ws), _nbytes(ws),
                                    _stream(stream)), "moe_layer_backward")


def grads_for(dw_gate, dw_up, dw_down) -> MoEExpertGrads:
    """MoEExpertGrads over [E, I, H], [E, I, H], [E, H, I] tensors."""
    g = MoEExpertGrads()
    g.gate, g.up, g.down = _p(dw_gate), _p(dw_up), _p(dw_down)
    g.gate_up_stride = dw_gate.shape[1] * dw_gate.shape[2]
    g.down_stride = dw_down.shape[1] * dw_down.shape[2]
    return g


# ---------------------------------------------------------------------------
# training operators (moe_train.h), name for name
# ---------------------------------------------------------------------------
MOE_CE_NONE, MOE_CE_SUM, MOE_CE_MEAN = 0, 1, 2


def _rows(t: torch.Tensor, rows: int, cols: int, dtype, name: str):
    """Address and row stride of a [rows, cols] matrix whose rows are contiguous and
    apart (a broadcast row's stride 0 would mean "dense" to the library)."""
    if tuple(t.shape) != (rows, cols) or t.dtype != dtype:
        raise ValueError("%s must be [%d, %d] %s, got %s %s" % (name, rows, cols, dtype,
                                                                tuple(t.shape), t.dtype))
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    if rows > 1 and t.stride(0) < cols:
        raise ValueError("the rows of %s share memory (row stride %d for %d columns): pass a copy, "
                         "for example %s.contiguous()" % (name, t.stride(0), cols, name))
    return t.data_ptr(), (t.stride(0) if rows > 1 else cols)


def _vec(t: torch.Tensor, n: int, dtype, name: str):
    if t.numel() != n or t.dtype != dtype:
        raise ValueError("%s must hold %d elements of %s, got %s %s" % (name, n, dtype,
                                                                        tuple(t.shape), t.dtype))
    return _p(t)


def _on_device(ws: torch.Tensor, **tensors):
    """The workspace is device memory, and the tensors lie where it does: an address
    of another memory must not reach a kernel."""
    if ws is None or not ws.is_cuda:
        raise ValueError("the workspace must be a CUDA tensor, got %s" % (ws if ws is None else ws.device))
    at = ws.get_device()
    for name, t in tensors.items():
        if t is not None and t.get_device() != at:
            raise ValueError("%s is on %s, the workspace on %s" % (name, t.device, ws.device))


def moe_linear_ce_workspace_bytes(shape: MoECeShape) -> int:
    return int(lib().moe_linear_ce_workspace_bytes(ctypes.byref(shape)))


def moe_linear_ce_forward(shape: MoECeShape, x, w, target, loss, lse, stats, total, ws,
                          stream=None):
    """x and w may be rows of wider buffers (the strides go into the shape)."""
    dt = torch.float32 if shape.dtype == MOE_F32 else torch.bfloat16
    xp, shape.x_stride = _rows(x, shape.tokens, shape.hidden, dt, "x")
    wp, shape.w_stride = _rows(w, shape.vocab, shape.hidden, dt, "w")
    f32, T = torch.float32, shape.tokens
    args = (_vec(target, T, torch.int32, "target"),
            None if loss is None else _vec(loss, T, f32, "loss"),
            None if lse is None else _vec(lse, T, f32, "lse"),
            None if stats is None else _vec(stats, 4 * T, f32, "stats"),
            None if total is None else _vec(total, 1, f32, "total"))
    _on_device(ws, x=x, w=w, target=target, loss=loss, lse=lse, stats=stats, total=total)
    _check(lib().moe_linear_ce_forward(ctypes.byref(shape), xp, wp, *args, _p(ws), _nbytes(ws),
                                       _stream(stream)), "moe_linear_ce_forward")


def moe_linear_ce_backward(shape: MoECeShape, x, w, target, stats, dloss, dx, dw, ws,
                           stream=None):
    dt = torch.float32 if shape.dtype == MOE_F32 else torch.bfloat16
    T, H, V = shape.tokens, shape.hidden, shape.vocab
    xp, shape.x_stride = _rows(x, T, H, dt, "x")
    wp, shape.w_stride = _rows(w, V, H, dt, "w")
    n = T if shape.reduction == MOE_CE_NONE else 1
    args = (_vec(target, T, torch.int32, "target"), _vec(stats, 4 * T, torch.float32, "stats"),
            None if dloss is None else _vec(dloss, n, torch.float32, "dloss"),
            None if dx is None else _vec(dx, T * H, dt, "dx"),
            None if dw is None else _vec(dw, V * H, dt, "dw"))
    _on_device(ws, x=x, w=w, target=target, stats=stats, dloss=dloss, dx=dx, dw=dw)
    _check(lib().moe_linear_ce_backward(ctypes.byref(shape), xp, wp, *args, _p(ws), _nbytes(ws),
                                        _stream(stream)), "moe_linear_ce_backward")


def moe_router_backward_workspace_bytes(shape: MoEShape) -> int:
    return int(lib().moe_router_backward_workspace_bytes(ctypes.byref(shape)))


def moe_router_backward(shape: MoEShape, x, w_router, topk_idx, d_topk_w, d_gate, balance_coef,
                        z_coef, dx_add, dx, dw_router, aux, ws, stream=None):
    E, k = shape.topk_shape >> 8, shape.topk_shape & 255   # moe_topk_unpack's fields
    T, H, f32 = shape.tokens, shape.hidden, torch.float32
    dt = f32 if shape.dtype == MOE_F32 else torch.bfloat16
    rows = E + shape.shared_gate

    def opt(t, n, d, name):
        return None if t is None else _vec(t, n, d, name)

    args = (_vec(x, T * H, dt, "x"), _vec(w_router, rows * H, dt, "w_router"),
            _vec(topk_idx, T * k, torch.int32, "topk_idx"), opt(d_topk_w, T * k, f32, "d_topk_w"),
            opt(d_gate, T, f32, "d_gate"), balance_coef, z_coef, opt(dx_add, T * H, dt, "dx_add"),
            _vec(dx, T * H, dt, "dx"), _vec(dw_router, rows * H, dt, "dw_router"),
            opt(aux, 2, f32, "aux"))
    _on_device(ws, x=x, w_router=w_router, topk_idx=topk_idx, d_topk_w=d_topk_w, d_gate=d_gate,
               dx_add=dx_add, dx=dx, dw_router=dw_router, aux=aux)
    _check(lib().moe_router_backward(ctypes.byref(shape), *args, _p(ws), _nbytes(ws),
                                     _stream(stream)), "moe_router_backward")


def grad_tensors(srcs, dsts):
    """MoEGradTensor array over gradients and destinations (an entry of dsts is
    None where only the norm counts)."""
    arr = (MoEGradTensor * len(srcs))()
    for e, s, d in zip(arr, srcs, dsts):
        if d is not None and d.numel() != s.numel():
            raise ValueError("a destination must hold as many elements as its gradient")
        if not s.is_cuda or (d is not None and d.device != s.device) or s.device != srcs[0].device:
            raise ValueError("gradients and destinations must be on one CUDA device")
        e.src, e.numel, e.src_dtype = _p(s), s.numel(), _dtype_code(s.dtype)
        e.dst, e.dst_dtype = _p(d), _dtype_code((s if d is None else d).dtype)
    return arr


def moe_grad_clip_workspace_bytes(tensors) -> int:
    return int(lib().moe_grad_clip_workspace_bytes(tensors, len(tensors)))


def moe_grad_clip_plan(tensors, ws, stream=None) -> MoEGradPlan:
    plan = MoEGradPlan()
    _on_device(ws)
    _check(lib().moe_grad_clip_plan(tensors, len(tensors), ctypes.byref(plan), _p(ws), _nbytes(ws),
                                    _stream(stream)), "moe_grad_clip_plan")
    return plan


def moe_grad_clip(plan: MoEGradPlan, max_norm: float, norm, ws, stream=None):
    at = _vec(norm, 1, torch.float32, "norm")
    _on_device(ws, norm=norm)
    _check(lib().moe_grad_clip(ctypes.byref(plan), max_norm, at, _p(ws), _nbytes(ws),
                               _stream(stream)), "moe_grad_clip")


# ---------------------------------------------------------------------------
# embedding, block norms, orthogonalised update (moe_model.h), name for name
# ---------------------------------------------------------------------------
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN = 0, 1, 2
MOE_MUON_SCALE_NONE, MOE_MUON_SCALE_SPECTRAL, MOE_MUON_SCALE_RMS = 0, 1, 2


def _device(t: torch.Tensor) -> int:
    """The device of a call's workspace (or first tensor): a CUDA device, and the
    current one, to whose stream the launch goes."""
    if t is None or not t.is_cuda:
        raise ValueError("the workspace and the tensors must be CUDA tensors, got %s"
                         % (t if t is None else t.device))
    at = t.get_device()
    if at != torch.cuda.current_device():
        raise ValueError("the tensors are on %s, the current device is cuda:%d"
                         % (t.device, torch.cuda.current_device()))
    return at


def _arg(t, n: int, dtype, at: int, name: str, none: bool = True):
    """Address of n contiguous elements on device `at` (all checks of an argument in one
    place: a small call is as long as its host side)."""
    if t is None:
        if none:
            return None
        raise ValueError("%s must be a tensor" % name)
    if t.dtype != dtype or t.numel() != n:
        raise ValueError("%s must hold %d elements of %s, got %s %s" % (name, n, dtype, tuple(t.shape),
                                                                        t.dtype))
    if t.get_device() != at:
        raise ValueError("%s is on %s, the workspace on cuda:%d" % (name, t.device, at))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


_ACT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def moe_embed_workspace_bytes(shape: MoEEmbedShape) -> int:
    return int(lib().moe_embed_workspace_bytes(ctypes.byref(shape)))


def moe_embed_forward(shape: MoEEmbedShape, w, ids, y, ws, stream=None):
    """w may be rows of a wider buffer (its stride goes into a copy of the shape)."""
    at, dt, T, H = _device(ws), _ACT[shape.dtype], shape.tokens, shape.hidden
    wp, ld = _rows(w, shape.vocab, H, dt, "w")
    if (shape.w_stride or H) != ld:
        shape = MoEEmbedShape.from_buffer_copy(shape)
        shape.w_stride = ld
    if w.get_device() != at:
        raise ValueError("w is on %s, the workspace on cuda:%d" % (w.device, at))
    st = lib().moe_embed_forward(ctypes.byref(shape), wp, _arg(ids, T, torch.int32, at, "ids", False),
                                 _arg(y, T * H, dt, at, "y", False), ws.data_ptr(), _nbytes(ws), _stream(stream))
    if st:
        _check(st, "moe_embed_forward")


def moe_embed_backward(shape: MoEEmbedShape, ids, dy, dw_add, dw, ws, stream=None):
    at, dt, T = _device(ws), _ACT[shape.dtype], shape.tokens
    n, all_ = T * shape.hidden, shape.vocab * shape.hidden
    st = lib().moe_embed_backward(ctypes.byref(shape), _arg(ids, T, torch.int32, at, "ids", False),
                                  _arg(dy, n, dt, at, "dy", False), _arg(dw_add, all_, dt, at, "dw_add"),
                                  _arg(dw, all_, dt, at, "dw", False), ws.data_ptr(), _nbytes(ws), _stream(stream))
    if st:
        _check(st, "moe_embed_backward")


def moe_block_norm_workspace_bytes(shape: MoEBlockNormShape) -> int:
    return int(lib().moe_block_norm_workspace_bytes(ctypes.byref(shape)))


def moe_block_norm_forward(shape: MoEBlockNormShape, x, y, w_post, gate, w_pre, s, h, rstd,
                           stream=None):
    at, dt, T, H = _device(x), _ACT[shape.dtype], shape.tokens, shape.hidden
    n, token = T * H, shape.gate == MOE_GATE_TOKEN
    st = lib().moe_block_norm_forward(
        ctypes.byref(shape), _arg(x, n, dt, at, "x", False), _arg(y, n, dt, at, "y"),
        _arg(w_post, H, dt, at, "w_post"),
        _arg(gate, T if token else H, torch.float32 if token else dt, at, "gate"),
        _arg(w_pre, H, dt, at, "w_pre"), _arg(s, n, dt, at, "s"), _arg(h, n, dt, at, "h"),
        _arg(rstd, 2 * T, torch.float32, at, "rstd"), _stream(stream))
    if st:
        _check(st, "moe_block_norm_forward")


def moe_block_norm_backward(shape: MoEBlockNormShape, ds, dh, x, y, w_post, gate, w_pre, rstd, dx,
                            dy, dw_post, dgate, dw_pre, ws, stream=None):
    at, dt, T, H = _device(ws), _ACT[shape.dtype], shape.tokens, shape.hidden
    n, token = T * H, shape.gate == MOE_GATE_TOKEN
    gn, gd = (T, torch.float32) if token else (H, dt)
    st = lib().moe_block_norm_backward(
        ctypes.byref(shape), _arg(ds, n, dt, at, "ds"), _arg(dh, n, dt, at, "dh"),
        _arg(x, n, dt, at, "x", False), _arg(y, n, dt, at, "y"), _arg(w_post, H, dt, at, "w_post"),
        _arg(gate, gn, gd, at, "gate"), _arg(w_pre, H, dt, at, "w_pre"),
        _arg(rstd, 2 * T, torch.float32, at, "rstd", False), _arg(dx, n, dt, at, "dx"),
        _arg(dy, n, dt, at, "dy"), _arg(dw_post, H, dt, at, "dw_post"), _arg(dgate, gn, gd, at, "dgate"),
        _arg(dw_pre, H, dt, at, "dw_pre"), ws.data_ptr(), _nbytes(ws), _stream(stream))
    if st:
        _check(st, "moe_block_norm_backward")


def orth_coefs(coefficients=(3.4445, -4.7750, 2.0315), steps: int = 5, eps: float = 1e-7) -> MoEOrthCoefs:
    """MoEOrthCoefs of one (a, b, c) for every step, or of a sequence of them, one a
    step (steps is then its length)."""
    each = list(coefficients)
    if each and not hasattr(each[0], "__len__"):
        each = [each] * steps
    if not 1 <= len(each) <= MOE_ORTH_MAX_STEPS or any(len(t) != 3 for t in each):
        raise ValueError("coefficients must be (a, b, c) with 1 to %d steps, or as many triples"
                         % MOE_ORTH_MAX_STEPS)
    c = MoEOrthCoefs()
    c.steps, c.eps = len(each), eps
    for i, t in enumerate(each):
        for j in range(3):
            c.coef[i][j] = t[j]
    return c


def moe_orthogonalize_workspace_bytes(shape: MoEOrthShape, coefs: MoEOrthCoefs) -> int:
    return int(lib().moe_orthogonalize_workspace_bytes(ctypes.byref(shape), ctypes.byref(coefs)))


def moe_orthogonalize(shape: MoEOrthShape, coefs: MoEOrthCoefs, x, out, ws, stream=None):
    at, dt, n = _device(ws), _ACT[shape.dtype], shape.batch * shape.rows * shape.cols
    st = lib().moe_orthogonalize(ctypes.byref(shape), ctypes.byref(coefs), _arg(x, n, dt, at, "x", False),
                                 _arg(out, n, dt, at, "out", False), ws.data_ptr(), _nbytes(ws),
                                 _stream(stream))
    if st:
        _check(st, "moe_orthogonalize")


def muon_tensors(params, grads, momenta):
    """MoEMuonTensor array over parameters [..., rows, cols] (the leading dimensions
    are a batch of matrices), their gradients and fp32 momenta."""
    params, grads, momenta = list(params), list(grads), list(momenta)
    if not len(params) == len(grads) == len(momenta):
        raise ValueError("every parameter needs one gradient and one momentum")
    arr = (MoEMuonTensor * len(params))()
    for e, w, g, v in zip(arr, params, grads, momenta):
        if w.dim() < 2 or g.shape != w.shape or v.shape != w.shape or v.dtype != torch.float32:
            raise ValueError("a parameter must be a matrix or a batch of them, its gradient and fp32 "
                             "momentum of the same shape, got %s, %s and %s %s"
                             % (tuple(w.shape), tuple(g.shape), tuple(v.shape), v.dtype))
        for t in (w, g, v):
            if not t.is_cuda or t.device != params[0].device:
                raise ValueError("parameters, gradients and momenta must be on one CUDA device")
        e.param, e.grad, e.momentum = _p(w), _p(g), _p(v)
        e.rows, e.cols = w.shape[-2], w.shape[-1]
        e.batch = w.numel() // max(1, w.shape[-2] * w.shape[-1])
        e.param_dtype, e.grad_dtype = _dtype_code(w.dtype), _dtype_code(g.dtype)
    # what a step writes is written once, and read as nothing else
    span = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
    written = sorted(span(t) for t in params + momenta if t.numel())
    ends = [hi for _, hi in written]
    if any(hi > lo for hi, (lo, _) in zip(ends, written[1:])):
        raise ValueError("no two parameters and momenta may overlap")
    for lo, hi in (span(g) for g in grads if g.numel()):
        i = bisect.bisect_right(ends, lo)   # the first that ends behind the gradient's start
        if i < len(written) and written[i][0] < hi:
            raise ValueError("a gradient must not overlap a parameter or a momentum")
    return arr


def moe_muon_workspace_bytes(tensors, config: MoEMuonConfig) -> int:
    return int(lib().moe_muon_workspace_bytes(tensors, len(tensors), ctypes.byref(config)))


def moe_muon_step(tensors, config: MoEMuonConfig, ws, stream=None):
    _device(ws)
    _check(lib().moe_muon_step(tensors, len(tensors), ctypes.byref(config), _p(ws), _nbytes(ws),
                               _stream(stream)), "moe_muon_step")


# ---------------------------------------------------------------------------
# conveniences over the ABI (allocation through torch, nothing else)
# ---------------------------------------------------------------------------
def shape_for(wl, T: Optional[int] = None) -> MoEShape:
    s = MoEShape()
    s.tokens = wl.T if T is None else T
    s.hidden, s.moe_inter, s.shared_inter = wl.H, wl.I, wl.I_sh
    s.topk_shape = moe_topk_pack(wl.E, wl.k)
    s.shared_gate = int(wl.shared_gate)
    s.norm_topk = int(wl.norm_topk)
    s.dtype = MOE_F32 if wl.dtype == "f32" else MOE_BF16
    s.input_norm = int(getattr(wl, "input_norm", False))
    s.residual = int(getattr(wl, "residual", False))
    s.norm_eps = float(getattr(wl, "norm_eps", 1e-6))
    s.train = int(getattr(wl, "train", False))
    s.weight_format = MOE_WEIGHTS_MXFP8 if getattr(wl, "weights", "act") == "mxfp8" else MOE_WEIGHTS_ACT
    return s


def alloc_workspace(shape: MoEShape, device="cuda", full: bool = True, stream=None):
    n = moe_workspace_bytes(shape) if full else moe_scratch_bytes(shape)
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "alloc_workspace", "invalid shape")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    moe_workspace_init(ws, stream)
    return ws


def weights_from(inputs: dict) -> MoEWeights:
    """MoEWeights over the tensors of a workloads.make_inputs() dict (split fc1)."""
    w = MoEWeights()
    g, d = inputs["w_gate"], inputs["w_down"]
    w.router = _p(inputs.get("w_router"))
    w.gate, w.up = _p(g), _p(inputs["w_up"])
    w.down = _p(d)
    if g.dtype == torch.uint8:   # packed MXFP8 [E, N*K*9/8]: strides in bytes
        w.gate_up_stride, w.down_stride = g.shape[1], d.shape[1]
    else:
        w.gate_up_stride = g.shape[1] * g.shape[2]
        w.down_stride = d.shape[1] * d.shape[2]
    w.shared_gate_proj = _p(inputs.get("sh_gate"))
    w.shared_up = _p(inputs.get("sh_up"))
    w.shared_down = _p(inputs.get("sh_down"))
    w.norm_weight = _p(inputs.get("norm_weight"))
    return w


class MoELayer:
    """One layer: shape, weight table and a workspace, over caller tensors."""

    def __init__(self, wl, inputs: dict, T: Optional[int] = None, device="cuda",
                 train: bool = False):
        self.wl = wl
        self.inputs = inputs
        self.shape = shape_for(wl, T if T is not None else inputs["x"].shape[0])
        self.shape.train = int(train)
        self.weights = weights_from(inputs)
        self.ws = alloc_workspace(self.shape, device)

    def forward(self, x, y=None, routes_idx=None, routes_w=None, stream=None):
        if y is None:
            y = torch.empty_like(x)
        moe_layer_forward(self.shape, self.weights, x, routes_idx, routes_w, y, self.ws, stream)
        return y

    def backward(self, dy, dx, d_topk_w, grads: MoEExpertGrads, stream=None):
        """Gradients after a train-mode forward on this layer's workspace."""
        moe_layer_backward(self.shape, self.weights, dy, dx, d_topk_w, grads, self.ws, stream)

    def views(self):
        return moe_workspace_views(self.shape, self.ws)

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


def _empty(stream, shape, dtype, device):
    """Memory of the stream that writes it: a block that another stream has freed may
    still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(stream, t):
    """_empty of t's shape and type (a tensor's own method on the current stream: a
    microsecond less)."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(stream, t.shape, t.dtype, t.device)


def _alloc_ws(n: int, device, stream, where: str):
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, where, "invalid shape")
    ws = _empty(stream, n + 256, torch.uint8, device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    moe_workspace_init(ws, stream)
    return ws


class LinearCrossEntropy:
    """Softmax cross entropy of x . w^T against target over a vocabulary, and its
    gradients, without the [tokens, vocab] logits: shape and a workspace over
    caller tensors.  x [tokens, hidden] and w [vocab, hidden] in bf16 or fp32 may
    be rows of wider buffers; target is int32 [tokens].  reduction: "none", "sum" or
    "mean" (over the tokens whose target is not ignore_index).  The workspace is made on
    the current stream, which another one has to wait for before its first call; outputs
    that a call makes belong to the stream it is given."""

    def __init__(self, tokens: int, hidden: int, vocab: int, dtype=torch.bfloat16,
                 reduction: str = "mean", ignore_index: int = -100, device="cuda"):
        s = MoECeShape()
        s.tokens, s.hidden, s.vocab, s.dtype = tokens, hidden, vocab, _dtype_code(dtype)
        s.reduction = {"none": MOE_CE_NONE, "sum": MOE_CE_SUM, "mean": MOE_CE_MEAN}[reduction]
        s.ignore_index = ignore_index
        self.shape, self.dtype = s, dtype
        self.ws = _alloc_ws(moe_linear_ce_workspace_bytes(s), device, None, "LinearCrossEntropy")
        self.lse = torch.zeros(tokens, dtype=torch.float32, device=device)
        self.stats = torch.zeros((tokens, 4), dtype=torch.float32, device=device)

    def forward(self, x, w, target, loss=None, total=None, stream=None):
        """The losses [tokens] ("none") or the reduced loss [1]; self.stats is
        what the backward needs."""
        none = self.shape.reduction == MOE_CE_NONE
        if none and loss is None:
            loss = _empty(stream, self.shape.tokens, torch.float32, x.device)
        if not none and total is None:
            total = _empty(stream, 1, torch.float32, x.device)
        moe_linear_ce_forward(self.shape, x, w, target, loss, self.lse, self.stats, total,
                              self.ws, stream)
        return loss if none else total

    def backward(self, x, w, target, dloss=None, dx=None, dw=None, stream=None):
        """(dx, dw) after a forward with the same x, w and target."""
        if dx is None:
            dx = _empty(stream, x.shape, x.dtype, x.device)
        if dw is None:
            dw = _empty(stream, w.shape, w.dtype, w.device)
        moe_linear_ce_backward(self.shape, x, w, target, self.stats, dloss, dx, dw, self.ws, stream)
        return dx, dw

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


class RouterGrad:
    """Gradient of the top-k softmax router (with the balance and z losses):
    shape, coefficients and a workspace over caller tensors.  Streams as in
    LinearCrossEntropy."""

    def __init__(self, tokens: int, hidden: int, experts: int, top_k: int, norm_topk: bool = True,
                 shared_gate: bool = False, dtype=torch.bfloat16, balance_coef: float = 0.0,
                 z_coef: float = 0.0, device="cuda"):
        s = MoEShape()
        s.tokens, s.hidden, s.moe_inter = tokens, hidden, 8   # moe_inter does not count here
        s.shared_inter = 8 if shared_gate else 0
        s.topk_shape = moe_topk_pack(experts, top_k)
        s.shared_gate, s.norm_topk = int(shared_gate), int(norm_topk)
        s.dtype, s.norm_eps = _dtype_code(dtype), 1e-6
        self.shape, self.balance_coef, self.z_coef = s, balance_coef, z_coef
        self.ws = _alloc_ws(moe_router_backward_workspace_bytes(s), device, None, "RouterGrad")

    def backward(self, x, w_router, topk_idx, d_topk_w, d_gate=None, dx_add=None, dx=None,
                 dw_router=None, aux=None, stream=None):
        """(dx, dw_router, aux); dx includes dx_add (the experts' dx), aux [2]
        holds the balance and z losses."""
        dx = _empty(stream, x.shape, x.dtype, x.device) if dx is None else dx
        if dw_router is None:
            dw_router = _empty(stream, w_router.shape, w_router.dtype, w_router.device)
        if aux is None:
            aux = _empty(stream, 2, torch.float32, x.device)
        moe_router_backward(self.shape, x, w_router, topk_idx, d_topk_w, d_gate, self.balance_coef,
                            self.z_coef, dx_add, dx, dw_router, aux, self.ws, stream)
        return dx, dw_router, aux

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


class GradClip:
    """Global norm of a list of gradients, and clipping: in place, or into out
    (one destination a gradient, fp32 or bf16).  The list's table is made once,
    here; the tensors must stay where they are."""

    def __init__(self, grads, out=None, stream=None):
        self.grads = list(grads)   # once: it may be a generator
        self.out = list(self.grads if out is None else out)
        if len(self.grads) != len(self.out):
            raise ValueError("out must have one destination for every gradient")
        if not self.grads:
            raise ValueError("the list of gradients is empty")
        device = self.grads[0].device
        table = grad_tensors(self.grads, self.out)
        self.ws = _alloc_ws(moe_grad_clip_workspace_bytes(table), device, stream, "GradClip")
        self.plan = moe_grad_clip_plan(table, self.ws, stream)

    def clip(self, max_norm: float, norm=None, stream=None):
        """The norm [1] before clipping."""
        if norm is None:
            norm = _empty(stream, 1, torch.float32, self.ws.device)
        moe_grad_clip(self.plan, max_norm, norm, self.ws, stream)
        return norm

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


class TokenEmbedding:
    """Rows of a table looked up by token id, times a scale, and the table's
    gradient: shape and a workspace over caller tensors.  w [vocab, hidden] may be rows
    of a wider buffer; ids is int32 [tokens].  Tokens of padding_idx get no gradient, an id
    out of range a zero row and a bit of the device status.  Streams as in
    LinearCrossEntropy."""

    def __init__(self, tokens: int, hidden: int, vocab: int, dtype=torch.bfloat16, scale: float = 1.0,
                 padding_idx: Optional[int] = None, device="cuda"):
        s = MoEEmbedShape()
        s.tokens, s.hidden, s.vocab, s.dtype = tokens, hidden, vocab, _dtype_code(dtype)
        s.padding_idx, s.scale = -1 if padding_idx is None else padding_idx, scale
        self.shape, self.dtype = s, dtype
        self.ws = _alloc_ws(moe_embed_workspace_bytes(s), device, None, "TokenEmbedding")

    def forward(self, w, ids, y=None, stream=None):
        """y [tokens, hidden]."""
        if y is None:
            y = _empty(stream, (self.shape.tokens, self.shape.hidden), self.dtype, w.device)
        moe_embed_forward(self.shape, w, ids, y, self.ws, stream)
        return y

    def backward(self, ids, dy, dw_add=None, dw=None, stream=None):
        """dw [vocab, hidden], plus dw_add where given (the gradient of a classifier
        that shares the table); dw_add may be dw: only rows with tokens are touched."""
        if dw is None:
            dw = _empty(stream, (self.shape.vocab, self.shape.hidden), self.dtype, dy.device)
        moe_embed_backward(self.shape, ids, dy, dw_add, dw, self.ws, stream)
        return dw

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


class BlockGrads(NamedTuple):
    """What BlockNorm.backward computes; None where the input is."""
    dx: torch.Tensor
    dy: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]


class BlockNorm:
    """The norms before and after a block with its gate and the residual, in one pass:

        s = residual_scale * x + gate * RMSNorm(y; w_post),  h = RMSNorm(s; w_pre)

    gate: None, "channel" ([hidden] in dtype) or "token" ([tokens] fp32); unit_offset:
    the weights count from 1.  Without y (the norm before the first block) s is
    residual_scale * x, without w_pre there is no h, without w_post y is taken as it is.
    self.rstd holds the norms of the last forward, which the backward needs: an object
    serves one place of a model, or several whose callers keep an rstd ([tokens, 2] fp32) for
    each and give it to both calls.  The status is the backward's; a forward whose rows never came
    shows it by NaN.  Streams as in LinearCrossEntropy."""

    def __init__(self, tokens: int, hidden: int, dtype=torch.bfloat16, gate: Optional[str] = None,
                 residual_scale: float = 1.0, eps: float = 1e-6, unit_offset: bool = False,
                 device="cuda"):
        s = MoEBlockNormShape()
        s.tokens, s.hidden, s.dtype = tokens, hidden, _dtype_code(dtype)
        s.gate = {None: MOE_GATE_NONE, "none": MOE_GATE_NONE, "channel": MOE_GATE_CHANNEL,
                  "token": MOE_GATE_TOKEN}[gate]
        s.residual_scale, s.eps, s.unit_offset = residual_scale, eps, int(unit_offset)
        self.shape, self.dtype = s, dtype
        self.ws = _alloc_ws(moe_block_norm_workspace_bytes(s), device, None, "BlockNorm")
        self.rstd = torch.zeros((tokens, 2), dtype=torch.float32, device=device)

    def forward(self, x, y=None, w_post=None, gate=None, w_pre=None, s=None, h=None, stream=None, rstd=None):
        """(s, h); rstd (self.rstd unless given) is what the backward needs."""
        if s is None:
            s = _like(stream, x)
        if h is None and w_pre is not None:
            h = _like(stream, x)
        moe_block_norm_forward(self.shape, x, y, w_post, gate, w_pre, s, h,
                               self.rstd if rstd is None else rstd, stream)
        return s, h

    def backward(self, ds, dh, x, y=None, w_post=None, gate=None, w_pre=None, dx=None, dy=None,
                 dw_post=None, dgate=None, dw_pre=None, stream=None, rstd=None) -> BlockGrads:
        """Gradients after a forward with the same inputs (the last one, or the one that was
        given this rstd), given ds (of s, or None for zeros) and dh (of h)."""
        def like(out, t):
            return _like(stream, t) if out is None and t is not None else out

        d = BlockGrads(like(dx, x), like(dy, y), like(dw_post, w_post), like(dgate, gate),
                       like(dw_pre, w_pre))
        moe_block_norm_backward(self.shape, ds, dh, x, y, w_post, gate, w_pre,
                                self.rstd if rstd is None else rstd, *d, self.ws, stream)
        return d

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


class Orthogonalize:
    """A batch of matrices with their singular values taken towards 1 by `steps`
    Newton-Schulz products: shape, coefficients and a workspace over caller tensors.
    coefficients: (a, b, c), or one triple a step.  Streams as in LinearCrossEntropy."""

    def __init__(self, batch: int, rows: int, cols: int, dtype=torch.bfloat16,
                 coefficients=(3.4445, -4.7750, 2.0315), steps: int = 5, eps: float = 1e-7,
                 device="cuda"):
        s = MoEOrthShape()
        s.batch, s.rows, s.cols, s.dtype = batch, rows, cols, _dtype_code(dtype)
        self.shape, self.coefs = s, orth_coefs(coefficients, steps, eps)
        self.ws = _alloc_ws(moe_orthogonalize_workspace_bytes(s, self.coefs), device, None, "Orthogonalize")

    def forward(self, x, out=None, stream=None):
        """out [batch, rows, cols]; may be x."""
        if out is None:
            out = _like(stream, x)
        moe_orthogonalize(self.shape, self.coefs, x, out, self.ws, stream)
        return out

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)


class Muon:
    """Momentum and orthogonalised update of a list of weight matrices (each [..., rows,
    cols], the leading dimensions a batch of matrices), in place.  scale: "none",
    "spectral" (sqrt(max(1, rows / cols))) or "rms" (0.2 sqrt(max(rows, cols))).  The
    tensors must stay where they are; momenta (fp32) are made here unless given.
    Streams as in LinearCrossEntropy."""

    def __init__(self, params, grads, momenta=None, lr: float = 0.02, momentum: float = 0.95,
                 nesterov: bool = True, weight_decay: float = 0.0, scale: str = "spectral",
                 coefficients=(3.4445, -4.7750, 2.0315), steps: int = 5, eps: float = 1e-7):
        self.params, self.grads = list(params), list(grads)
        if not self.params:
            raise ValueError("the list of parameters is empty")
        if momenta is None:
            momenta = [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
        self.momenta = list(momenta)
        self.tensors = muon_tensors(self.params, self.grads, self.momenta)
        c = MoEMuonConfig()
        c.lr, c.momentum, c.weight_decay, c.nesterov = lr, momentum, weight_decay, int(nesterov)
        c.scale = {"none": MOE_MUON_SCALE_NONE, "spectral": MOE_MUON_SCALE_SPECTRAL,
                   "rms": MOE_MUON_SCALE_RMS}[scale]
        c.coefs = orth_coefs(coefficients, steps, eps)
        self.config = c
        self.ws = _alloc_ws(moe_muon_workspace_bytes(self.tensors, c), self.params[0].device, None, "Muon")

    def step(self, lr: Optional[float] = None, stream=None):
        """One update; lr stays what it was last set to (a captured step keeps the lr that it
        was captured with)."""
        if lr is not None:
            self.config.lr = lr
        moe_muon_step(self.tensors, self.config, self.ws, stream)

    def device_status(self, stream=None):
        return moe_get_device_status(self.ws, stream)

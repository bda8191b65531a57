"""Python binding of libw4a16moe, the GB300 (sm_103a) W4A16 routed-expert MoE layer.

Argument marshalling only: each function here takes torch CUDA tensors (device
memory and streams come from PyTorch), derives the layer dims from their
shapes, and calls the C entry point of the same name in ``libw4a16moe.so``.
Every step of the layer runs in the library's CUDA kernels; there is no
fallback, and importing this module fails loudly if the library is missing.

Weights follow the storage of the model card "Minachist/Qwen3.8-Flash-Next-
INT4-Mixed-AutoRound" ("What is quantized", group A): int32 words holding
eight int4 values q + 8, lowest nibble first, with one bf16 scale per row and
128-wide K group. Shapes (E experts, hidden H, intermediate I):
w1_packed [E, 2I, H/8] int32 (gate rows then up rows), w1_scales [E, 2I, H/128]
bf16, w2_packed [E, H, I/8] int32, w2_scales [E, H, I/128] bf16.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "MoeError", "moe_dims", "lib", "build", "moe_status_str", "moe_version", "moe_workspace_size",
    "workspace", "moe_route", "moe_route_shared", "shared_workspace", "moe_w4a16_forward", "moe_w4a16_forward_rms", "moe_permute",
    "moe_pack_int4", "moe_quantize_int4", "moe_w8a16_linear", "moe_w8a16_workspace_size", "moe_check_device_error", "moe_profile_events", "moe_w4a16_forward_noalloc",
    "moe_noalloc_check_device_error", "moe_forward_plan", "STATUS", "Kv4Cache", "kv4_cache", "kv4_workspace",
    "moe_kv4_workspace_size", "moe_qk_norm_rope", "moe_kv4_append", "moe_kv4_read", "moe_kv4_attention",
    "moe_w4a16_linear", "moe_w4a16_workspace_size", "moe_verify_drafts", "moe_verify_workspace_size", "verify_workspace",
    "moe_kv4_attention_window",
]

_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_DIR, "libw4a16moe.so")

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE", 6: "MOE_ERR_TIMEOUT"}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), moe_status_str(status)))


class moe_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32)]

    def __repr__(self):
        return "moe_dims(T=%d, H=%d, E=%d, k=%d, I=%d)" % (self.T, self.H, self.E, self.k, self.I)


class moe_strides(ctypes.Structure):
    _fields_ = [("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class moe_kv4_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("D", ctypes.c_int32)]


_lib = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libw4a16moe.so in-tree for sm_103a (nvcc)."""
    from . import _build
    return _build.build(force=force, verbose=verbose)


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libw4a16moe.so is not built (%s); run w4a16_mixture_experts_gb300.build()"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        D = moe_dims
        L.moe_status_str.argtypes, L.moe_status_str.restype = [I], ctypes.c_char_p
        L.moe_version.argtypes, L.moe_version.restype = [], I
        L.moe_workspace_size.argtypes, L.moe_workspace_size.restype = [D, ctypes.POINTER(Z)], I
        L.moe_route.argtypes, L.moe_route.restype = [P, P, P, D, P, P, P, Z, P], I
        L.moe_route_shared.argtypes, L.moe_route_shared.restype = [P, P, P, D, P, P, P, Z, P], I
        L.moe_w4a16_forward.argtypes = [P, P, P, P, P, P, P, P, D, P, Z, P]
        L.moe_w4a16_forward.restype = I
        L.moe_w4a16_forward_rms.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_float, D, P, Z, P]
        L.moe_w4a16_forward_rms.restype = I
        L.moe_layer_forward.argtypes = [P, P, P, ctypes.c_int32, P, P, P, P, P, P, ctypes.c_float, P, P, D, P, Z, P]
        L.moe_layer_forward.restype = I
        L.moe_w4a16_forward_noalloc.argtypes = [P, P, P, P, P, P, P, P, D, P]
        L.moe_w4a16_forward_noalloc.restype = I
        L.moe_permute.argtypes, L.moe_permute.restype = [P, D, P, P, P, Z, P], I
        L.moe_pack_int4.argtypes, L.moe_pack_int4.restype = [P, I64, I64, P, P, P], I
        L.moe_quantize_int4.argtypes = [P, I64, I64, ctypes.c_int32, P, P, P, P]
        L.moe_quantize_int4.restype = I
        L.moe_w8a16_linear.argtypes = [P, P, P, ctypes.c_int32, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, Z,
                                       P]
        L.moe_w8a16_linear.restype = I
        L.moe_w8a16_workspace_size.argtypes = [ctypes.c_int32] * 4 + [ctypes.POINTER(Z)]
        L.moe_w8a16_workspace_size.restype = I
        L.moe_check_device_error.argtypes, L.moe_check_device_error.restype = [P, Z, P], I
        L.moe_noalloc_check_device_error.argtypes, L.moe_noalloc_check_device_error.restype = [P], I
        L.moe_profile_events.argtypes, L.moe_profile_events.restype = [P, P], I
        L.moe_forward_plan.argtypes, L.moe_forward_plan.restype = [D, ctypes.POINTER(ctypes.c_int32)], I
        S, C, I32, F = moe_strides, moe_kv4_cache, ctypes.c_int32, ctypes.c_float
        L.moe_qk_norm_rope.argtypes = [P, S, P, S, P, P, P, P, I32, I32, F, P, S, P, S, I32, I32, I32, I32, P]
        L.moe_qk_norm_rope.restype = I
        L.moe_kv4_append.argtypes, L.moe_kv4_append.restype = [P, S, P, S, P, I32, C, P, Z, P], I
        L.moe_kv4_read.argtypes, L.moe_kv4_read.restype = [P, I32, C, P, P, P, Z, P], I
        L.moe_kv4_workspace_size.argtypes = [I32, I32, I32, I32, ctypes.POINTER(Z)]
        L.moe_kv4_workspace_size.restype = I
        L.moe_kv4_attention.argtypes = [P, S, C, P, I32, P, P, I32, I32, I32, I32, F, P, S, P, P, Z, P]
        L.moe_kv4_attention.restype = I
        L.moe_kv4_attention_window.argtypes = [P, S, C, P, I32, P, P, I32, I32, I32, I32, F, I32, I32, P, S, P, P, Z, P]
        L.moe_kv4_attention_window.restype = I
        L.moe_w4a16_linear.argtypes, L.moe_w4a16_linear.restype = [P, P, P, P, I32, I32, I32, P, Z, P], I
        L.moe_w4a16_workspace_size.argtypes = [I32, I32, I32, ctypes.POINTER(Z)]
        L.moe_w4a16_workspace_size.restype = I
        L.moe_verify_drafts.argtypes = [P, I64, P, I64, P, P, P, P, P, I64, I32, I32, I32, P, P, P, Z, P]
        L.moe_verify_drafts.restype = I
        L.moe_verify_workspace_size.argtypes, L.moe_verify_workspace_size.restype = [I32, I32, I32, ctypes.POINTER(Z)], I
        _lib = L
    return _lib


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The current stream's handle, without a Stream object around it where PyTorch has the call.
_raw_stream, _device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _device is not None:
            return _raw_stream(_device())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream))


def _check(rc: int, where: str):
    if rc != 0:
        raise MoeError(rc, where)


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype or t.dim() != ndim:
        raise ValueError("%s must be %s with %d dims, got %s %s" % (name, dtype, ndim, t.dtype, tuple(t.shape)))
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA tensor" % name)


def moe_status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def moe_version() -> int:
    return lib().moe_version()


def moe_workspace_size(T: int, H: int, E: int, k: int, I: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(moe_dims(T, H, E, k, I), ctypes.byref(n)), "moe_workspace_size")
    return n.value


def workspace(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace of moe_workspace_size bytes (owned by torch)."""
    return torch.zeros(moe_workspace_size(T, H, E, k, I), dtype=torch.uint8,
                       device=device if device is not None else "cuda")


def _ws(ws, dims: moe_dims, device):
    if ws is None:
        ws = workspace(dims.T, dims.H, dims.E, dims.k, dims.I, device)
    return ws


def moe_route(hidden, router_w, k: int, bias=None, ws=None, topk_ids=None, topk_w=None, stream=None):
    """Router GEMM, softmax, top-k (ties to the lower id) and renormalised weights.

    Returns (topk_ids int32 [T, k], topk_w f32 [T, k]).
    """
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(router_w, "router_w", torch.bfloat16, 2)
    T, H = hidden.shape
    E = router_w.shape[0]
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
    dims = moe_dims(T, H, E, k, 128)
    ws = _ws(ws, dims, hidden.device)
    if topk_ids is None:
        topk_ids = torch.empty(T, k, dtype=torch.int32, device=hidden.device)
    if topk_w is None:
        topk_w = torch.empty(T, k, dtype=torch.float32, device=hidden.device)
    _check(lib().moe_route(_p(hidden), _p(router_w), _p(bias), dims, _p(topk_ids), _p(topk_w), _p(ws),
                           ws.numel(), _stream(stream)), "moe_route")
    return topk_ids, topk_w


def shared_workspace(T: int, H: int, E: int, k: int, I: int, device=None) -> torch.Tensor:
    """A zeroed workspace that serves moe_route_shared (routed dims E, k) and the
    forward of the layer with its shared expert (E + 1 experts, k + 1 slots)."""
    n = max(moe_workspace_size(T, H, E, k, I), moe_workspace_size(T, H, E + 1, k + 1, I))
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def moe_route_shared(hidden, router_w, k: int, bias=None, ws=None, topk_ids=None, topk_w=None, stream=None):
    """Routing of a layer with a shared expert: router_w [E+1, H], row E the shared gate.

    Returns (topk_ids int32 [T, k+1], topk_w f32 [T, k+1]); slot k is expert E with
    weight sigmoid(gate). Pass them to moe_w4a16_forward with the E+1 experts' weights.
    """
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(router_w, "router_w", torch.bfloat16, 2)
    T, H = hidden.shape
    E = router_w.shape[0] - 1
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
    dims = moe_dims(T, H, E, k, 128)
    if ws is None:
        ws = shared_workspace(T, H, E, k, 128, hidden.device)
    if topk_ids is None:
        topk_ids = torch.empty(T, k + 1, dtype=torch.int32, device=hidden.device)
    if topk_w is None:
        topk_w = torch.empty(T, k + 1, dtype=torch.float32, device=hidden.device)
    _check(lib().moe_route_shared(_p(hidden), _p(router_w), _p(bias), dims, _p(topk_ids), _p(topk_w), _p(ws),
                                  ws.numel(), _stream(stream)), "moe_route_shared")
    return topk_ids, topk_w


def _expert_dims(hidden, topk_ids, w1_packed, w2_packed):
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(w1_packed, "w1_packed", torch.int32, 3)
    _need(w2_packed, "w2_packed", torch.int32, 3)
    T, H = hidden.shape
    E, two_i, _ = w1_packed.shape
    return moe_dims(T, H, E, topk_ids.shape[1], two_i // 2)


def moe_w4a16_forward(hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales,
                      out=None, ws=None, stream=None):
    """Routed-expert forward: bf16 out [T, H] = sum_j w_j * W2 (SiLU(W1g x) * W1u x)."""
    dims = _expert_dims(hidden, topk_ids, w1_packed, w2_packed)
    _need(topk_w, "topk_w", torch.float32, 2)
    _need(w1_scales, "w1_scales", torch.bfloat16, 3)
    _need(w2_scales, "w2_scales", torch.bfloat16, 3)
    ws = _ws(ws, dims, hidden.device)
    if out is None:
        out = torch.empty_like(hidden)
    _check(lib().moe_w4a16_forward(_p(hidden), _p(topk_ids), _p(topk_w), _p(w1_packed), _p(w1_scales),
                                   _p(w2_packed), _p(w2_scales), _p(out), dims, _p(ws), ws.numel(),
                                   _stream(stream)), "moe_w4a16_forward")
    return out


def moe_w4a16_forward_noalloc(hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales,
                              out=None, stream=None):
    """moe_w4a16_forward for decode batches (T <= 8) with the library's own static scratch.

    No workspace is passed or allocated; calls on one device must not overlap.
    """
    dims = _expert_dims(hidden, topk_ids, w1_packed, w2_packed)
    _need(topk_w, "topk_w", torch.float32, 2)
    _need(w1_scales, "w1_scales", torch.bfloat16, 3)
    _need(w2_scales, "w2_scales", torch.bfloat16, 3)
    if out is None:
        out = torch.empty_like(hidden)
    _check(lib().moe_w4a16_forward_noalloc(_p(hidden), _p(topk_ids), _p(topk_w), _p(w1_packed), _p(w1_scales),
                                           _p(w2_packed), _p(w2_scales), _p(out), dims, _stream(stream)),
           "moe_w4a16_forward_noalloc")
    return out


def moe_w4a16_forward_rms(hidden, topk_ids, topk_w, w1_packed, w1_scales, w2_packed, w2_scales,
                          eps: float = 1e-6, next=None, ws=None, stream=None):
    """Forward, then next = bf16((hidden + moe) / rms(hidden + moe)) (stack epilogue)."""
    dims = _expert_dims(hidden, topk_ids, w1_packed, w2_packed)
    _need(topk_w, "topk_w", torch.float32, 2)
    _need(w1_scales, "w1_scales", torch.bfloat16, 3)
    _need(w2_scales, "w2_scales", torch.bfloat16, 3)
    ws = _ws(ws, dims, hidden.device)
    if next is None:
        next = torch.empty_like(hidden)
    _check(lib().moe_w4a16_forward_rms(_p(hidden), _p(topk_ids), _p(topk_w), _p(w1_packed), _p(w1_scales),
                                       _p(w2_packed), _p(w2_scales), _p(next), float(eps), dims, _p(ws),
                                       ws.numel(), _stream(stream)), "moe_w4a16_forward_rms")
    return next


def moe_layer_forward(hidden, router_w, k: int, w1_packed, w1_scales, w2_packed, w2_scales, bias=None,
                      shared: bool = False, rms: bool = False, eps: float = 1e-6, out=None, topk_ids=None,
                      topk_w=None, ws=None, stream=None):
    """Router and experts in one call: moe_route (moe_route_shared with shared)
    then moe_w4a16_forward (moe_w4a16_forward_rms with rms), one kernel for
    decode batches. router_w [E (+1), H]; the weights hold E (+1) experts.

    Returns (out or next bf16 [T, H], topk_ids int32 [T, k (+1)], topk_w f32 [T, k (+1)]).
    """
    _need(hidden, "hidden", torch.bfloat16, 2)
    _need(router_w, "router_w", torch.bfloat16, 2)
    _need(w1_packed, "w1_packed", torch.int32, 3)
    _need(w2_packed, "w2_packed", torch.int32, 3)
    _need(w1_scales, "w1_scales", torch.bfloat16, 3)
    _need(w2_scales, "w2_scales", torch.bfloat16, 3)
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
    T, H = hidden.shape
    g = 1 if shared else 0
    E = router_w.shape[0] - g
    I = w1_packed.shape[1] // 2
    if w1_packed.shape[0] != E + g or w2_packed.shape[0] != E + g:
        raise ValueError("the weights must hold %d experts (router rows %d%s), got %d and %d"
                         % (E + g, router_w.shape[0], ", the last the shared gate" if g else "",
                            w1_packed.shape[0], w2_packed.shape[0]))
    dims = moe_dims(T, H, E, k, I)
    if ws is None:
        ws = shared_workspace(T, H, E, k, I, hidden.device) if shared else workspace(T, H, E, k, I, hidden.device)
    if topk_ids is None:
        topk_ids = torch.empty(T, k + g, dtype=torch.int32, device=hidden.device)
    if topk_w is None:
        topk_w = torch.empty(T, k + g, dtype=torch.float32, device=hidden.device)
    if out is None:
        out = torch.empty_like(hidden)
    _check(lib().moe_layer_forward(_p(hidden), _p(router_w), _p(bias), g, _p(w1_packed), _p(w1_scales),
                                   _p(w2_packed), _p(w2_scales), None if rms else _p(out), _p(out) if rms else None,
                                   float(eps), _p(topk_ids), _p(topk_w), dims, _p(ws), ws.numel(), _stream(stream)),
           "moe_layer_forward")
    return out, topk_ids, topk_w


def moe_permute(topk_ids, E: int, H: int = 128, I: int = 128, ws=None, stream=None):
    """(offsets int32 [E+1], perm int32 [T*k]) of the stable token-to-expert permutation."""
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    dims = moe_dims(T, H, E, k, I)
    ws = _ws(ws, dims, topk_ids.device)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=topk_ids.device)
    perm = torch.empty(T * k, dtype=torch.int32, device=topk_ids.device)
    _check(lib().moe_permute(_p(topk_ids), dims, _p(offsets), _p(perm), _p(ws), ws.numel(), _stream(stream)),
           "moe_permute")
    return offsets, perm


def moe_pack_int4(q, bad_count=None, stream=None):
    """int32 [N, K/8] storage words of int8 q [N, K] in [-8, 7]."""
    _need(q, "q", torch.int8, 2)
    N, K = q.shape
    packed = torch.empty(N, K // 8, dtype=torch.int32, device=q.device)
    if bad_count is not None:
        _need(bad_count, "bad_count", torch.int32, 1)
    _check(lib().moe_pack_int4(_p(q), N, K, _p(packed), _p(bad_count), _stream(stream)), "moe_pack_int4")
    return packed


def moe_forward_plan(T: int, H: int, E: int, k: int, I: int):
    """None if a forward of these dims takes the tensor-core pipeline, else
    (staged, groups_per_chunk, separate_block_buffers, routes_itself) of the
    fused decode kernel it runs; routes_itself: moe_layer_forward runs the
    router in the same kernel for these (forward) dims."""
    v = ctypes.c_int32(-1)
    _check(lib().moe_forward_plan(moe_dims(T, H, E, k, I), ctypes.byref(v)), "moe_forward_plan")
    if v.value == 0:
        return None
    return (v.value & 15) == 1, (v.value >> 4) & 15, bool(v.value & 256), bool(v.value & 512)


def moe_quantize_int4(w, nclip: int = 50, with_choice: bool = False, stream=None):
    """RTN INT4 g128 symmetric quantisation of bf16 w [N, K] with a per-group clip search.

    Returns (packed int32 [N, K/8], scales bf16 [N, K/128]) and, with with_choice,
    the chosen clip index int32 [N, K/128] (clip = (100 - j) / 100).
    """
    _need(w, "w", torch.bfloat16, 2)
    N, K = w.shape
    packed = torch.empty(N, K // 8, dtype=torch.int32, device=w.device)
    scales = torch.empty(N, K // 128, dtype=torch.bfloat16, device=w.device)
    choice = torch.empty(N, K // 128, dtype=torch.int32, device=w.device) if with_choice else None
    _check(lib().moe_quantize_int4(_p(w), N, K, nclip, _p(packed), _p(scales), _p(choice), _stream(stream)),
           "moe_quantize_int4")
    return (packed, scales, choice) if with_choice else (packed, scales)


def moe_w8a16_linear(x, w_packed, scales, gs: int, y=None, ws=None, stream=None):
    """bf16 y [T, N] = x . W^T for INT8 pack-quantized W (q + 128, four per int32 word, LSB first)
    with bf16 scales per gs (64 or 128) values of K. T <= 8: the decode GEMV; larger T: the
    tensor-core GEMM, whose error word (and split partial results) live in ws (a zeroed uint8
    tensor of moe_w8a16_workspace_size bytes; allocated here when not given)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(w_packed, "w_packed", torch.int32, 2)
    _need(scales, "scales", torch.bfloat16, 2)
    T, K = x.shape
    N = w_packed.shape[0]
    if w_packed.shape[1] * 4 != K or scales.shape != (N, K // gs):
        raise ValueError("w_packed must be [N, K/4] and scales [N, K/gs]")
    if y is None:
        y = torch.empty(T, N, dtype=torch.bfloat16, device=x.device)
    if ws is None and T > 8:
        ws = torch.zeros(moe_w8a16_workspace_size(T, N, K, gs), dtype=torch.uint8, device=x.device)
    nbytes = 0 if ws is None else ws.numel()
    _check(lib().moe_w8a16_linear(_p(x), _p(w_packed), _p(scales), gs, _p(y), T, N, K, _p(ws), nbytes,
                                  _stream(stream)), "moe_w8a16_linear")
    return y


def moe_w8a16_workspace_size(T: int, N: int, K: int, gs: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_w8a16_workspace_size(T, N, K, gs, ctypes.byref(n)), "moe_w8a16_workspace_size")
    return n.value


_BF16, _I32, _F32, _Tensor = torch.bfloat16, torch.int32, torch.float32, torch.Tensor


class Kv4Cache:
    """One layer's paged 4-bit KV cache: codes int32 [pages, Hkv, page_size, D/8] (q + 8, eight to a
    word, lowest nibble first) and scales bf16 [pages, Hkv, page_size], of K and of V. The slot of a
    token is page * page_size + its place in the page. Iterates over its four tensors."""
    __slots__ = ("k_codes", "k_scales", "v_codes", "v_scales", "_c")

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self._c = (None, None)

    def __iter__(self):
        return iter((self.k_codes, self.k_scales, self.v_codes, self.v_scales))

    def c(self):
        """(C struct, KV heads, D). The tensors are checked at every call, also where one has been
        replaced, resized or viewed anew at the same address."""
        kc, ks, vc, vs = self.k_codes, self.k_scales, self.v_codes, self.v_scales
        try:
            n, h, p, w = shape = kc.shape
            rows = (n, h, p)
            good = (kc.dtype is _I32 and vc.dtype is _I32 and ks.dtype is _BF16 and vs.dtype is _BF16
                    and vc.shape == shape and ks.shape == rows and vs.shape == rows
                    and kc.is_cuda and ks.is_cuda and vc.is_cuda and vs.is_cuda
                    and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous())
        except (AttributeError, ValueError):   # not tensors, or of other dimensions
            good = False
        if not good:
            _need(kc, "k_codes", torch.int32, 4)
            _need(ks, "k_scales", torch.bfloat16, 3)
            _need(vc, "v_codes", torch.int32, 4)
            _need(vs, "v_scales", torch.bfloat16, 3)
            raise ValueError("a cache holds codes [pages, Hkv, page_size, D/8] and scales [pages, Hkv, page_size], "
                             "got %s %s %s %s" % tuple(tuple(t.shape) for t in self))
        at = (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), shape)
        if self._c[0] != at:   # (forming the struct takes longer than finding that it holds these values)
            self._c = at, moe_kv4_cache(*at[:4], n, h, p, w * 8)
        return self._c[1], h, w * 8


def kv4_cache(n_pages: int, Hkv: int, page_size: int, D: int, device=None) -> Kv4Cache:
    """A cache of zeroed rows (D 64 or 128; page_size a power of two from 16 to 1024)."""
    device = device if device is not None else "cuda"
    codes = [torch.full((n_pages, Hkv, page_size, D // 8), -0x77777778, dtype=torch.int32, device=device)
             for _ in range(2)]
    scales = [torch.zeros(n_pages, Hkv, page_size, dtype=torch.bfloat16, device=device) for _ in range(2)]
    return Kv4Cache(codes[0], scales[0], codes[1], scales[1])


def moe_kv4_workspace_size(T: int, Hq: int, Hkv: int, D: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_kv4_workspace_size(T, Hq, Hkv, D, ctypes.byref(n)), "moe_kv4_workspace_size")
    return n.value


def kv4_workspace(T: int = 0, Hq: int = 1, Hkv: int = 1, D: int = 128, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace of moe_kv4_workspace_size bytes (with no dims: what
    moe_kv4_append and moe_kv4_read need)."""
    n = moe_kv4_workspace_size(T, Hq, Hkv, D) if T else 256
    return torch.zeros(n, dtype=torch.uint8, device=device if device is not None else "cuda")


_strides = {}   # (token, head) -> the struct: few pairs occur, and forming one costs more than finding it


def _heads(t, name, T=None, heads=None, D=None):
    """The strides, and the shape, of a bf16 [T, heads, D] CUDA tensor with contiguous D."""
    if type(t) is not _Tensor and not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    shape = t.shape
    good = t.dtype is _BF16 and len(shape) == 3
    if good:
        n, h, d = shape
        good = (T is None or n == T) and (heads is None or h == heads) and (D is None or d == D)
    if not good:
        raise ValueError("%s must be bf16 [%s, %s, %s], got %s %s" % (
            name, "T" if T is None else T, "heads" if heads is None else heads, "D" if D is None else D, t.dtype,
            tuple(shape)))
    token, head, one = t.stride()
    if not t.is_cuda or (one != 1 and d > 1):
        raise ValueError("%s must be a CUDA tensor with contiguous head values" % name)
    # (a dimension of one entry has no stride that matters)
    key = (token if n > 1 else 0, head if h > 1 else 0)
    st = _strides.get(key)
    if st is None:
        if len(_strides) > 4096:
            _strides.clear()
        st = _strides[key] = moe_strides(*key)
    return st, shape


def _vec(t, name, dtype, n=None):
    if type(t) is not _Tensor and not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    shape = t.shape
    if t.dtype is not dtype or (len(shape) != 1 if n is None else shape != (n,)) or not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s CUDA tensor%s, got %s %s"
                         % (name, dtype, "" if n is None else " of %d values" % n, t.dtype, tuple(shape)))
    return t.data_ptr()


def _made_on(stream):
    """Outputs and workspaces that a call makes belong to the stream that it runs on: their clears come before the
    kernels, and their memory is not given to another stream's tensors while the kernels run."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _ws_bytes(ws):
    """(address, bytes) of a workspace."""
    if type(ws) is not _Tensor and not isinstance(ws, _Tensor):
        raise TypeError("ws must be a torch.Tensor")
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor")
    return ws.data_ptr(), ws.nbytes


def _cache(c):
    """(C struct, KV heads, D) of a Kv4Cache, or of four tensors in its order."""
    return (c if isinstance(c, Kv4Cache) else Kv4Cache(*c)).c()


def moe_qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of each head of q [T, Hq, D] and k [T, Hkv, D], then the rotary turn of the first
    2 * len(inv_freq) values by positions[t] * inv_freq[i], in one pass.

    q and k are bf16 and may be views (their D values contiguous); the outputs may be the inputs.
    positions int32 [T], inv_freq f32 [rot/2] (both None: norms alone), weights bf16 [D] or None.
    The pairs are (i, i + rot/2), or (2i, 2i + 1) with interleaved. Returns (q_out, k_out).
    """
    if stream is not None and (q_out is None or k_out is None):
        with _made_on(stream):
            return moe_qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out)
    qs, (T, Hq, D) = _heads(q, "q")
    ks, (_, Hkv, _) = _heads(k, "k", T, None, D)
    if q_out is None:
        q_out = torch.empty(T, Hq, D, dtype=_BF16, device=q.device)
    if k_out is None:
        k_out = torch.empty(T, Hkv, D, dtype=_BF16, device=q.device)
    qos, kos = _heads(q_out, "q_out", T, Hq, D)[0], _heads(k_out, "k_out", T, Hkv, D)[0]
    pos = fr = None
    rot = 0
    if inv_freq is not None:
        fr, rot = _vec(inv_freq, "inv_freq", torch.float32), 2 * inv_freq.shape[0]
        pos = _vec(positions, "positions", torch.int32, T)
    _check(lib().moe_qk_norm_rope(q.data_ptr(), qs, k.data_ptr(), ks,
                                  None if q_weight is None else _vec(q_weight, "q_weight", torch.bfloat16, D),
                                  None if k_weight is None else _vec(k_weight, "k_weight", torch.bfloat16, D),
                                  pos, fr, rot, 1 if interleaved else 0, eps, q_out.data_ptr(), qos, k_out.data_ptr(),
                                  kos, T, Hq, Hkv, D, _stream(stream)), "moe_qk_norm_rope")
    return q_out, k_out


def moe_kv4_append(k, v, slots, cache: Kv4Cache, ws=None, stream=None):
    """Quantises token t's rows k[t], v[t] (bf16 [T, Hkv, D], views allowed) into the cache at
    slots[t] (int32 [T]; -1: not stored). ws: kv4_workspace(), whose error word
    moe_check_device_error reads. Returns the cache."""
    if stream is not None and ws is None:
        with _made_on(stream):
            return moe_kv4_append(k, v, slots, cache)
    c, Hkv, D = _cache(cache)
    ks, (T, _, _) = _heads(k, "k", None, Hkv, D)
    vs = _heads(v, "v", T, Hkv, D)[0]
    if ws is None:
        ws = kv4_workspace(device=k.device)
    _check(lib().moe_kv4_append(k.data_ptr(), ks, v.data_ptr(), vs, _vec(slots, "slots", torch.int32, T), T, c,
                                *_ws_bytes(ws), _stream(stream)), "moe_kv4_append")
    return cache


def moe_kv4_read(slots, cache: Kv4Cache, k_out=None, v_out=None, ws=None, stream=None):
    """The cache's rows at slots (int32 [T]; -1 reads as zero) as bf16 values: (k, v) [T, Hkv, D]."""
    if stream is not None and (k_out is None or v_out is None or ws is None):
        with _made_on(stream):
            return moe_kv4_read(slots, cache, k_out, v_out, ws)
    c, Hkv, D = _cache(cache)
    at = _vec(slots, "slots", torch.int32)
    shape = (slots.shape[0], Hkv, D)
    if k_out is None:
        k_out = torch.empty(shape, dtype=torch.bfloat16, device=slots.device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=torch.bfloat16, device=slots.device)
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        _need(t, name, torch.bfloat16, 3)
        if t.shape != shape:
            raise ValueError("%s must be %s, got %s" % (name, shape, tuple(t.shape)))
    if ws is None:
        ws = kv4_workspace(device=slots.device)
    _check(lib().moe_kv4_read(at, shape[0], c, k_out.data_ptr(), v_out.data_ptr(), *_ws_bytes(ws),
                              _stream(stream)), "moe_kv4_read")
    return k_out, v_out


def moe_kv4_attention(q, cache: Kv4Cache, page_table, lens, cu_q=None, max_q=None, scale=None, out=None,
                      lse=None, ws=None, stream=None):
    """Causal attention of q [T, Hq, D] (bf16, views allowed) over the 4-bit cache.

    Sequence b has the queries [cu_q[b], cu_q[b+1]) (cu_q int32 [B+1]; None: one each) and lens[b] keys
    (int32 [B]), the new tokens' own among them, in the pages page_table[b] (int32 [B, max_pages]).
    max_q is the largest number of queries of a sequence: it chooses the kernel, never the result (None: 1
    without cu_q, else the mean, rounded up; give it where the counts differ). scale defaults to D ** -0.5.
    ws: kv4_workspace(T, Hq, Hkv, D). Returns out, or (out, lse f32 [T, Hq]) where lse is given
    (a tensor, or True to have it made)."""
    if stream is not None and (out is None or lse is True or ws is None):
        with _made_on(stream):
            return moe_kv4_attention(q, cache, page_table, lens, cu_q, max_q, scale, out, lse, ws)
    return _attention(q, cache, page_table, lens, cu_q, max_q, scale, out, lse, ws, stream, None, 0)


def moe_kv4_attention_window(q, cache: Kv4Cache, page_table, lens, window: int, sinks: int = 0, cu_q=None, max_q=None,
                             scale=None, out=None, lse=None, ws=None, stream=None):
    """moe_kv4_attention with a sliding window: the query at position i sees the keys j <= i with j > i - window
    or j < sinks. Pages that lie wholly before the windows of a sequence's queries (and hold no first keys)
    may be gone: their entries in page_table are not looked at."""
    if stream is not None and (out is None or lse is True or ws is None):
        with _made_on(stream):
            return moe_kv4_attention_window(q, cache, page_table, lens, window, sinks, cu_q, max_q, scale, out, lse, ws)
    return _attention(q, cache, page_table, lens, cu_q, max_q, scale, out, lse, ws, stream, window, sinks)


def _attention(q, cache, page_table, lens, cu_q, max_q, scale, out, lse, ws, stream, window, sinks):
    c, Hkv, D = _cache(cache)
    qs, (T, Hq, _) = _heads(q, "q", None, None, D)
    at = _vec(lens, "lens", torch.int32)
    B = lens.shape[0]
    cu = None if cu_q is None else _vec(cu_q, "cu_q", torch.int32, B + 1)
    if max_q is None:
        max_q = 1 if cu is None else -(-T // max(B, 1))
    _need(page_table, "page_table", torch.int32, 2)
    if page_table.shape[0] != B:
        raise ValueError("page_table must have a row for each of the %d sequences, got %s" % (B, tuple(page_table.shape)))
    if out is None:
        out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=q.device)
    os_ = _heads(out, "out", T, Hq, D)[0]
    if lse is True:
        lse = torch.empty(T, Hq, dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", _F32, 2)
        if lse.shape != (T, Hq):
            raise ValueError("lse must be [%d, %d], got %s" % (T, Hq, tuple(lse.shape)))
    if ws is None:   # for this call alone: of what the call leaves zero it uses the control block only
        ws = torch.empty(moe_kv4_workspace_size(T, Hq, Hkv, D), dtype=torch.uint8, device=q.device)
        ws[:256].zero_()
    args = (q.data_ptr(), qs, c, page_table.data_ptr(), page_table.shape[1], at, cu, B, T, Hq, max_q,
            D ** -0.5 if scale is None else scale)
    rest = (out.data_ptr(), os_, None if lse is None else lse.data_ptr(), *_ws_bytes(ws), _stream(stream))
    if window is None:
        _check(lib().moe_kv4_attention(*args, *rest), "moe_kv4_attention")
    else:
        if not (0 <= window <= 0x7FFFFFFF and 0 <= sinks <= 0x7FFFFFFF):
            # the C call counts in 32 bits, past which nothing is hidden; what is below its range stays below it
            window, sinks = min(max(window, -1), 0x7FFFFFFF), min(max(sinks, -1), 0x7FFFFFFF)
        _check(lib().moe_kv4_attention_window(*args, window, sinks, *rest), "moe_kv4_attention_window")
    return out if lse is None else (out, lse)


def _mat(t, name, dtype, rows=None, cols=None):
    """The address and shape of a contiguous CUDA matrix."""
    if type(t) is not _Tensor and not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    shape = t.shape
    good = t.dtype is dtype and len(shape) == 2 and t.is_cuda and t.is_contiguous()
    if not good or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError("%s must be a contiguous %s CUDA tensor [%s, %s], got %s %s" % (
            name, dtype, "rows" if rows is None else rows, "columns" if cols is None else cols, t.dtype, tuple(shape)))
    return t.data_ptr(), shape


def moe_w4a16_workspace_size(T: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_w4a16_workspace_size(T, N, K, ctypes.byref(n)), "moe_w4a16_workspace_size")
    return n.value


def moe_w4a16_linear(x, w_packed, scales, y=None, ws=None, stream=None):
    """bf16 y [T, N] = x . W^T for INT4 weights in the experts' storage (moe_quantize_int4's): w_packed
    int32 [N, K/8] (q + 8, eight to a word, lowest nibble first), scales bf16 [N, K/128]. ws: a
    uint8 tensor of moe_w4a16_workspace_size bytes (allocated here when not given); the call neither reads
    nor writes it."""
    if stream is not None and (y is None or ws is None):
        with _made_on(stream):
            return moe_w4a16_linear(x, w_packed, scales, y, ws)
    xp, (T, K) = _mat(x, "x", _BF16)
    if K % 128:
        raise ValueError("x must have a multiple of 128 columns, got %d" % K)
    wp, (N, _) = _mat(w_packed, "w_packed", _I32, None, K // 8)
    sp, _ = _mat(scales, "scales", _BF16, N, K // 128)
    if y is None:
        y = torch.empty(T, N, dtype=_BF16, device=x.device)
    yp, _ = _mat(y, "y", _BF16, T, N)
    if ws is None:   # (nothing is kept in it)
        ws = torch.empty(moe_w4a16_workspace_size(T, N, K), dtype=torch.uint8, device=x.device)
    _check(lib().moe_w4a16_linear(xp, wp, sp, yp, T, N, K, *_ws_bytes(ws), _stream(stream)), "moe_w4a16_linear")
    return y


def moe_verify_workspace_size(B: int, T: int, V: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_verify_workspace_size(B, T, V, ctypes.byref(n)), "moe_verify_workspace_size")
    return n.value


def verify_workspace(B: int, T: int, V: int, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace of moe_verify_workspace_size bytes."""
    return torch.zeros(moe_verify_workspace_size(B, T, V), dtype=torch.uint8, device=device if device is not None else "cuda")


def _wide(t, name, dtype, rows=None, cols=None):
    """Address, row stride and shape of a CUDA matrix with contiguous rows (a view of a wider one, say)."""
    if type(t) is not _Tensor and not isinstance(t, _Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    shape = t.shape
    good = t.dtype is dtype and len(shape) == 2 and t.is_cuda and (rows is None or shape[0] == rows) and (cols is None or shape[1] == cols)
    if good:
        n, m = shape
        stride, one = t.stride()
        good = one == 1 or m <= 1
    if not good:
        raise ValueError("%s must be a %s CUDA tensor [%s, %s] with contiguous rows, got %s %s" % (
            name, dtype, "rows" if rows is None else rows, "columns" if cols is None else cols, t.dtype, tuple(shape)))
    return t.data_ptr(), stride if n > 1 else 0, shape


def moe_verify_drafts(logits, drafts, cu_rows, uniform, noise, draft_logits=None, temperature=None, tokens=None,
                      accepted=None, ws=None, stream=None):
    """Which drafted tokens the target accepts, and the token after them.

    Sequence b has the rows [cu_rows[b], cu_rows[b+1]) (int32 [B+1]) of logits (bf16 [T, V], rows a multiple of 8
    values apart): its drafts' and one more. drafts int32 [T] (the draft at each row; a last row's is not read);
    uniform f32 [T] from [0, 1); noise f32 [B, V] from Exp(1) (rows a multiple of 4 apart); draft_logits as logits,
    or None where the drafts were not drawn from probabilities; temperature f32 [B] (0: the largest logit; None: 1).
    ws: verify_workspace(B, T, V). Returns (tokens int32 [T]: the accepted drafts, the next token, then -1;
    accepted int32 [B])."""
    if stream is not None and (tokens is None or accepted is None or ws is None):
        with _made_on(stream):
            return moe_verify_drafts(logits, drafts, cu_rows, uniform, noise, draft_logits, temperature, tokens, accepted, ws)
    lp, ls, (T, V) = _wide(logits, "logits", _BF16)
    dp, ds = (None, 0) if draft_logits is None else _wide(draft_logits, "draft_logits", _BF16, T, V)[:2]
    cu = _vec(cu_rows, "cu_rows", _I32)
    B = cu_rows.shape[0] - 1
    if B < 0:
        raise ValueError("cu_rows must hold an offset for each sequence and one more")
    ep, es = _wide(noise, "noise", _F32, B, V)[:2]
    if tokens is None:
        tokens = torch.empty(T, dtype=_I32, device=logits.device)
    if accepted is None:
        accepted = torch.empty(B, dtype=_I32, device=logits.device)
    if ws is None:   # for this call alone: of what the call leaves zero it uses the control block only
        ws = torch.empty(moe_verify_workspace_size(B, T, V), dtype=torch.uint8, device=logits.device)
        ws[:256].zero_()
    _check(lib().moe_verify_drafts(lp, ls, dp, ds, _vec(drafts, "drafts", _I32, T), cu,
                                   None if temperature is None else _vec(temperature, "temperature", _F32, B),
                                   _vec(uniform, "uniform", _F32, T), ep, es, B, T, V, _vec(tokens, "tokens", _I32, T),
                                   _vec(accepted, "accepted", _I32, B), *_ws_bytes(ws), _stream(stream)), "moe_verify_drafts")
    return tokens, accepted


def moe_profile_events(before=None, after=None):
    """Record two torch.cuda.Events (enable_timing=True, external=True) around
    the expert kernel of every later forward call; (None, None) stops."""
    b = None if before is None else ctypes.c_void_p(before.cuda_event)
    a = None if after is None else ctypes.c_void_p(after.cuda_event)
    _check(lib().moe_profile_events(b, a), "moe_profile_events")


def moe_check_device_error(ws, stream=None) -> int:
    """Synchronise the stream; return (and clear) the workspace's device error status."""
    return lib().moe_check_device_error(_p(ws), ws.numel(), _stream(stream))


def moe_noalloc_check_device_error(stream=None) -> int:
    """Synchronise the stream; return (and clear) the error status of the no-alloc scratch."""
    return lib().moe_noalloc_check_device_error(_stream(stream))

"""Python binding of the NVFP4 routed-expert MoE library (libnvfp4moe.so, sm_100a).

Every function here has the name of a C entry point in ``include/nvfp4_moe.h`` and only
marshals arguments: it checks tensors, allocates outputs and workspaces with PyTorch,
passes raw device pointers and the current CUDA stream through ctypes, and turns a
negative status into an exception.  All arithmetic runs in the library's kernels; there is
no fallback.  If the shared library is missing, the first call raises (importing the
package alone does not, so the build script inside it stays importable).

Format (page "GLM-5-NVFP4-MTP", "Model Description"): 4-bit E2M1 values, one E4M3 scale per
16 consecutive elements, one fp32 global scale per tensor.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "PATH_AUTO", "PATH_GEMV", "PATH_GEMM", "NVFP4Error", "lib", "library_path",
    "nvfp4_quantize", "nvfp4_quantize_workspace_size", "nvfp4_dequantize", "nvfp4_cast_f32",
    "moe_nvfp4_route", "moe_nvfp4_workspace_size", "moe_nvfp4_forward",
    "moe_nvfp4_read_error_flag", "moe_nvfp4_forward_profiled", "alloc_moe_workspace",
    "moe_nvfp4_forward_static", "nvfp4_selftest_wait_timeout",
    "nvfp4_selftest_gate_up_timeout", "nvfp4_selftest_int8_matmul_timeout", "nvfp4_amax",
    "nvfp4_quantize_with_amax", "moe_nvfp4_ep_local_experts", "moe_nvfp4_forward_ep",
    "moe_nvfp4_ep_reduce", "EP_MAX_PARTS", "moe_nvfp4_router", "moe_nvfp4_forward_logits",
    "moe_nvfp4_shared_expert", "moe_nvfp4_layer", "moe_nvfp4_layer_workspace_size",
    "nvfp4_w4a4_prepare_scales", "moe_nvfp4_forward_w4a4", "moe_nvfp4_w4a4_workspace_size",
    "moe_nvfp4_pre_norm", "moe_nvfp4_pre_norm_int8", "moe_nvfp4_pre_norm_backward",
    "moe_nvfp4_post_norm", "moe_nvfp4_post_norm_backward",
    "moe_nvfp4_norm_backward_workspace_size", "ACT_SILU", "ACT_GELU", "moe_nvfp4_gate_up",
    "moe_nvfp4_gate_up_backward", "moe_nvfp4_gate_up_backward_workspace_size",
    "nvfp4_int8_quantize", "nvfp4_int8_matmul",
]

PATH_AUTO, PATH_GEMV, PATH_GEMM = 0, 1, 2
ACT_SILU, ACT_GELU = 0, 1    # gate activations of moe_nvfp4_gate_up
WORKSPACE_ZERO_BYTES = 512   # head of a workspace that must be zero before first use
EP_MAX_PARTS = 16            # partial outputs one moe_nvfp4_ep_reduce call sums
_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libnvfp4moe.so")


class NVFP4Error(RuntimeError):
    pass


def _load() -> ctypes.CDLL:
    if not os.path.exists(library_path):
        raise ImportError(
            f"{library_path} is missing: build it with "
            "`python -m bit_quantized_moe_nvfp4_b200.build` (nvcc, sm_100a)")
    L = ctypes.CDLL(library_path)
    P, I64, SZ, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    F32 = ctypes.c_float
    sig = {
        "nvfp4_status_string": (ctypes.c_char_p, [I32]),
        "nvfp4_last_cuda_error": (ctypes.c_char_p, []),
        "nvfp4_quantize_workspace_size": (SZ, [I64, I64, I64]),
        "nvfp4_quantize": (I32, [P, I64, I64, I64, P, P, P, P, SZ, P]),
        "nvfp4_dequantize": (I32, [P, P, P, I64, I64, I64, P, P]),
        "nvfp4_cast_f32": (I32, [P, I64, P, P, P]),
        "moe_nvfp4_workspace_size": (SZ, [I64, I64, I64, I64, I64]),
        "moe_nvfp4_forward": (I32, [P, P, P, I64, I64, I64, I64, I64,
                                    P, P, P, P, P, P, P, P, SZ, P]),
        "moe_nvfp4_forward_path": (I32, [P, P, P, I64, I64, I64, I64, I64,
                                         P, P, P, P, P, P, P, P, SZ, I32, P]),
        "moe_nvfp4_forward_profiled": (I32, [P, P, P, I64, I64, I64, I64, I64,
                                             P, P, P, P, P, P, P, P, SZ, I32, P, P]),
        "moe_nvfp4_read_error_flag": (I32, [P, P, P]),
        "moe_nvfp4_route": (I32, [P, I64, I64, I64, P, P, P, P, P, P]),
        "moe_nvfp4_forward_static": (I32, [P, P, P, I64, I64, I64, I64, I64,
                                           P, P, P, P, P, P, P, P, P]),
        "nvfp4_selftest_wait_timeout": (I32, [P, I32, I64, P]),
        "nvfp4_amax": (I32, [P, I64, I64, I64, P, I32, P]),
        "nvfp4_quantize_with_amax": (I32, [P, I64, I64, I64, P, P, P, P, P]),
        "moe_nvfp4_ep_local_experts": (I64, [I64, I64, I64]),
        "moe_nvfp4_forward_ep": (I32, [P, P, P, I64, I64, I64, I64, I64, I64, I64,
                                       P, P, P, P, P, P, P, P, SZ, I32, P]),
        "moe_nvfp4_ep_reduce": (I32, [P, I64, I64, I64, P, P]),
        "moe_nvfp4_router": (I32, [P, I64, I64, I64, P, P, P]),
        "nvfp4_w4a4_prepare_scales": (I32, [P, I64, I64, I64, I64, P, P]),
        "moe_nvfp4_w4a4_workspace_size": (SZ, [I64, I64, I64, I64, I64]),
        "moe_nvfp4_forward_w4a4_profiled": (I32, [P, P, P, I64, I64, I64, I64, I64,
                                                  P, P, P, P, P, P, P, P, SZ, P, P]),
        "moe_nvfp4_forward_w4a4": (I32, [P, P, P, I64, I64, I64, I64, I64,
                                         P, P, P, P, P, P, P, P, SZ, P]),
        "moe_nvfp4_pre_norm": (I32, [P, P, I64, I64, F32, P, P]),
        "moe_nvfp4_pre_norm_int8": (I32, [P, P, I64, I64, F32, P, P, P]),
        "moe_nvfp4_post_norm": (I32, [P, P, P, P, I64, I64, I64, I64, F32, F32, P, P, P, P]),
        "moe_nvfp4_norm_backward_workspace_size": (SZ, [I64, I64]),
        "moe_nvfp4_pre_norm_backward": (I32, [P, P, P, P, I64, I64, F32, P, P, P, SZ, P]),
        "moe_nvfp4_post_norm_backward": (I32, [P, P, P, P, I64, I64, I64, I64, F32, F32,
                                               P, P, P, P, P, SZ, P]),
        "moe_nvfp4_gate_up": (I32, [P, P, I64, I64, I64, I32, P, P, P, P]),
        "moe_nvfp4_gate_up_backward_workspace_size": (SZ, [I64, I64]),
        "moe_nvfp4_gate_up_backward": (I32, [P, P, P, P, I64, I64, I64, I32, P, P, P, SZ, P, P]),
        "nvfp4_selftest_gate_up_timeout": (I32, [P, P, I64, I64, I64, P, P, P, P]),
        "nvfp4_selftest_int8_matmul_timeout": (I32, [P, P, P, P, I64, I64, I64, P, P, P]),
        "nvfp4_int8_quantize": (I32, [P, I64, I64, P, P, P]),
        "nvfp4_int8_matmul": (I32, [P, P, P, P, I64, I64, I64, P, P, P]),
        "moe_nvfp4_shared_workspace_size": (SZ, [I64, I64]),
        "moe_nvfp4_shared_expert": (I32, [P, I64, I64, I64, P, P, P, P, P, SZ, P]),
        "moe_nvfp4_layer_workspace_size": (SZ, [I64, I64, I64, I64, I64, I64]),
        "moe_nvfp4_layer": (I32, [P, P, I64, I64, I64, I64, I64, P, P, P, P, P, P, P, P, I64,
                                  P, P, P, P, SZ, I32, P]),
        "moe_nvfp4_forward_logits": (I32, [P, P, I64, I64, I64, I64, I64,
                                           P, P, P, P, P, P, P, P, P, P, SZ, I32, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    return L


_LIB = None


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


def _check(status: int) -> None:
    lib = _lib()
    if status != 0:
        msg = lib.nvfp4_status_string(status).decode()
        if status == -4:
            msg += " -- " + lib.nvfp4_last_cuda_error().decode()
        raise NVFP4Error(msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor of {dtype}")


# ------------------------------------------------------------------------------ codec
def nvfp4_quantize_workspace_size(n_tensors: int, rows: int, cols: int) -> int:
    return int(_lib().nvfp4_quantize_workspace_size(n_tensors, rows, cols))


def nvfp4_quantize(x: torch.Tensor, packed=None, scales=None, global_scale=None,
                   workspace=None):
    """bf16 [n, rows, cols] (or [rows, cols]) -> (packed u8 [..., cols/2],
    scales u8 (E4M3 codes) [..., cols/16], global_scale fp32 [n])."""
    _need(x, torch.bfloat16, "x")
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    n, rows, cols = x3.shape
    dev = x.device
    if packed is None:
        packed = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((n, rows, cols // 16), dtype=torch.uint8, device=dev)
    if global_scale is None:
        global_scale = torch.empty((n,), dtype=torch.float32, device=dev)
    ws_bytes = nvfp4_quantize_workspace_size(n, rows, cols)
    if workspace is None:
        workspace = torch.empty((max(ws_bytes, 1),), dtype=torch.uint8, device=dev)
    _check(_lib().nvfp4_quantize(_ptr(x3), n, rows, cols, _ptr(packed), _ptr(scales),
                              _ptr(global_scale), _ptr(workspace), workspace.numel(),
                              _stream(dev)))
    if squeeze:
        return packed[0], scales[0], global_scale
    return packed, scales, global_scale


def nvfp4_amax(x: torch.Tensor, out=None, merge: bool = False) -> torch.Tensor:
    """Per-tensor max |x| of bf16 [n, rows, cols] (or [rows, cols]) -> fp32 [n].  With
    merge=True, `out` holds the amax of earlier calibration passes and becomes the
    element-wise max of it and this pass's."""
    _need(x, torch.bfloat16, "x")
    x3 = x.unsqueeze(0) if x.dim() == 2 else x
    n, rows, cols = x3.shape
    if out is None:
        if merge:
            raise ValueError("merge=True needs the running amax in `out`")
        out = torch.empty((n,), dtype=torch.float32, device=x.device)
    _need(out, torch.float32, "out")
    _check(_lib().nvfp4_amax(_ptr(x3), n, rows, cols, _ptr(out), int(bool(merge)),
                             _stream(x.device)))
    return out


def nvfp4_quantize_with_amax(x: torch.Tensor, amax: torch.Tensor, packed=None, scales=None,
                             global_scale=None):
    """nvfp4_quantize with the per-tensor amax given (a calibrated one): g = amax / 2688.
    -> (packed, scales, global_scale) as nvfp4_quantize."""
    _need(x, torch.bfloat16, "x")
    _need(amax, torch.float32, "amax")
    squeeze = x.dim() == 2
    x3 = x.unsqueeze(0) if squeeze else x
    n, rows, cols = x3.shape
    dev = x.device
    if packed is None:
        packed = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((n, rows, cols // 16), dtype=torch.uint8, device=dev)
    if global_scale is None:
        global_scale = torch.empty((n,), dtype=torch.float32, device=dev)
    _check(_lib().nvfp4_quantize_with_amax(_ptr(x3), n, rows, cols, _ptr(amax), _ptr(packed),
                                           _ptr(scales), _ptr(global_scale), _stream(dev)))
    if squeeze:
        return packed[0], scales[0], global_scale
    return packed, scales, global_scale


def nvfp4_dequantize(packed: torch.Tensor, scales: torch.Tensor, global_scale: torch.Tensor,
                     out=None) -> torch.Tensor:
    """Inverse of nvfp4_quantize up to rounding: bf16( fp32(e2m1 * e4m3) * g )."""
    _need(packed, torch.uint8, "packed")
    _need(scales, torch.uint8, "scales")
    _need(global_scale, torch.float32, "global_scale")
    squeeze = packed.dim() == 2
    p3 = packed.unsqueeze(0) if squeeze else packed
    n, rows, half = p3.shape
    cols = half * 2
    if out is None:
        out = torch.empty((n, rows, cols), dtype=torch.bfloat16, device=packed.device)
    _check(_lib().nvfp4_dequantize(_ptr(p3), _ptr(scales), _ptr(global_scale), n, rows, cols,
                                _ptr(out), _stream(packed.device)))
    return out[0] if squeeze else out


def nvfp4_cast_f32(v: torch.Tensor):
    """fp32 values -> (E4M3 codes u8, E2M1 codes u8), as the quantizer rounds them."""
    _need(v, torch.float32, "v")
    e4 = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    e2 = torch.empty(v.shape, dtype=torch.uint8, device=v.device)
    _check(_lib().nvfp4_cast_f32(_ptr(v), v.numel(), _ptr(e4), _ptr(e2), _stream(v.device)))
    return e4, e2


# ------------------------------------------------------------------------------ MoE
def moe_nvfp4_workspace_size(T: int, H: int, I: int, E: int, K: int) -> int:
    return int(_lib().moe_nvfp4_workspace_size(T, H, I, E, K))


def alloc_moe_workspace(T, H, I, E, K, device="cuda") -> torch.Tensor:
    """Workspace for moe_nvfp4_forward: its head (error flag and work counters) zeroed."""
    ws = torch.empty((moe_nvfp4_workspace_size(T, H, I, E, K),), dtype=torch.uint8,
                     device=device)
    ws[:WORKSPACE_ZERO_BYTES].zero_()
    return ws


def moe_nvfp4_route(topk_ids: torch.Tensor, E: int):
    """int32 [T, K] -> (counts [E], offsets [E+1], perm [T*K], inv [T*K], flag [1])."""
    _need(topk_ids, torch.int32, "topk_ids")
    T, K = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    perm = torch.full((T * K,), -1, dtype=torch.int32, device=dev)
    inv = torch.empty((T * K,), dtype=torch.int32, device=dev)
    flag = torch.zeros((1,), dtype=torch.int32, device=dev)
    _check(_lib().moe_nvfp4_route(_ptr(topk_ids), T, K, E, _ptr(counts), _ptr(offsets),
                               _ptr(perm), _ptr(inv), _ptr(flag), _stream(dev)))
    return counts, offsets, perm, inv, flag


def moe_nvfp4_forward(x, topk_ids, topk_w, w_gu, s_gu, g_gu, w_dn, s_dn, g_dn,
                      out=None, workspace=None, path: int = PATH_AUTO) -> torch.Tensor:
    """Routed-expert MoE MLP from NVFP4 weights (see include/nvfp4_moe.h).

    x bf16 [T,H]; topk_ids int32 [T,K]; topk_w fp32 [T,K]; w_gu u8 [E,2I,H/2];
    s_gu u8 [E,2I,H/16]; g_gu fp32 [E]; w_dn u8 [E,H,I/2]; s_dn u8 [E,H,I/16];
    g_dn fp32 [E].  Returns out bf16 [T,H]."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_w, torch.float32, "topk_w")
    for t, n in ((w_gu, "w_gu"), (s_gu, "s_gu"), (w_dn, "w_dn"), (s_dn, "s_dn")):
        _need(t, torch.uint8, n)
    _need(g_gu, torch.float32, "g_gu")
    _need(g_dn, torch.float32, "g_dn")
    T, H = x.shape
    K = topk_ids.shape[1]
    E, twoI, _ = w_gu.shape
    I = twoI // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_moe_workspace(T, H, I, E, K, x.device)
    _check(_lib().moe_nvfp4_forward_path(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, H, I, E, K, _ptr(w_gu), _ptr(s_gu),
        _ptr(g_gu), _ptr(w_dn), _ptr(s_dn), _ptr(g_dn), _ptr(out), _ptr(workspace),
        workspace.numel(), int(path), _stream(x.device)))
    return out


def moe_nvfp4_router(logits: torch.Tensor, K: int, ids=None, w=None):
    """Top-K experts and renormalised softmax weights from fp32 logits [T, E] (see
    include/nvfp4_moe.h).  Returns (ids int32 [T, K], w fp32 [T, K])."""
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    if ids is None:
        ids = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    _need(ids, torch.int32, "ids")
    _need(w, torch.float32, "w")
    _check(_lib().moe_nvfp4_router(_ptr(logits), T, E, K, _ptr(ids), _ptr(w),
                                   _stream(logits.device)))
    return ids, w


def moe_nvfp4_forward_logits(x, router_logits, K: int, w_gu, s_gu, g_gu, w_dn, s_dn, g_dn,
                             out=None, ids_out=None, w_out=None, workspace=None,
                             path: int = PATH_AUTO) -> torch.Tensor:
    """The router on fp32 logits [T, E], then the layer on its decisions, in one call.
    ids_out / w_out (optional, [T, K]) receive the router's decisions."""
    _need(x, torch.bfloat16, "x")
    _need(router_logits, torch.float32, "router_logits")
    for t, n in ((w_gu, "w_gu"), (s_gu, "s_gu"), (w_dn, "w_dn"), (s_dn, "s_dn")):
        _need(t, torch.uint8, n)
    _need(g_gu, torch.float32, "g_gu")
    _need(g_dn, torch.float32, "g_dn")
    if ids_out is not None:
        _need(ids_out, torch.int32, "ids_out")
    if w_out is not None:
        _need(w_out, torch.float32, "w_out")
    T, H = x.shape
    E, twoI, _ = w_gu.shape
    I = twoI // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = alloc_moe_workspace(T, H, I, E, K, x.device)
    _check(_lib().moe_nvfp4_forward_logits(
        _ptr(x), _ptr(router_logits), T, H, I, E, K, _ptr(w_gu), _ptr(s_gu), _ptr(g_gu),
        _ptr(w_dn), _ptr(s_dn), _ptr(g_dn), _ptr(out), _ptr(ids_out), _ptr(w_out),
        _ptr(workspace), workspace.numel(), int(path), _stream(x.device)))
    return out


def moe_nvfp4_shared_expert(x, w_gu, w_dn, routed=None, out=None, workspace=None):
    """The BF16 shared expert (see include/nvfp4_moe.h): out = bf16(routed + W_dn .
    bf16(silu(W_g x) * W_u x)) per token.  x bf16 [T,H]; w_gu bf16 [2Is,H]; w_dn bf16
    [H,Is]; routed fp32 [T,H] or None.  Returns out bf16 [T,H]."""
    _need(x, torch.bfloat16, "x")
    _need(w_gu, torch.bfloat16, "w_gu")
    _need(w_dn, torch.bfloat16, "w_dn")
    if routed is not None:
        _need(routed, torch.float32, "routed")
    T, H = x.shape
    Is = w_gu.shape[0] // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        n = int(_lib().moe_nvfp4_shared_workspace_size(T, Is))
        workspace = torch.empty((max(n, 16),), dtype=torch.uint8, device=x.device)
    _check(_lib().moe_nvfp4_shared_expert(_ptr(x), T, H, Is, _ptr(w_gu), _ptr(w_dn),
                                          _ptr(routed), _ptr(out), _ptr(workspace),
                                          workspace.numel(), _stream(x.device)))
    return out


def moe_nvfp4_layer_workspace_size(T, H, I, E, K, Is) -> int:
    return int(_lib().moe_nvfp4_layer_workspace_size(T, H, I, E, K, Is))


def moe_nvfp4_layer(x, router_logits, K: int, w_gu, s_gu, g_gu, w_dn, s_dn, g_dn,
                    shared_gu, shared_dn, out=None, ids_out=None, w_out=None, workspace=None,
                    path: int = PATH_AUTO) -> torch.Tensor:
    """The whole MoE layer in one call: router on the logits, the routed NVFP4 experts,
    and the BF16 shared expert added before the single rounding to bf16."""
    _need(x, torch.bfloat16, "x")
    _need(router_logits, torch.float32, "router_logits")
    for t, n in ((w_gu, "w_gu"), (s_gu, "s_gu"), (w_dn, "w_dn"), (s_dn, "s_dn")):
        _need(t, torch.uint8, n)
    _need(g_gu, torch.float32, "g_gu")
    _need(g_dn, torch.float32, "g_dn")
    _need(shared_gu, torch.bfloat16, "shared_gu")
    _need(shared_dn, torch.bfloat16, "shared_dn")
    T, H = x.shape
    E, twoI, _ = w_gu.shape
    I, Is = twoI // 2, shared_gu.shape[0] // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty((moe_nvfp4_layer_workspace_size(T, H, I, E, K, Is),),
                                dtype=torch.uint8, device=x.device)
        workspace[:WORKSPACE_ZERO_BYTES].zero_()
    _check(_lib().moe_nvfp4_layer(
        _ptr(x), _ptr(router_logits), T, H, I, E, K, _ptr(w_gu), _ptr(s_gu), _ptr(g_gu),
        _ptr(w_dn), _ptr(s_dn), _ptr(g_dn), _ptr(shared_gu), _ptr(shared_dn), Is, _ptr(out),
        _ptr(ids_out), _ptr(w_out), _ptr(workspace), workspace.numel(), int(path),
        _stream(x.device)))
    return out


def nvfp4_w4a4_prepare_scales(scales: torch.Tensor, gate_rows: int = 0, out=None):
    """A weight's E4M3 scales [n, rows, cols/16] rearranged into the block-scaled tensor
    cores' layout (see include/nvfp4_moe.h); gate_rows = I for a fused gate/up weight."""
    _need(scales, torch.uint8, "scales")
    n, rows, c16 = scales.shape
    if out is None:
        out = torch.empty_like(scales)
    _need(out, torch.uint8, "out")
    _check(_lib().nvfp4_w4a4_prepare_scales(_ptr(scales), n, rows, c16 * 16, int(gate_rows),
                                            _ptr(out), _stream(scales.device)))
    return out


def moe_nvfp4_w4a4_workspace_size(T, H, I, E, K) -> int:
    return int(_lib().moe_nvfp4_w4a4_workspace_size(T, H, I, E, K))


def moe_nvfp4_forward_w4a4(x, topk_ids, topk_w, w_gu, sf_gu, g_gu, w_dn, sf_dn, g_dn,
                           out=None, workspace=None) -> torch.Tensor:
    """The routed layer on the FP4 tensor cores with NVFP4 activations (W4A4); sf_gu / sf_dn
    are the prepared scales.  Returns out bf16 [T, H]."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_w, torch.float32, "topk_w")
    for t, n in ((w_gu, "w_gu"), (sf_gu, "sf_gu"), (w_dn, "w_dn"), (sf_dn, "sf_dn")):
        _need(t, torch.uint8, n)
    _need(g_gu, torch.float32, "g_gu")
    _need(g_dn, torch.float32, "g_dn")
    T, H = x.shape
    K = topk_ids.shape[1]
    E, twoI, _ = w_gu.shape
    I = twoI // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty((moe_nvfp4_w4a4_workspace_size(T, H, I, E, K),),
                                dtype=torch.uint8, device=x.device)
        workspace[:WORKSPACE_ZERO_BYTES].zero_()
    _check(_lib().moe_nvfp4_forward_w4a4(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, H, I, E, K, _ptr(w_gu), _ptr(sf_gu),
        _ptr(g_gu), _ptr(w_dn), _ptr(sf_dn), _ptr(g_dn), _ptr(out), _ptr(workspace),
        workspace.numel(), _stream(x.device)))
    return out


def moe_nvfp4_forward_w4a4_profiled(x, topk_ids, topk_w, w_gu, sf_gu, g_gu, w_dn, sf_dn, g_dn,
                                    out, workspace, stage_events):
    """moe_nvfp4_forward_w4a4 with five torch.cuda.Event recorded between its stages."""
    T, H = x.shape
    K = topk_ids.shape[1]
    E, twoI, _ = w_gu.shape
    arr = (ctypes.c_void_p * 5)(*[ctypes.c_void_p(e.cuda_event) for e in stage_events])
    _check(_lib().moe_nvfp4_forward_w4a4_profiled(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, H, twoI // 2, E, K, _ptr(w_gu), _ptr(sf_gu),
        _ptr(g_gu), _ptr(w_dn), _ptr(sf_dn), _ptr(g_dn), _ptr(out), _ptr(workspace),
        workspace.numel(), arr, _stream(x.device)))
    return out


def moe_nvfp4_ep_local_experts(E: int, ep_size: int, ep_rank: int) -> int:
    """Experts rank ep_rank of ep_size owns (those e < E with e % ep_size == ep_rank)."""
    return int(_lib().moe_nvfp4_ep_local_experts(E, ep_size, ep_rank))


def moe_nvfp4_forward_ep(x, topk_ids, topk_w, E: int, ep_size: int, ep_rank: int,
                         w_gu, s_gu, g_gu, w_dn, s_dn, g_dn, out=None, workspace=None,
                         path: int = PATH_AUTO) -> torch.Tensor:
    """This rank's experts only (expert-parallel forward; see include/nvfp4_moe.h).

    topk_ids hold global ids in [0, E); the weight tensors hold this rank's experts,
    local index l = expert l * ep_size + ep_rank.  Returns the fp32 partial [T,H]."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_w, torch.float32, "topk_w")
    for t, n in ((w_gu, "w_gu"), (s_gu, "s_gu"), (w_dn, "w_dn"), (s_dn, "s_dn")):
        _need(t, torch.uint8, n)
    _need(g_gu, torch.float32, "g_gu")
    _need(g_dn, torch.float32, "g_dn")
    T, H = x.shape
    K = topk_ids.shape[1]
    E_loc, twoI, _ = w_gu.shape
    if E_loc != moe_nvfp4_ep_local_experts(E, ep_size, ep_rank):
        raise ValueError(f"w_gu holds {E_loc} experts; rank {ep_rank} of {ep_size} owns "
                         f"{moe_nvfp4_ep_local_experts(E, ep_size, ep_rank)} of {E}")
    I = twoI // 2
    if out is None:
        out = torch.empty((T, H), dtype=torch.float32, device=x.device)
    _need(out, torch.float32, "out")
    if workspace is None:
        workspace = alloc_moe_workspace(T, H, I, E_loc, K, x.device)
    _check(_lib().moe_nvfp4_forward_ep(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, H, I, E, K, ep_size, ep_rank, _ptr(w_gu),
        _ptr(s_gu), _ptr(g_gu), _ptr(w_dn), _ptr(s_dn), _ptr(g_dn), _ptr(out),
        _ptr(workspace), workspace.numel(), int(path), _stream(x.device)))
    return out


def moe_nvfp4_ep_reduce(partials, out=None) -> torch.Tensor:
    """bf16(partials[0] + partials[1] + ...) in fp32, in list order.  partials: fp32
    [rows, cols] CUDA tensors (this device's, or peer memory it can read)."""
    partials = list(partials)
    if not partials:
        raise ValueError("partials: at least one tensor")
    for j, p in enumerate(partials):
        _need(p, torch.float32, f"partials[{j}]")
        if p.shape != partials[0].shape or p.dim() != 2:
            raise ValueError("partials: fp32 tensors of one [rows, cols] shape")
    rows, cols = partials[0].shape
    dev = partials[0].device
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    _need(out, torch.bfloat16, "out")
    arr = (ctypes.c_void_p * len(partials))(*[p.data_ptr() for p in partials])
    _check(_lib().moe_nvfp4_ep_reduce(arr, len(partials), rows, cols, _ptr(out),
                                      _stream(dev)))
    return out


def moe_nvfp4_forward_profiled(x, topk_ids, topk_w, w_gu, s_gu, g_gu, w_dn, s_dn, g_dn,
                               out, workspace, stage_events, path: int = PATH_AUTO):
    """moe_nvfp4_forward with five torch.cuda.Event (enable_timing=True) recorded around
    the stages: before route, after route, after gate/up, after down, after combine."""
    T, H = x.shape
    K = topk_ids.shape[1]
    E, twoI, _ = w_gu.shape
    evs = [ctypes.c_void_p(e.cuda_event) for e in stage_events]
    arr = (ctypes.c_void_p * 5)(*evs)
    _check(_lib().moe_nvfp4_forward_profiled(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, H, twoI // 2, E, K, _ptr(w_gu), _ptr(s_gu),
        _ptr(g_gu), _ptr(w_dn), _ptr(s_dn), _ptr(g_dn), _ptr(out), _ptr(workspace),
        workspace.numel(), int(path), arr, _stream(x.device)))
    return out


def moe_nvfp4_forward_static(x, topk_ids, topk_w, w_gu, s_gu, g_gu, w_dn, s_dn, g_dn,
                             out=None, error_flag=None) -> torch.Tensor:
    """The small-batch forward with the library's fixed scratch instead of a workspace
    (see include/nvfp4_moe.h).  error_flag: optional int32 [1] device tensor that
    receives the error bits.  Returns out bf16 [T,H]."""
    _need(x, torch.bfloat16, "x")
    _need(topk_ids, torch.int32, "topk_ids")
    _need(topk_w, torch.float32, "topk_w")
    for t, n in ((w_gu, "w_gu"), (s_gu, "s_gu"), (w_dn, "w_dn"), (s_dn, "s_dn")):
        _need(t, torch.uint8, n)
    _need(g_gu, torch.float32, "g_gu")
    _need(g_dn, torch.float32, "g_dn")
    if error_flag is not None:
        _need(error_flag, torch.int32, "error_flag")
    T, H = x.shape
    K = topk_ids.shape[1]
    E, twoI, _ = w_gu.shape
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(_lib().moe_nvfp4_forward_static(
        _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, H, twoI // 2, E, K, _ptr(w_gu), _ptr(s_gu),
        _ptr(g_gu), _ptr(w_dn), _ptr(s_dn), _ptr(g_dn), _ptr(out),
        _ptr(error_flag) if error_flag is not None else None, _stream(x.device)))
    return out


# ------------------------------------------------------------------------------ dense operators
# None of these calls is recorded by autograd, also where an input requires a gradient (as all
# calls of this module): a training step calls the *_backward functions, for instance from a
# torch.autograd.Function of its own.
# One token's call is shorter on the GPU than in Python, so these helpers do little: the raw
# stream handle instead of a Stream object (2 us less a call), one attribute test each.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",   # absent without CUDA
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _arg(t, dtype, shape, dev: int, name: str):
    """Address of a contiguous tensor of this type and shape on CUDA device `dev`."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0 \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on "
                     + (f"cuda:{dev}" if dev >= 0 else "a CUDA device"))


def _optional(t, dtype, shape, dev: int, name: str):
    return None if t is None else _arg(t, dtype, shape, dev, name)


def _out(t, like, dtype, shape, dev: int, name: str):
    """(`t`, or a new tensor beside `like`; its address)."""
    if t is None:
        t = torch.empty(*shape, dtype=dtype, device=like.device)
        return t, t.data_ptr()
    return t, _arg(t, dtype, shape, dev, name)


def _twin(t, like, dev: int, name: str):
    """_out with the type and shape of `like` (empty_like is quicker than empty)."""
    if t is None:
        t = torch.empty_like(like)
        return t, t.data_ptr()
    return t, _arg(t, like.dtype, like.shape, dev, name)


def _matrix(x, dtype, name: str):
    """(rows, columns, device index, address) of a contiguous two-dimensional CUDA tensor."""
    try:
        T, H = x.shape
        dev = x.get_device()
        if x.dtype is dtype and dev >= 0 and x.is_contiguous():
            return T, H, dev, x.data_ptr()
    except (AttributeError, ValueError):
        pass
    raise ValueError(f"{name}: expected a contiguous two-dimensional CUDA tensor of {dtype}")


def _weight(w, dtype, cols: int, dev: int, name: str):
    """(rows, address) of a matrix with `cols` columns on device `dev`."""
    rows, n, where, address = _matrix(w, dtype, name)
    if n != cols or where != dev:
        raise ValueError(f"{name}: expected rows of {cols} values on cuda:{dev}")
    return rows, address


def _scratch(workspace, nbytes: int, like):
    """(workspace, its address, its bytes), allocated beside `like` when none is given."""
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 \
            or workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous torch.uint8 tensor on the inputs' "
                         "device")
    return workspace, workspace.data_ptr(), workspace.numel()


def _on(dev: int, call, *args):
    """call(*args) with CUDA device `dev` current."""
    with torch.cuda.device(dev):
        return call(*args)


def _done(status: int) -> None:
    if status:
        _check(status)


def _flag(error_flag, dev: int):
    return None if error_flag is None else _arg(error_flag, torch.int32, (1,), dev, "error_flag")


def moe_nvfp4_pre_norm(x, weight, eps: float, out=None) -> torch.Tensor:
    """weight * x / sqrt(mean(x^2) + eps) for each row of x bf16 [T, H]; weight bf16 [H]."""
    T, H, dev, px = _matrix(x, torch.bfloat16, "x")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_pre_norm, x, weight, eps, out)
    pw = _arg(weight, torch.bfloat16, (H,), dev, "weight")
    out, po = _twin(out, x, dev, "out")
    _done((_LIB or _lib()).moe_nvfp4_pre_norm(px, pw, T, H, eps, po, _raw_stream(dev)))
    return out


def moe_nvfp4_pre_norm_int8(x, weight, eps: float, codes=None, scales=None):
    """moe_nvfp4_pre_norm's rows as 8-bit codes and one scale each, for nvfp4_int8_matmul.
    Returns (codes int8 [T, H], scales fp32 [T])."""
    T, H, dev, px = _matrix(x, torch.bfloat16, "x")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_pre_norm_int8, x, weight, eps, codes, scales)
    pw = _arg(weight, torch.bfloat16, (H,), dev, "weight")
    codes, pc = _out(codes, x, torch.int8, (T, H), dev, "codes")
    scales, ps = _out(scales, x, torch.float32, (T,), dev, "scales")
    _done((_LIB or _lib()).moe_nvfp4_pre_norm_int8(px, pw, T, H, eps, pc, ps, _raw_stream(dev)))
    return codes, scales


def _gate(gate, T, H, dev):
    if gate is None:
        return None, 0, 0
    rows, cols, where, address = _matrix(gate, torch.bfloat16, "gate")
    if rows not in (1, T) or cols not in (1, H) or where != dev:
        raise ValueError(f"gate: expected a shape that broadcasts to {(T, H)}, on cuda:{dev}")
    return address, rows, cols


def moe_nvfp4_post_norm(y, weight, residual, eps: float, gate=None, residual_scale: float = 1.0,
                        next_weight=None, out=None, next_out=None):
    """out = residual_scale * residual + gate * norm(y), with the norm of moe_nvfp4_pre_norm;
    gate bf16 [1 or T, 1 or H] or None.  With next_weight [H] also the following block's
    pre-norm of out.  Returns out bf16 [T, H], or (out, next).  The gradient of next is that of
    moe_nvfp4_pre_norm at out; it reaches moe_nvfp4_post_norm_backward through dout."""
    bf = torch.bfloat16
    T, H, dev, py = _matrix(y, bf, "y")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_post_norm, y, weight, residual, eps, gate, residual_scale,
                   next_weight, out, next_out)
    pw = _arg(weight, bf, (H,), dev, "weight")
    pr = _arg(residual, bf, (T, H), dev, "residual")
    pg, rows, cols = _gate(gate, T, H, dev)
    pn = _optional(next_weight, bf, (H,), dev, "next_weight")
    if pn is None and next_out is not None:
        raise ValueError("next_out needs next_weight")
    out, po = _twin(out, y, dev, "out")
    po2 = None
    if pn is not None:
        next_out, po2 = _twin(next_out, y, dev, "next_out")
    _done((_LIB or _lib()).moe_nvfp4_post_norm(
        py, pw, pr, pg, T, H, rows, cols, eps, residual_scale, pn, po, po2, _raw_stream(dev)))
    return out if pn is None else (out, next_out)


def moe_nvfp4_norm_backward_workspace_size(T: int, H: int) -> int:
    return int(_lib().moe_nvfp4_norm_backward_workspace_size(T, H))


def moe_nvfp4_pre_norm_backward(dy, x, weight, eps: float, dskip=None, dx=None, dweight=None,
                                workspace=None):
    """Gradients of moe_nvfp4_pre_norm; dskip [T, H] (the gradient that reaches x past the
    block) is added to dx.  Returns (dx bf16 [T, H], dweight bf16 [H])."""
    bf = torch.bfloat16
    T, H, dev, px = _matrix(x, bf, "x")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_pre_norm_backward, dy, x, weight, eps, dskip, dx, dweight,
                   workspace)
    pd = _arg(dy, bf, (T, H), dev, "dy")
    pw = _arg(weight, bf, (H,), dev, "weight")
    ps = _optional(dskip, bf, (T, H), dev, "dskip")
    dx, pdx = _twin(dx, x, dev, "dx")
    dweight, pdw = _twin(dweight, weight, dev, "dweight")
    workspace, pws, nws = _scratch(workspace, _norm_scratch(T, H, dev), x)
    _done((_LIB or _lib()).moe_nvfp4_pre_norm_backward(
        pd, px, pw, ps, T, H, eps, pdx, pdw, pws, nws, _raw_stream(dev)))
    return dx, dweight


@functools.lru_cache(maxsize=256)   # a size: it depends on the arguments alone
def _norm_scratch(T, H, dev):
    return _lib().moe_nvfp4_norm_backward_workspace_size(T, H)   # of the current device, dev


def moe_nvfp4_post_norm_backward(dout, y, weight, eps: float, gate=None,
                                 residual_scale: float = 1.0, dy=None, dweight=None, dgate=None,
                                 dresidual=None, need_dresidual: bool = True, workspace=None):
    """Gradients of moe_nvfp4_post_norm's out.  Returns (dy bf16 [T, H], dweight bf16 [H],
    dgate of gate's shape or None without a gate, dresidual bf16 [T, H] or None when
    need_dresidual is false)."""
    bf = torch.bfloat16
    T, H, dev, py = _matrix(y, bf, "y")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_post_norm_backward, dout, y, weight, eps, gate, residual_scale,
                   dy, dweight, dgate, dresidual, need_dresidual, workspace)
    pd = _arg(dout, bf, (T, H), dev, "dout")
    pw = _arg(weight, bf, (H,), dev, "weight")
    pg, rows, cols = _gate(gate, T, H, dev)
    dy, pdy = _twin(dy, y, dev, "dy")
    dweight, pdw = _twin(dweight, weight, dev, "dweight")
    pdg = pdr = None
    if gate is not None:
        dgate, pdg = _twin(dgate, gate, dev, "dgate")
    elif dgate is not None:
        raise ValueError("dgate needs gate")
    if need_dresidual or dresidual is not None:
        dresidual, pdr = _twin(dresidual, y, dev, "dresidual")
    workspace, pws, nws = _scratch(workspace, _norm_scratch(T, H, dev), y)
    _done((_LIB or _lib()).moe_nvfp4_post_norm_backward(
        pd, py, pw, pg, T, H, rows, cols, eps, residual_scale, pdy, pdw, pdg, pdr, pws, nws,
        _raw_stream(dev)))
    return dy, dweight, dgate, dresidual


def _gate_up_rows(w_gu, H, dev):
    rows, address = _weight(w_gu, torch.bfloat16, H, dev, "w_gu")
    if rows % 2:
        raise ValueError("w_gu: expected gate rows and as many up rows")
    return rows // 2, address


def moe_nvfp4_gate_up(x, w_gu, act: int = ACT_SILU, h=None, gu=None,
                      error_flag=None) -> torch.Tensor:
    """h = act(x W_g^T) * (x W_u^T) in one kernel; x bf16 [T, H]; w_gu bf16 [2I, H], gate rows
    first.  gu bf16 [T, 2I], when given, receives the pre-activations that
    moe_nvfp4_gate_up_backward takes.  error_flag int32 [1], when given, gets bit 1 if a wait on
    the device gave up; what could then not be computed is NaN.  Returns h bf16 [T, I]."""
    bf = torch.bfloat16
    T, H, dev, px = _matrix(x, bf, "x")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_gate_up, x, w_gu, act, h, gu, error_flag)
    I, pw = _gate_up_rows(w_gu, H, dev)
    h, ph = _out(h, x, bf, (T, I), dev, "h")
    pgu = _optional(gu, bf, (T, 2 * I), dev, "gu")
    _done((_LIB or _lib()).moe_nvfp4_gate_up(
        px, pw, T, H, I, act, ph, pgu, _flag(error_flag, dev), _raw_stream(dev)))
    return h


def moe_nvfp4_gate_up_backward_workspace_size(T: int, I: int) -> int:
    return int(_lib().moe_nvfp4_gate_up_backward_workspace_size(T, I))


def moe_nvfp4_gate_up_backward(dh, x, w_gu, gu, act: int = ACT_SILU, dx=None, dw_gu=None,
                               need_dx: bool = True, need_dw: bool = True, workspace=None,
                               error_flag=None):
    """Gradients of moe_nvfp4_gate_up from dh bf16 [T, I] and the kept gu.  Returns
    (dx bf16 [T, H], dw_gu bf16 [2I, H]), None in the place of one that is not needed."""
    bf = torch.bfloat16
    T, H, dev, px = _matrix(x, bf, "x")
    if dev != _current_device():
        return _on(dev, moe_nvfp4_gate_up_backward, dh, x, w_gu, gu, act, dx, dw_gu, need_dx,
                   need_dw, workspace, error_flag)
    I, pw = _gate_up_rows(w_gu, H, dev)
    pd = _arg(dh, bf, (T, I), dev, "dh")
    pgu = _arg(gu, bf, (T, 2 * I), dev, "gu")
    pdx = pdw = None
    if need_dx or dx is not None:
        dx, pdx = _twin(dx, x, dev, "dx")
    if need_dw or dw_gu is not None:
        dw_gu, pdw = _twin(dw_gu, w_gu, dev, "dw_gu")
    workspace, pws, nws = _scratch(workspace, moe_nvfp4_gate_up_backward_workspace_size(T, I), x)
    _done((_LIB or _lib()).moe_nvfp4_gate_up_backward(
        pd, px, pw, pgu, T, H, I, act, pdx, pdw, pws, nws, _flag(error_flag, dev),
        _raw_stream(dev)))
    return dx, dw_gu


def nvfp4_int8_quantize(x, codes=None, scales=None):
    """Rows of x bf16 [rows, cols] -> (codes int8 [rows, cols], scales fp32 [rows]):
    scale = max |x| / 127, code = the integer nearest to x / scale.  A row with NaN or an infinity
    gets the scale NaN."""
    T, K, dev, px = _matrix(x, torch.bfloat16, "x")
    if dev != _current_device():
        return _on(dev, nvfp4_int8_quantize, x, codes, scales)
    codes, pc = _out(codes, x, torch.int8, (T, K), dev, "codes")
    scales, ps = _out(scales, x, torch.float32, (T,), dev, "scales")
    _done((_LIB or _lib()).nvfp4_int8_quantize(px, T, K, pc, ps, _raw_stream(dev)))
    return codes, scales


def nvfp4_int8_matmul(a, a_scales, w, w_scales, out=None, error_flag=None) -> torch.Tensor:
    """bf16 [T, N] = (a [T, K] int8 times w [N, K] int8 transposed, exact) scaled by a_scales
    fp32 [T] and w_scales fp32 [N]."""
    T, K, dev, pa = _matrix(a, torch.int8, "a")
    if dev != _current_device():
        return _on(dev, nvfp4_int8_matmul, a, a_scales, w, w_scales, out, error_flag)
    N, pw = _weight(w, torch.int8, K, dev, "w")
    pas = _arg(a_scales, torch.float32, (T,), dev, "a_scales")
    pws = _arg(w_scales, torch.float32, (N,), dev, "w_scales")
    out, po = _out(out, a, torch.bfloat16, (T, N), dev, "out")
    _done((_LIB or _lib()).nvfp4_int8_matmul(
        pa, pas, pw, pws, T, N, K, po, _flag(error_flag, dev), _raw_stream(dev)))
    return out


def nvfp4_selftest_wait_timeout(flag: torch.Tensor, kind: int, limit_ns: int) -> None:
    """Test hook: one kernel waits for something nothing completes (kind 0: an mbarrier
    phase, 1: bulk-copy bytes, 2: a global counter) with a limit of limit_ns; the wait
    runs out and bit 1 is ORed into flag's first int32 (device tensor, e.g. a forward
    workspace)."""
    if not isinstance(flag, torch.Tensor) or not flag.is_cuda:
        raise ValueError("flag: expected a CUDA tensor")
    _check(_lib().nvfp4_selftest_wait_timeout(_ptr(flag), int(kind), int(limit_ns),
                                              _stream(flag.device)))


def nvfp4_selftest_gate_up_timeout(x, w_gu, h, gu, error_flag) -> None:
    """Test hook: moe_nvfp4_gate_up (SiLU) with loads that never come and waits of 2 ms; bit 1 of
    error_flag is set and h and gu (or None) are NaN where they could not be computed."""
    bf = torch.bfloat16
    T, H, dev, px = _matrix(x, bf, "x")
    I, pw = _gate_up_rows(w_gu, H, dev)
    ph, pgu = _arg(h, bf, (T, I), dev, "h"), _optional(gu, bf, (T, 2 * I), dev, "gu")
    _check(_lib().nvfp4_selftest_gate_up_timeout(px, pw, T, H, I, ph, pgu, _flag(error_flag, dev),
                                                 _stream(x.device)))


def nvfp4_selftest_int8_matmul_timeout(a, a_scales, w, w_scales, out, error_flag) -> None:
    """Test hook: nvfp4_int8_matmul in the same way."""
    T, K, dev, pa = _matrix(a, torch.int8, "a")
    N, pw = _weight(w, torch.int8, K, dev, "w")
    pas = _arg(a_scales, torch.float32, (T,), dev, "a_scales")
    pws = _arg(w_scales, torch.float32, (N,), dev, "w_scales")
    po = _arg(out, torch.bfloat16, (T, N), dev, "out")
    _check(_lib().nvfp4_selftest_int8_matmul_timeout(pa, pas, pw, pws, T, N, K, po,
                                                     _flag(error_flag, dev), _stream(a.device)))


def moe_nvfp4_read_error_flag(workspace: torch.Tensor) -> int:
    """Error bits of the last forward on this workspace (1 = id out of range,
    2 = a device wait gave up).  Synchronises the current stream."""
    flag = ctypes.c_int32(0)
    _check(_lib().moe_nvfp4_read_error_flag(_ptr(workspace), ctypes.byref(flag),
                                         _stream(workspace.device)))
    return int(flag.value)

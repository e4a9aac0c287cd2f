"""ctypes binding of libw4a4moe (include/w4a4_moe.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  Loading
fails loudly when the library has not been built.
"""
import ctypes
import functools
import json
import os

import torch

from . import build as _build

_lib = None

c_i64, c_int, c_sz, c_vp = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p

_SIGS = {
    "w4a4_rows_capacity": (c_i64, [c_i64, c_int, c_int, c_int]),
    "w4a4_workspace_size": (c_sz, [c_int, c_i64, c_int, c_int, c_int, c_int, c_int]),
    "w4a4_quantize_permute": (c_int, [c_vp, c_i64, c_int, c_vp, c_int, c_int, c_int,
                                      c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_grouped_expert_fwd": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                        c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                        c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                        c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                        c_vp, c_sz, c_vp]),
    "w4a4_grouped_expert_fwd_ckpt": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                             c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                             c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                             c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_mx_grouped_expert_fwd_ckpt": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                                c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                                c_vp, c_vp, c_vp, c_vp,
                                                c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_expert_bwd": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_expert_bwd_ckpt": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                     c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                     c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_quantize_permute_domain": (c_int, [c_vp, c_i64, c_int, c_vp, c_int, c_int, c_int, c_i64,
                                             c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_linear_fwd": (c_int, [c_i64, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                c_vp, c_vp]),
    "w4a4_linear_bwd": (c_int, [c_i64, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                c_vp, c_sz, c_vp]),
    "w4a4_mx_quantize_permute": (c_int, [c_vp, c_i64, c_int, c_vp, c_int, c_int, c_int,
                                         c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_mx_grouped_expert_fwd": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                           c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                           c_vp, c_vp, c_vp, c_vp,
                                           c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                           c_vp, c_sz, c_vp]),
    "w4a4_mx8_expert_bwd": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int,
                                    c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                    c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_mx8_quantize": (c_int, [c_vp, c_i64, c_int, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp]),
    "w4a4_mx_quantize_rows": (c_int, [c_i64, c_int, c_int, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp]),
    "w4a4_add_rmsnorm_fwd": (c_int, [c_i64, c_int, ctypes.c_float, c_vp, c_i64, c_vp, c_int, c_vp, c_int,
                                     c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "w4a4_add_rmsnorm_bwd": (c_int, [c_i64, c_int, c_vp, c_vp, c_int, c_vp, c_int, c_vp, c_vp,
                                     c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_mx_linear_fwd": (c_int, [c_i64, c_int, c_int, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp]),
    "w4a4_permute_fwd": (c_int, [c_i64, c_int, c_int, c_int, c_int, c_int, c_vp, c_i64, c_vp,
                                 c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
    "w4a4_permute_bwd": (c_int, [c_i64, c_int, c_int, c_i64, c_int, c_vp, c_vp, c_vp, c_i64, c_vp]),
    "w4a4_unpermute_fwd": (c_int, [c_i64, c_int, c_int, c_i64, c_int, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp]),
    "w4a4_unpermute_bwd": (c_int, [c_i64, c_int, c_int, c_int, c_i64, c_int, c_vp, c_i64, c_vp, c_vp, c_vp,
                                   c_vp, c_vp, c_vp, c_vp, c_vp]),
    "w4a4_swiglu_fwd": (c_int, [c_i64, c_int, c_vp, c_i64, c_vp, c_int, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "w4a4_swiglu_bwd": (c_int, [c_i64, c_int, c_vp, c_vp, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "w4a4_check_routing": (c_int, [c_vp, c_i64, c_int, c_int, c_vp, c_vp]),
    "w4a4_quantize_permute_noalloc": (c_int, [c_vp, c_i64, c_int, c_vp, c_int, c_int, c_int,
                                              c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]),
    "w4a4_status_string": (ctypes.c_char_p, [c_int]),
    "w4a4_last_error": (ctypes.c_char_p, []),
    "w4a4_profiler_enable": (c_int, [c_int]),
    "w4a4_profiler_report": (c_int, [ctypes.c_char_p, c_sz]),
}

WS_QUANTIZE_PERMUTE, WS_FORWARD, WS_BACKWARD, WS_LINEAR_BACKWARD = 0, 1, 2, 3
WS_QUANTIZE_PERMUTE_DOMAIN = 4
WS_MX8_BACKWARD = 5
WS_RMSNORM_BACKWARD = 6
WS_PERMUTE = 8
WS_BACKWARD_CKPT = 9

# Element formats of the MX calls (w4a4_mx_format) and types (w4a4_dtype)
MX_NONE, MX_FP4, MX_FP8 = -1, 0, 1
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


class W4A4Error(RuntimeError):
    pass


def lib_path():
    return _build.LIB


def load():
    """Load the built library (no build here: build with ``precision_rl_amd.build``)."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise W4A4Error(f"HIP library not built: {path} is missing "
                            "(run `python -m precision_rl_amd.build`)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status):
    if status != 0:
        lib = load()
        raise W4A4Error(f"{lib.w4a4_status_string(status).decode()} ({status}): "
                        f"{lib.w4a4_last_error().decode()}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def rows_capacity(T, k, E, row_align=1):
    return int(load().w4a4_rows_capacity(T, k, E, row_align))


def workspace_size(kind, T, H, I, E, k, row_align=1):
    return int(load().w4a4_workspace_size(kind, T, H, I, E, k, row_align))


def _workspace(nbytes, device, ws=None):
    if ws is not None and ws.numel() >= nbytes:
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------- wrappers
def w4a4_quantize_permute(x, topk_idx, E, row_align=1, out=None, workspace=None):
    """Route + per-token amax + NVFP4 encode + scatter.  x: [T, K] bf16 cuda; topk_idx: [T, k] int32 or None
    (identity routing, one encoded row per input row).  Returns a dict of
    tensors: codes [cap, K/2] u8, scales [cap, K/16] u8, outer [cap] f32,
    offsets [E+1], row_map [T, k], src_row [cap] (int32)."""
    lib = load()
    T, K = x.shape
    dev = x.device
    if topk_idx is None:
        k, E, row_align = 1, 1, 1
    else:
        k = topk_idx.shape[1]
    cap = rows_capacity(T, k, E, row_align)
    if out is None:
        out = dict(
            codes=torch.empty(cap, K // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(cap, K // 16, dtype=torch.uint8, device=dev),
            outer=torch.empty(cap, dtype=torch.float32, device=dev),
            offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            row_map=torch.empty(T, k, dtype=torch.int32, device=dev),
            src_row=torch.empty(cap, dtype=torch.int32, device=dev))
    need = workspace_size(WS_QUANTIZE_PERMUTE, T, K, 0, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_quantize_permute(
        _p(x), T, K, _p(topk_idx), k, E, row_align,
        _p(out["codes"]), _p(out["scales"]), _p(out["outer"]), _p(out["offsets"]),
        _p(out["row_map"]), _p(out["src_row"]), _p(ws), ws.numel(), _stream()))
    return out


def w4a4_quantize_permute_domain(x, topk_idx, E, row_align=1, group_rows=1, out=None, workspace=None):
    """w4a4_quantize_permute with one outer scale per group of `group_rows` consecutive
    input rows (T: per tensor).  Same outputs."""
    lib = load()
    T, K = x.shape
    dev = x.device
    if topk_idx is None:
        k, E, row_align = 1, 1, 1
    else:
        k = topk_idx.shape[1]
    cap = rows_capacity(T, k, E, row_align)
    if out is None:
        out = dict(
            codes=torch.empty(cap, K // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(cap, K // 16, dtype=torch.uint8, device=dev),
            outer=torch.empty(cap, dtype=torch.float32, device=dev),
            offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            row_map=torch.empty(T, k, dtype=torch.int32, device=dev),
            src_row=torch.empty(cap, dtype=torch.int32, device=dev))
    need = workspace_size(WS_QUANTIZE_PERMUTE_DOMAIN, T, K, 0, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_quantize_permute_domain(
        _p(x), T, K, _p(topk_idx), k, E, row_align, group_rows,
        _p(out["codes"]), _p(out["scales"]), _p(out["outer"]), _p(out["offsets"]),
        _p(out["row_map"]), _p(out["src_row"]), _p(ws), ws.numel(), _stream()))
    return out


def w4a4_quantize_permute_noalloc(x, topk_idx, E, row_align=1, out=None):
    """w4a4_quantize_permute without a workspace (the library's per-GPU scratch holds
    the routing counts).  `out`: preallocated outputs as w4a4_quantize_permute returns
    them (allocated here when None)."""
    lib = load()
    T, K = x.shape
    dev = x.device
    if topk_idx is None:
        k, E, row_align = 1, 1, 1
    else:
        k = topk_idx.shape[1]
    cap = rows_capacity(T, k, E, row_align)
    if out is None:
        out = dict(
            codes=torch.empty(cap, K // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(cap, K // 16, dtype=torch.uint8, device=dev),
            outer=torch.empty(cap, dtype=torch.float32, device=dev),
            offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            row_map=torch.empty(T, k, dtype=torch.int32, device=dev),
            src_row=torch.empty(cap, dtype=torch.int32, device=dev))
    _check(lib.w4a4_quantize_permute_noalloc(
        _p(x), T, K, _p(topk_idx), k, E, row_align,
        _p(out["codes"]), _p(out["scales"]), _p(out["outer"]), _p(out["offsets"]),
        _p(out["row_map"]), _p(out["src_row"]), _stream()))
    return out


def w4a4_check_routing(topk_idx, E, out=None):
    """Routing validity of topk_idx [T, k] int32 cuda.  Returns an int32 [2] device
    tensor: (number of invalid entries, smallest flat index of one or INT32_MAX)."""
    lib = load()
    T, k = topk_idx.shape
    if out is None:
        out = torch.empty(2, dtype=torch.int32, device=topk_idx.device)
    _check(lib.w4a4_check_routing(_p(topk_idx), T, k, E, _p(out), _stream()))
    return out


def quantize_weights(w, per_expert=False):
    """NVFP4 of stacked expert weights w [E, N, K] bf16 (offline, identity routing): one
    outer scale per row, or per expert weight tensor with `per_expert`.
    Returns dict(codes [E, N, K/2], scales [E, N, K/16], outer [E, N])."""
    E, N, K = w.shape
    if per_expert:
        q = w4a4_quantize_permute_domain(w.reshape(E * N, K), None, 1, group_rows=N)
    else:
        q = w4a4_quantize_permute(w.reshape(E * N, K), None, 1)
    return dict(codes=q["codes"].view(E, N, K // 2), scales=q["scales"].view(E, N, K // 16),
                outer=q["outer"].view(E, N))


def w4a4_grouped_expert_fwd(xq, topk_w, w1q, w2q, T, H, I, E, k, row_align=1,
                            save=False, debug=False, y=None, workspace=None, saved=None):
    """Grouped expert forward: FC1 -> SwiGLU -> requantise -> FC2 -> unpermute.  xq: result of ``w4a4_quantize_permute``; w1q / w2q: results
    of ``quantize_weights``.  Returns dict(y, and h/a when ``save``, and the
    FC1 pre-cast values plus the FC2-input encoding when ``debug``)."""
    lib = load()
    dev = xq["codes"].device
    cap = rows_capacity(T, k, E, row_align)
    res = {}
    res["y"] = y if y is not None else torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if save:
        if saved is None:
            saved = dict(h=torch.empty(cap, 2 * I, dtype=torch.bfloat16, device=dev),
                         a=torch.empty(cap, I, dtype=torch.bfloat16, device=dev))
        res.update(saved)
    if debug:
        res["fc1_f32"] = torch.empty(cap, 2 * I, dtype=torch.float32, device=dev)
        res["a_codes"] = torch.empty(cap, I // 2, dtype=torch.uint8, device=dev)
        res["a_scales"] = torch.empty(cap, I // 16, dtype=torch.uint8, device=dev)
        res["a_outer"] = torch.empty(cap, dtype=torch.float32, device=dev)
    need = workspace_size(WS_FORWARD, T, H, I, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_grouped_expert_fwd(
        T, H, I, E, k, row_align,
        _p(xq["codes"]), _p(xq["scales"]), _p(xq["outer"]),
        _p(xq["offsets"]), _p(xq["row_map"]), _p(xq["src_row"]), _p(topk_w),
        _p(w1q["codes"]), _p(w1q["scales"]), _p(w1q["outer"]),
        _p(w2q["codes"]), _p(w2q["scales"]), _p(w2q["outer"]),
        _p(res["y"]), _p(res.get("h")), _p(res.get("a")), _p(res.get("fc1_f32")),
        _p(res.get("a_codes")), _p(res.get("a_scales")), _p(res.get("a_outer")),
        _p(ws), ws.numel(), _stream()))
    return res


def w4a4_expert_bwd(dy, x, w1, w2, h, a, topk_w, xq, T, H, I, E, k, row_align=1,
                    out=None, workspace=None):
    """Straight-through BF16 backward.  Returns dict(dx [T, H], dw1 [E, 2I, H], dw2 [E, H, I]) bf16."""
    lib = load()
    dev = dy.device
    if out is None:
        out = dict(dx=torch.empty(T, H, dtype=torch.bfloat16, device=dev),
                   dw1=torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device=dev),
                   dw2=torch.empty(E, H, I, dtype=torch.bfloat16, device=dev))
    need = workspace_size(WS_BACKWARD, T, H, I, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_expert_bwd(
        T, H, I, E, k, row_align, _p(dy), _p(x), _p(w1), _p(w2), _p(h), _p(a), _p(topk_w),
        _p(xq["offsets"]), _p(xq["row_map"]), _p(xq["src_row"]),
        _p(out["dx"]), _p(out["dw1"]), _p(out["dw2"]), _p(ws), ws.numel(), _stream()))
    return out


def w4a4_mx8_expert_bwd(dy, x, w1, w2, h, a, topk_w, xq, T, H, I, E, k, row_align=128,
                        out=None, workspace=None):
    """Straight-through backward with MXFP8 GEMM operands (row_align 128).
    Returns dict(dx [T, H], dw1 [E, 2I, H], dw2 [E, H, I]) bf16."""
    lib = load()
    dev = dy.device
    if out is None:
        out = dict(dx=torch.empty(T, H, dtype=torch.bfloat16, device=dev),
                   dw1=torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device=dev),
                   dw2=torch.empty(E, H, I, dtype=torch.bfloat16, device=dev))
    need = workspace_size(WS_MX8_BACKWARD, T, H, I, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_mx8_expert_bwd(
        T, H, I, E, k, row_align, _p(dy), _p(x), _p(w1), _p(w2), _p(h), _p(a), _p(topk_w),
        _p(xq["offsets"]), _p(xq["row_map"]), _p(xq["src_row"]),
        _p(out["dx"]), _p(out["dw1"]), _p(out["dw2"]), _p(ws), ws.numel(), _stream()))
    return out


def w4a4_mx8_quantize(x):
    """MXFP8 (E4M3 + E8M0 per 32) of x [R, C] bf16 along rows and along columns.
    Returns dict(q_rows [R, C], s_rows [R, C/32], q_cols [C, R], s_cols [C, R/32]) uint8."""
    lib = load()
    R, C = x.shape
    dev = x.device
    pitch = (R + 127) // 128 * 128
    out = dict(q_rows=torch.empty(R, C, dtype=torch.uint8, device=dev),
               s_rows=torch.empty(R, C // 32, dtype=torch.uint8, device=dev),
               q_cols=torch.empty(C, pitch, dtype=torch.uint8, device=dev),
               s_cols=torch.empty(C, pitch // 32, dtype=torch.uint8, device=dev))
    _check(lib.w4a4_mx8_quantize(_p(x), R, C, _p(out["q_rows"]), _p(out["s_rows"]), _p(out["q_cols"]),
                                 _p(out["s_cols"]), pitch, _stream()))
    out["q_cols"] = out["q_cols"][:, :R]
    out["s_cols"] = out["s_cols"][:, :R // 32]
    return out


def w4a4_linear_fwd(xq, wq, T, K, N, y=None):
    """Dense per-token NVFP4 linear layer y = x W^T.  xq: w4a4_quantize_permute(x, None, 1)
    of x [T, K]; wq: the same of W [N, K].  Returns y [T, N] bf16."""
    lib = load()
    dev = wq["codes"].device
    if y is None:
        y = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    _check(lib.w4a4_linear_fwd(T, K, N, _p(xq["codes"]), _p(xq["scales"]), _p(xq["outer"]),
                               _p(xq["offsets"]), _p(wq["codes"]), _p(wq["scales"]),
                               _p(wq["outer"]), _p(y), _stream()))
    return y


def w4a4_linear_bwd(dy, x, w, xq, T, K, N, out=None, workspace=None):
    """Straight-through BF16 backward of w4a4_linear_fwd.  Returns dict(dx [T, K], dw [N, K]) bf16."""
    lib = load()
    dev = w.device
    if out is None:
        out = dict(dx=torch.empty(T, K, dtype=torch.bfloat16, device=dev),
                   dw=torch.empty(N, K, dtype=torch.bfloat16, device=dev))
    ws = _workspace(workspace_size(WS_LINEAR_BACKWARD, 0, K, N, 1, 1), dev, workspace)
    _check(lib.w4a4_linear_bwd(T, K, N, _p(dy), _p(x), _p(w), _p(xq["offsets"]),
                               _p(out["dx"]), _p(out["dw"]), _p(ws), ws.numel(), _stream()))
    return out


# ------------------------------------------------------------ MXFP4 recipe
def w4a4_mx_quantize_permute(x, topk_idx, E, row_align=1, out=None, workspace=None):
    """Route + MXFP4 encode (E2M1, one E8M0 scale per 32) + scatter.  x: [T, K] bf16 cuda,
    K % 32 == 0; topk_idx: [T, k] int32 or None (identity routing).  Returns a dict:
    codes [cap, K/2] u8, scales [cap, K/32] u8, offsets [E+1], row_map [T, k], src_row [cap]."""
    lib = load()
    T, K = x.shape
    dev = x.device
    if topk_idx is None:
        k, E, row_align = 1, 1, 1
    else:
        k = topk_idx.shape[1]
    cap = rows_capacity(T, k, E, row_align)
    if out is None:
        out = dict(
            codes=torch.empty(cap, K // 2, dtype=torch.uint8, device=dev),
            scales=torch.empty(cap, K // 32, dtype=torch.uint8, device=dev),
            offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            row_map=torch.empty(T, k, dtype=torch.int32, device=dev),
            src_row=torch.empty(cap, dtype=torch.int32, device=dev))
    need = workspace_size(WS_QUANTIZE_PERMUTE, T, K, 0, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_mx_quantize_permute(
        _p(x), T, K, _p(topk_idx), k, E, row_align, _p(out["codes"]), _p(out["scales"]),
        _p(out["offsets"]), _p(out["row_map"]), _p(out["src_row"]), _p(ws), ws.numel(), _stream()))
    return out


def quantize_weights_mx(w):
    """MXFP4 of stacked expert weights w [E, N, K] bf16 along K (offline, identity routing).
    Returns dict(codes [E, N, K/2], scales [E, N, K/32])."""
    E, N, K = w.shape
    q = w4a4_mx_quantize_permute(w.reshape(E * N, K), None, 1)
    return dict(codes=q["codes"].view(E, N, K // 2), scales=q["scales"].view(E, N, K // 32))


def w4a4_mx_grouped_expert_fwd(xq, topk_w, w1q, w2q, T, H, I, E, k, row_align=1,
                               save=False, debug=False, y=None, workspace=None, saved=None):
    """MXFP4 grouped expert forward: FC1 -> SwiGLU -> requantise -> FC2 -> unpermute on the
    scaled FP4 MFMA.  xq: result of ``w4a4_mx_quantize_permute``; w1q / w2q: of
    ``quantize_weights_mx``.  Returns dict(y, h/a when ``save``, fc1_f32 and the FC2-input
    encoding a_codes / a_scales when ``debug``)."""
    lib = load()
    dev = xq["codes"].device
    cap = rows_capacity(T, k, E, row_align)
    res = {}
    res["y"] = y if y is not None else torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if save:
        if saved is None:
            saved = dict(h=torch.empty(cap, 2 * I, dtype=torch.bfloat16, device=dev),
                         a=torch.empty(cap, I, dtype=torch.bfloat16, device=dev))
        res.update(saved)
    if debug:
        res["fc1_f32"] = torch.empty(cap, 2 * I, dtype=torch.float32, device=dev)
        res["a_codes"] = torch.empty(cap, I // 2, dtype=torch.uint8, device=dev)
        res["a_scales"] = torch.empty(cap, I // 32, dtype=torch.uint8, device=dev)
    need = workspace_size(WS_FORWARD, T, H, I, E, k, row_align)
    ws = _workspace(need, dev, workspace)
    _check(lib.w4a4_mx_grouped_expert_fwd(
        T, H, I, E, k, row_align, _p(xq["codes"]), _p(xq["scales"]),
        _p(xq["offsets"]), _p(xq["row_map"]), _p(xq["src_row"]), _p(topk_w),
        _p(w1q["codes"]), _p(w1q["scales"]), _p(w2q["codes"]), _p(w2q["scales"]),
        _p(res["y"]), _p(res.get("h")), _p(res.get("a")), _p(res.get("fc1_f32")),
        _p(res.get("a_codes")), _p(res.get("a_scales")), _p(ws), ws.numel(), _stream()))
    return res


# ------------------------------------------ pre-norm and the dense MX product
# These calls launch on the current stream of their tensors' device (which is
# made current for the call), and check types, shapes and layouts.
def _ptr(t, name, shape, dtype, device, rows=False):
    """Address of t (None: no tensor).  A dense tensor, or with `rows` one whose rows may be
    further apart."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device.index:
        raise W4A4Error(f"{name}: {dtype} {tuple(shape)} on {device} expected, "
                        f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    if not t.is_contiguous() and not (rows and (t.stride(1) == 1 or t.shape[0] == 0)):
        raise W4A4Error(f"{name} is not {'row-contiguous' if rows else 'contiguous'}")
    return t.data_ptr()


def _matrix(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda or (dtype and t.dtype != dtype):
        raise W4A4Error(f"{name} must be a 2-d {dtype or ''} tensor on the GPU")
    return t.shape, t.device


def _pitch(t):
    """Elements between the rows of t (one row has no other pitch than its own length)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _dtype(t, name):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise W4A4Error(f"{name} must be bfloat16 or float32, got {t.dtype}") from None


# The handle of a device's current stream, without building the Stream object that
# torch.cuda.current_stream returns (1.8 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

# The current device, without torch.cuda.current_device's look whether the GPU is initialised:
# a tensor lies on it here.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, device, *args):
    stream = _raw_stream(device.index)
    if device.index == _current_device():
        _check(fn(*args, stream))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, stream))


def _code_shape(T, K, fmt):
    if fmt not in (MX_FP4, MX_FP8):
        raise W4A4Error(f"format {fmt} is neither MX_FP4 nor MX_FP8")
    return (T, K // 2) if fmt == MX_FP4 else (T, K)


def _mx_buffers(out, T, K, fmt, device):
    """The code and scale buffers of `out`, allocated where it has none, and their addresses."""
    cs, ss = _code_shape(T, K, fmt), (T, K // 32)
    codes, scales = out.get("codes"), out.get("scales")
    if codes is None:
        codes = out["codes"] = torch.empty(cs, dtype=torch.uint8, device=device)
    if scales is None:
        scales = out["scales"] = torch.empty(ss, dtype=torch.uint8, device=device)
    return (_ptr(codes, "codes", cs, torch.uint8, device), _ptr(scales, "scales", ss, torch.uint8, device))


def _check_workspace(ws, nbytes, index):
    """A caller's workspace: enough dense bytes on device `index`, or an error (one that is too small
    is not replaced, which a program that captures a graph would not notice)."""
    if ws.dtype is not torch.uint8 or ws.get_device() != index or not ws.is_contiguous() or ws.numel() < nbytes:
        raise W4A4Error(f"workspace: {nbytes} contiguous bytes (torch.uint8) on device {index} expected, "
                        f"got {ws.dtype} {tuple(ws.shape)} with strides {ws.stride()} on {ws.device}")


def w4a4_mx_quantize_rows(x, fmt, out=None):
    """MXFP4 (fmt MX_FP4) or MXFP8 (MX_FP8) of the rows of x [T, K] bf16 (K % 32 == 0; a column slice
    of a wider matrix will do).  Returns a dict: codes [T, K/2] or [T, K] u8, scales [T, K/32] u8
    (the tensors of `out` where given).  An `offsets` tensor ([2] int32) in `out` receives {0, T}
    for ``w4a4_linear_bwd``."""
    (T, K), dev = _matrix(x, "x", torch.bfloat16)
    res = {} if out is None else dict(out)
    codes, scales = _mx_buffers(res, T, K, fmt, dev)
    _call(load().w4a4_mx_quantize_rows, dev, T, K, fmt, _ptr(x, "x", x.shape, torch.bfloat16, dev, rows=True),
          _pitch(x), codes, scales, _ptr(res.get("offsets"), "offsets", (2,), torch.int32, dev))
    return res


def w4a4_add_rmsnorm_fwd(x, gamma, eps=1e-6, residual=None, fmt=None, y=True, save=False, out=None):
    """s = x + residual (rounded to the residual's type), y = bf16(s * rstd * gamma) with
    rstd = (mean s^2 + eps)^-1/2, and the MX encoding of y.

    x [T, H] bf16 (a column slice will do), residual [T, H] bf16 or float32 or None (s = x),
    gamma [H] bf16 or float32; fmt: None, MX_FP4 or MX_FP8; y: whether the bf16 output is wanted;
    save: whether rstd is (for the backward).  Returns a dict with what was asked for: sum (with a
    residual), y, codes and scales (with fmt), rstd.  Tensors of `out` are used where given; its
    `sum` may be the residual itself (in place), and its `offsets` ([2] int32) receives {0, T}."""
    (T, H), dev = _matrix(x, "x", torch.bfloat16)
    res = {} if out is None else dict(out)
    total = res.get("sum")
    if total is None and residual is not None:
        total = res["sum"] = torch.empty(T, H, dtype=residual.dtype, device=dev)
    stream = residual if residual is not None else total if total is not None else x
    rt = _dtype(stream, "residual")
    if y and res.get("y") is None:
        res["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    if save and res.get("rstd") is None:
        res["rstd"] = torch.empty(T, dtype=torch.float32, device=dev)
    codes, scales = (None, None) if fmt is None else _mx_buffers(res, T, H, fmt, dev)
    _call(load().w4a4_add_rmsnorm_fwd, dev, T, H, eps, _ptr(x, "x", x.shape, torch.bfloat16, dev, rows=True),
          _pitch(x), _ptr(residual, "residual", x.shape, stream.dtype, dev), rt,
          _ptr(gamma, "gamma", (H,), gamma.dtype, dev), _dtype(gamma, "gamma"), MX_NONE if fmt is None else fmt,
          _ptr(total, "sum", x.shape, stream.dtype, dev), _ptr(res.get("y"), "y", x.shape, torch.bfloat16, dev),
          codes, scales, _ptr(res.get("rstd"), "rstd", (T,), torch.float32, dev),
          _ptr(res.get("offsets"), "offsets", (2,), torch.int32, dev))
    return res


def w4a4_add_rmsnorm_bwd(dy, sum, gamma, rstd, dsum=None, dgamma=True, out=None, workspace=None):
    """Gradients of ``w4a4_add_rmsnorm_fwd`` for dy [T, H] bf16, the gradient of y, and dsum (optional,
    the type of `sum`), the gradient that reaches the sum along the residual stream.

    sum: the forward's (its x where there was no residual), rstd: the forward's.  Returns a dict:
    dres [T, H] (the type of `sum`), the gradient of the residual and of x, and dgamma [H] float32
    unless `dgamma` is false.  Tensors of `out` are used where given; a `dx` there ([T, H] bf16)
    receives dres rounded to bf16.  workspace: at least workspace_size(WS_RMSNORM_BACKWARD, T, H, 0, 1, 1)
    bytes (uint8) where dgamma is wanted; allocated where it is not given."""
    (T, H), dev = _matrix(dy, "dy", torch.bfloat16)
    rt = _dtype(sum, "sum")
    res = {} if out is None else dict(out)
    if res.get("dres") is None:
        res["dres"] = torch.empty(T, H, dtype=sum.dtype, device=dev)
    nbytes = 0
    if dgamma:
        if res.get("dgamma") is None:
            res["dgamma"] = torch.empty(H, dtype=torch.float32, device=dev)
        nbytes = workspace_size(WS_RMSNORM_BACKWARD, T, H, 0, 1, 1)
        if workspace is not None:
            _check_workspace(workspace, nbytes, dev.index)
        elif nbytes:
            workspace = _workspace(nbytes, dev)
    _call(load().w4a4_add_rmsnorm_bwd, dev, T, H, _ptr(dy, "dy", dy.shape, torch.bfloat16, dev),
          _ptr(sum, "sum", dy.shape, sum.dtype, dev), rt, _ptr(gamma, "gamma", (H,), gamma.dtype, dev),
          _dtype(gamma, "gamma"), _ptr(rstd, "rstd", (T,), torch.float32, dev),
          _ptr(dsum, "dsum", dy.shape, sum.dtype, dev), _ptr(res["dres"], "dres", dy.shape, sum.dtype, dev),
          _ptr(res.get("dx"), "dx", dy.shape, torch.bfloat16, dev),
          _ptr(res["dgamma"], "dgamma", (H,), torch.float32, dev) if dgamma else None,
          workspace.data_ptr() if nbytes else None, workspace.numel() if nbytes else 0)
    return res


def w4a4_mx_linear_fwd(xq, wq, T, K, N, y=None):
    """y [T, N] = x W^T on MX operands, bf16 out, FP32 accumulation.

    xq: codes and scales of ``w4a4_add_rmsnorm_fwd`` or ``w4a4_mx_quantize_rows`` (MXFP8 or MXFP4, told
    apart by the codes' width); wq: ``w4a4_mx_quantize_rows(w, MX_FP4)`` of the weight w [N, K].
    K % 128 == 0, N % 8 == 0 (``w4a4_linear_bwd``, its backward: both % 256 == 0 and <= 8192).
    y: where to write (a column slice will do).  A row's bits do not depend on T or on the other rows."""
    codes = xq["codes"]
    _, dev = _matrix(codes, "xq codes", torch.uint8)
    fmt = MX_FP8 if codes.shape[1] == K else MX_FP4
    if y is None:
        y = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    _call(load().w4a4_mx_linear_fwd, dev, T, K, N, fmt,
          _ptr(codes, "xq codes", _code_shape(T, K, fmt), torch.uint8, dev),
          _ptr(xq["scales"], "xq scales", (T, K // 32), torch.uint8, dev),
          _ptr(wq["codes"], "wq codes", (N, K // 2), torch.uint8, dev),
          _ptr(wq["scales"], "wq scales", (N, K // 32), torch.uint8, dev),
          _ptr(y, "y", (T, N), torch.bfloat16, dev, rows=True), _pitch(y))
    return y


# ------------------------------------------------ token dispatch and SwiGLU
# Checks and streams as the calls above.
def _row(t):
    """(T, k) of a routing tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        raise W4A4Error("topk_idx and row_map must be 2-d tensors on the GPU")
    return t.shape


@functools.lru_cache(maxsize=1024)
def _permute_workspace(T, k, E):
    """Its bytes (a call into the library takes as long as all checks of two tensors)."""
    return workspace_size(WS_PERMUTE, T, 0, 0, E, k)


def w4a4_permute_fwd(x, topk_idx, E, row_align=1, out=None, workspace=None):
    """Rows of x [T, H] (bf16 or float32; a column slice will do) sorted by expert, one for each of a token's
    k slots: xp[row_map[t, j]] = x[t], each expert's rows in ascending token order and padded with zeros to
    a multiple of row_align.  topk_idx [T, k] int32; ids outside [0, E) are slots that are not dispatched
    (row_map -1).  x None: the maps alone.

    Returns a dict: xp [cap, H] (with x), offsets [E + 1], row_map [T, k], src_row [cap] int32, where cap =
    rows_capacity(T, k, E, row_align); rows from offsets[E] on are not written.  Tensors of `out` are used where
    given.  workspace: at least workspace_size(WS_PERMUTE, T, 0, 0, E, k) bytes (uint8), allocated where it is not
    given."""
    T, k = _row(topk_idx)
    dev, i32 = topk_idx.device, torch.int32
    res = {} if out is None else dict(out)
    cap = max(0, T * k + E * (row_align - 1))
    H, dtype, pitch, xptr, xpptr = 8, 0, 8, None, None
    if x is not None:
        H = _matrix(x, "x")[0][1]
        dtype, pitch = _dtype(x, "x"), _pitch(x)
        xptr = _ptr(x, "x", (T, H), x.dtype, dev, rows=True)
        xp = res.get("xp")
        if xp is None:
            xp = res["xp"] = torch.empty(cap, H, dtype=x.dtype, device=dev)
        xpptr = _ptr(xp, "xp", (cap, H), x.dtype, dev)
    offsets, row_map, src_row = res.get("offsets"), res.get("row_map"), res.get("src_row")
    if offsets is None:
        offsets = res["offsets"] = torch.empty(max(0, E) + 1, dtype=i32, device=dev)
    if row_map is None:
        row_map = res["row_map"] = torch.empty(T, k, dtype=i32, device=dev)
    if src_row is None:
        src_row = res["src_row"] = torch.empty(cap, dtype=i32, device=dev)
    nbytes = _permute_workspace(T, k, E)
    if workspace is not None:
        _check_workspace(workspace, nbytes, dev.index)
    elif nbytes:
        workspace = _workspace(nbytes, dev)
    _call(_lib.w4a4_permute_fwd, dev, T, H, k, E, row_align, dtype, xptr, pitch,
          _ptr(topk_idx, "topk_idx", (T, k), i32, dev), xpptr, _ptr(offsets, "offsets", (E + 1,), i32, dev),
          _ptr(row_map, "row_map", (T, k), i32, dev), _ptr(src_row, "src_row", (cap,), i32, dev),
          workspace.data_ptr() if nbytes else None, workspace.numel() if nbytes else 0)
    return res


def w4a4_permute_bwd(dxp, perm, dx=None):
    """Gradient of ``w4a4_permute_fwd``: dx[t] = sum_j dxp[row_map[t, j]] in FP32, rounded once.  dxp [rows, H] bf16
    or float32; perm: the maps (row_map is read).  dx: where to write (a column slice will do)."""
    (rows, H), dev = _matrix(dxp, "dxp")
    row_map = perm["row_map"]
    T, k = _row(row_map)
    if dx is None:
        dx = torch.empty(T, H, dtype=dxp.dtype, device=dev)
    _call(load().w4a4_permute_bwd, dev, T, H, k, rows, _dtype(dxp, "dxp"), _ptr(dxp, "dxp", (rows, H), dxp.dtype, dev),
          _ptr(row_map, "row_map", (T, k), torch.int32, dev), _ptr(dx, "dx", (T, H), dxp.dtype, dev, rows=True),
          _pitch(dx))
    return dx


def w4a4_unpermute_fwd(o, perm, topk_w, y=None):
    """y[t] = sum_j topk_w[t, j] o[row_map[t, j]] in FP32 over the dispatched slots, rounded once.  o [rows, H] bf16
    or float32; perm: the maps (row_map is read); topk_w [T, k] float32.  y: where to write (a column slice will
    do)."""
    (rows, H), dev = _matrix(o, "o")
    row_map = perm["row_map"]
    T, k = _row(row_map)
    if y is None:
        y = torch.empty(T, H, dtype=o.dtype, device=dev)
    _call(load().w4a4_unpermute_fwd, dev, T, H, k, rows, _dtype(o, "o"), _ptr(o, "o", (rows, H), o.dtype, dev),
          _ptr(row_map, "row_map", (T, k), torch.int32, dev), _ptr(topk_w, "topk_w", (T, k), torch.float32, dev),
          _ptr(y, "y", (T, H), o.dtype, dev, rows=True), _pitch(y))
    return y


def w4a4_unpermute_bwd(dy, o, perm, topk_w, do=True, dtopk_w=True, out=None):
    """Gradients of ``w4a4_unpermute_fwd`` for dy [T, H], the gradient of y (a column slice will do): do [rows, H]
    (the type of dy; do[row_map[t, j]] = topk_w[t, j] dy[t], pad rows zero, rows from offsets[E] on not written)
    and dtopk_w [T, k] float32 (<dy[t], o[row_map[t, j]]>, 0 where not dispatched).  o: the forward's; None will do
    without dtopk_w.  perm: the dict of ``w4a4_permute_fwd`` (or of a quantise-and-permute call); where o holds fewer
    rows than that call's (those in use), with its src_row cut to as many.  Returns a dict of what `do` and `dtopk_w`
    ask for; tensors of `out` are used where given."""
    (T, H), dev = _matrix(dy, "dy")
    row_map, offsets, src_row = perm["row_map"], perm["offsets"], perm["src_row"]
    k = _row(row_map)[1]
    res = {} if out is None else dict(out)
    rows = (o if o is not None else src_row).shape[0]
    d_o = dw = None
    if do:
        d_o = res.get("do")
        if d_o is None:
            d_o = res["do"] = torch.empty(rows, H, dtype=dy.dtype, device=dev)
        d_o = _ptr(d_o, "do", (rows, H), dy.dtype, dev)
    if dtopk_w:
        dw = res.get("dtopk_w")
        if dw is None:
            dw = res["dtopk_w"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        dw = _ptr(dw, "dtopk_w", (T, k), torch.float32, dev)
    i32 = torch.int32
    _call(load().w4a4_unpermute_bwd, dev, T, H, k, offsets.shape[0] - 1, rows, _dtype(dy, "dy"),
          _ptr(dy, "dy", (T, H), dy.dtype, dev, rows=True), _pitch(dy), _ptr(o, "o", (rows, H), dy.dtype, dev),
          _ptr(row_map, "row_map", (T, k), i32, dev), _ptr(topk_w, "topk_w", (T, k), torch.float32, dev),
          _ptr(offsets, "offsets", offsets.shape, i32, dev), _ptr(src_row, "src_row", (rows,), i32, dev), d_o, dw)
    return res


def _checkpoint(kept, T, width, dev):
    """Addresses of an MXFP8 checkpoint's codes and scales [T, width]."""
    return (_ptr(kept["h_codes"], "h_codes", (T, width), torch.uint8, dev),
            _ptr(kept["h_scales"], "h_scales", (T, width // 32), torch.uint8, dev))


def w4a4_swiglu_fwd(h, fmt=None, a=True, checkpoint=False, rows=None, out=None):
    """a = gate sigmoid(gate) up of h = (gate, up) [T, 2I] bf16 (a column slice of a wider matrix will do), rounded
    to bf16, with the MX encoding of a (fmt MX_FP4 or MX_FP8) and the MXFP8 checkpoint of h for
    ``w4a4_swiglu_bwd``.

    rows: int32 tensor of one element on the GPU, the number of rows in use (None: all T); rows behind them are
    left as they are.  Returns a dict with what was asked for: a [T, I], codes and scales (with fmt), h_codes [T, 2I]
    and h_scales [T, 2I/32] uint8 (with checkpoint).  Tensors of `out` are used where given."""
    (T, W), dev = _matrix(h, "h", torch.bfloat16)
    I = W // 2  # noqa: E741
    if W % 2:
        raise W4A4Error(f"h has an odd number of columns ({W})")
    res = {} if out is None else dict(out)
    if a and res.get("a") is None:
        res["a"] = torch.empty(T, I, dtype=torch.bfloat16, device=dev)
    codes, scales = (None, None) if fmt is None else _mx_buffers(res, T, I, fmt, dev)
    hc = hs = None
    if checkpoint:
        if res.get("h_codes") is None:
            res["h_codes"] = torch.empty(T, W, dtype=torch.uint8, device=dev)
        if res.get("h_scales") is None:
            res["h_scales"] = torch.empty(T, W // 32, dtype=torch.uint8, device=dev)
        hc, hs = _checkpoint(res, T, W, dev)
    _call(load().w4a4_swiglu_fwd, dev, T, I, _ptr(h, "h", (T, W), torch.bfloat16, dev, rows=True), _pitch(h),
          _ptr(rows, "rows", (1,), torch.int32, dev), MX_NONE if fmt is None else fmt,
          _ptr(res["a"], "a", (T, I), torch.bfloat16, dev) if a else None, codes, scales, hc, hs)
    return res


def w4a4_swiglu_bwd(da, kept, a=False, dh=True, rows=None, out=None):
    """Gradient of ``w4a4_swiglu_fwd`` for da [T, I] bf16, the gradient of a.  kept: the bf16 h [T, 2I] (a column slice
    will do) or a dict with its checkpoint (h_codes, h_scales), whose values then stand for h throughout.

    Returns a dict: dh [T, 2I] bf16 unless `dh` is false (da may be None then), and with `a` the forward's output
    once more [T, I] (for the next product's weight gradient).  rows as in the forward.  Tensors of `out` are
    used where given: its dh may be a dense kept h, its a may be da."""
    ckpt = isinstance(kept, dict)
    (T, W), dev = _matrix(kept["h_codes"], "h_codes", torch.uint8) if ckpt else _matrix(kept, "h", torch.bfloat16)
    I = W // 2  # noqa: E741
    res = {} if out is None else dict(out)
    if dh and res.get("dh") is None:
        res["dh"] = torch.empty(T, W, dtype=torch.bfloat16, device=dev)
    if a and res.get("a") is None:
        res["a"] = torch.empty(T, I, dtype=torch.bfloat16, device=dev)
    hc, hs = _checkpoint(kept, T, W, dev) if ckpt else (None, None)
    _call(load().w4a4_swiglu_bwd, dev, T, I, _ptr(da, "da", (T, I), torch.bfloat16, dev),
          None if ckpt else _ptr(kept, "h", (T, W), torch.bfloat16, dev, rows=True), W if ckpt else _pitch(kept),
          hc, hs, _ptr(rows, "rows", (1,), torch.int32, dev),
          _ptr(res["dh"], "dh", (T, W), torch.bfloat16, dev) if dh else None,
          _ptr(res["a"], "a", (T, I), torch.bfloat16, dev) if a else None)
    return res


def w4a4_grouped_expert_fwd_ckpt(xq, topk_w, w1q, w2q, T, H, I, E, k, row_align=1, save_o=False, out=None,  # noqa: E741
                                 workspace=None):
    """``w4a4_grouped_expert_fwd``, or with xq of ``w4a4_mx_quantize_permute`` (which has no outer scales)
    ``w4a4_mx_grouped_expert_fwd``, that keeps h in MXFP8 for ``w4a4_expert_bwd_ckpt`` in place of bf16 h and a.

    Returns dict(y [T, H], h_codes [cap, 2I] and h_scales [cap, 2I/32] uint8, and with `save_o` the experts' outputs o
    [cap, H] bf16, which ``w4a4_unpermute_bwd`` takes for the gradient of topk_w); rows of h and o from
    offsets[E] on are not written.  Tensors of `out` are used where given.  workspace: at least
    workspace_size(WS_FORWARD, T, H, I, E, k, row_align) bytes (uint8)."""
    dev, bf16, i32, u8, f32 = xq["codes"].device, torch.bfloat16, torch.int32, torch.uint8, torch.float32
    mx = "outer" not in xq
    cap, block = rows_capacity(T, k, E, row_align), 32 if mx else 16
    res = {} if out is None else dict(out)
    for name, shape, dtype in (("y", (T, H), bf16), ("h_codes", (cap, 2 * I), u8), ("h_scales", (cap, 2 * I // 32), u8)):
        if res.get(name) is None:
            res[name] = torch.empty(shape, dtype=dtype, device=dev)
    if save_o and res.get("o") is None:
        res["o"] = torch.empty(cap, H, dtype=bf16, device=dev)
    nbytes = workspace_size(WS_FORWARD, T, H, I, E, k, row_align)
    if workspace is not None:
        _check_workspace(workspace, nbytes, dev.index)
    else:
        workspace = _workspace(nbytes, dev)

    def operand(q, name, *rows, width):
        got = [_ptr(q["codes"], f"{name} codes", (*rows, width // 2), u8, dev),
               _ptr(q["scales"], f"{name} scales", (*rows, width // block), u8, dev)]
        return got if mx else got + [_ptr(q["outer"], f"{name} outer", rows, f32, dev)]

    lib = load()
    _call(lib.w4a4_mx_grouped_expert_fwd_ckpt if mx else lib.w4a4_grouped_expert_fwd_ckpt, dev, T, H, I, E, k,
          row_align, *operand(xq, "xq", cap, width=H), _ptr(xq["offsets"], "offsets", (E + 1,), i32, dev),
          _ptr(xq["row_map"], "row_map", (T, k), i32, dev), _ptr(xq["src_row"], "src_row", (cap,), i32, dev),
          _ptr(topk_w, "topk_w", (T, k), f32, dev), *operand(w1q, "w1q", E, 2 * I, width=H),
          *operand(w2q, "w2q", E, H, width=I), _ptr(res["y"], "y", (T, H), bf16, dev),
          *_checkpoint(res, cap, 2 * I, dev), _ptr(res["o"], "o", (cap, H), bf16, dev) if save_o else None,
          workspace.data_ptr(), workspace.numel())
    return res


def w4a4_expert_bwd_ckpt(dy, x, w1, w2, kept, topk_w, xq, T, H, I, E, k, row_align=1, out=None, workspace=None):  # noqa: E741
    """``w4a4_expert_bwd`` from an MXFP8 checkpoint of h in place of the bf16 h and a: kept is a dict with h_codes
    [cap, 2I] and h_scales [cap, 2I/32] uint8, of ``w4a4_grouped_expert_fwd_ckpt`` (or ``w4a4_swiglu_fwd(h, a=False,
    checkpoint=True, rows=xq["offsets"][E:])`` of a bf16 h).  Returns dict(dx [T, H], dw1 [E, 2I, H], dw2 [E, H, I])
    bf16.  workspace: at least workspace_size(WS_BACKWARD_CKPT, T, H, I, E, k, row_align) bytes (uint8)."""
    dev, bf16, i32 = w1.device, torch.bfloat16, torch.int32
    cap = rows_capacity(T, k, E, row_align)
    res = {} if out is None else dict(out)
    for name, shape in (("dx", (T, H)), ("dw1", (E, 2 * I, H)), ("dw2", (E, H, I))):
        if res.get(name) is None:
            res[name] = torch.empty(shape, dtype=bf16, device=dev)
    nbytes = workspace_size(WS_BACKWARD_CKPT, T, H, I, E, k, row_align)
    if workspace is not None:
        _check_workspace(workspace, nbytes, dev.index)
    else:
        workspace = _workspace(nbytes, dev)
    codes, scales = _checkpoint(kept, cap, 2 * I, dev)
    _call(load().w4a4_expert_bwd_ckpt, dev, T, H, I, E, k, row_align, _ptr(dy, "dy", (T, H), bf16, dev),
          _ptr(x, "x", (T, H), bf16, dev), _ptr(w1, "w1", (E, 2 * I, H), bf16, dev),
          _ptr(w2, "w2", (E, H, I), bf16, dev), codes, scales, _ptr(topk_w, "topk_w", (T, k), torch.float32, dev),
          _ptr(xq["offsets"], "offsets", (E + 1,), i32, dev), _ptr(xq["row_map"], "row_map", (T, k), i32, dev),
          _ptr(xq["src_row"], "src_row", (cap,), i32, dev), _ptr(res["dx"], "dx", (T, H), bf16, dev),
          _ptr(res["dw1"], "dw1", (E, 2 * I, H), bf16, dev), _ptr(res["dw2"], "dw2", (E, H, I), bf16, dev),
          workspace.data_ptr(), workspace.numel())
    return res


def w4a4_profiler_enable(on=True):
    load().w4a4_profiler_enable(1 if on else 0)


def w4a4_profiler_report():
    lib = load()
    n = lib.w4a4_profiler_report(None, 0)
    if n < 0:
        raise W4A4Error("profiler report failed")
    buf = ctypes.create_string_buffer(n + 1)
    lib.w4a4_profiler_report(buf, n + 1)
    return json.loads(buf.value.decode())

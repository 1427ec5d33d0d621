"""Thin Python binding of libmoe (include/moe.h) over torch device tensors.

Argument marshalling only: every step runs in the library's HIP kernels.
torch provides device memory and the current stream.  If the library has not
been built, loading fails with an error (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
F32, BF16, INT4_B32, INT2_B32, INT3_B32, FP8_E4M3 = 0, 1, 2, 3, 4, 5
_QUANT_BY_BITS = {4: INT4_B32, 3: INT3_B32, 2: INT2_B32}

EXPORTS = ["moe_abi_version", "moe_status_string", "moe_route_workspace_size", "moe_route",
           "moe_permute_workspace_size", "moe_permute", "moe_ffn_workspace_size", "moe_ffn",
           "moe_route_group_workspace_size", "moe_route_group", "moe_route_group_noalloc", "moe_combine", "moe_combine_steer", "moe_layer_workspace_size", "moe_layer", "moe_expert_freq", "moe_profile_workspace_size", "moe_profile_rank",
           "moe_profile_hits", "moe_strp_size", "moe_strp_write", "moe_strp_read", "moe_profile_remap",
           "moe_kv_plan", "moe_qk_norm_rope", "moe_paged_attn_workspace_size", "moe_paged_attn",
           "moe_linear_workspace_size", "moe_linear"]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class ExpertWeights(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p),
                ("s_down", ctypes.c_void_p)]


class KVCacheStruct(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


_lib = None


def lib_path() -> str:
    return _build.LIB


def load():
    """Load libmoe.so (raises if it is missing: build it first)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m routed_expert_ffn_amd.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.moe_abi_version.restype = ctypes.c_int
    L.moe_abi_version.argtypes = []
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [ctypes.c_int]
    L.moe_route_workspace_size.restype = sz
    L.moe_route_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.moe_route.restype = ctypes.c_int
    L.moe_route.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.moe_permute_workspace_size.restype = sz
    L.moe_permute_workspace_size.argtypes = [i32, i32, i32]
    L.moe_permute.restype = ctypes.c_int
    L.moe_permute.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.moe_ffn_workspace_size.restype = sz
    L.moe_ffn_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    L.moe_ffn.restype = ctypes.c_int
    L.moe_ffn.argtypes = [vp, i32, ctypes.POINTER(ExpertWeights), vp, vp, i32, i32, i32, i32, i32, vp, i32, vp, sz,
                          vp]
    L.moe_combine.restype = ctypes.c_int
    L.moe_combine.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    L.moe_route_group_workspace_size.restype = sz
    L.moe_route_group_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.moe_route_group.restype = ctypes.c_int
    L.moe_route_group.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_route_group_noalloc.restype = ctypes.c_int
    L.moe_route_group_noalloc.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.moe_combine_steer.restype = ctypes.c_int
    L.moe_combine_steer.argtypes = [vp, i32, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp]
    L.moe_layer_workspace_size.restype = sz
    L.moe_layer_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    L.moe_layer.restype = ctypes.c_int
    L.moe_layer.argtypes = [vp, i32, vp, vp, ctypes.POINTER(ExpertWeights), i32, i32, i32, i32, i32, vp, vp, vp,
                            vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_expert_freq.restype = ctypes.c_int
    L.moe_expert_freq.argtypes = [vp, i32, i64, i32, i32, vp, i32, i32, vp, vp, vp]
    L.moe_profile_workspace_size.restype = sz
    L.moe_profile_workspace_size.argtypes = [i32, i32]
    L.moe_profile_rank.restype = ctypes.c_int
    L.moe_profile_rank.argtypes = [vp, i32, i32, vp, vp, vp, sz, vp]
    L.moe_profile_hits.restype = ctypes.c_int
    L.moe_profile_hits.argtypes = [vp, i32, i64, i32, vp, i32, i64, vp, vp]
    L.moe_strp_size.restype = sz
    L.moe_strp_size.argtypes = [i32, i32, i32]
    L.moe_strp_write.restype = ctypes.c_int
    L.moe_strp_write.argtypes = [vp, i32, i32, i32, vp, sz]
    L.moe_strp_read.restype = ctypes.c_int
    L.moe_strp_read.argtypes = [vp, sz, vp, vp, vp, vp, i32, vp, i64]
    L.moe_profile_remap.restype = ctypes.c_int
    L.moe_profile_remap.argtypes = [vp, i32, i32, i32, vp, i32, vp, vp]
    f32, kvp = ctypes.c_float, ctypes.POINTER(KVCacheStruct)
    L.moe_kv_plan.restype = ctypes.c_int
    L.moe_kv_plan.argtypes = [vp, vp, i32, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp]
    L.moe_qk_norm_rope.restype = ctypes.c_int
    L.moe_qk_norm_rope.argtypes = [vp, i32, i64, i32, i32, kvp, vp, vp, f32, vp, i32, i32, f32, vp, vp, vp, vp]
    L.moe_paged_attn_workspace_size.restype = sz
    L.moe_paged_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.moe_paged_attn.restype = ctypes.c_int
    L.moe_paged_attn.argtypes = [vp, i32, i64, i32, i32, kvp, vp, i32, vp, vp, i32, f32, f32, i32, vp, vp, sz, vp]
    L.moe_linear_workspace_size.restype = sz
    L.moe_linear_workspace_size.argtypes = [i32, i32, i32]
    L.moe_linear.restype = ctypes.c_int
    L.moe_linear.argtypes = [vp, i32, i64, vp, i32, vp, i32, vp, i32, i32, i32, vp, i32, vp, sz, vp]
    _lib = L
    return L


def status_string(s: int) -> str:
    return load().moe_status_string(int(s)).decode()


def abi_version() -> int:
    return int(load().moe_abi_version())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _chk(rc, what):
    if rc != MOE_OK:
        raise MoeError(rc, what)


def _act_dtype(t) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"activations must be float32 or bfloat16, not {t.dtype}")


def _need(t, name, dtype=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _workspace(nbytes: int, device, ws=None):
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ moe_route
def route_workspace_size(T, H, E, K, x_dtype=BF16) -> int:
    return int(load().moe_route_workspace_size(T, H, E, K, x_dtype))


def route(x, w_router, K: int, bias=None, logits_out=None, workspace=None, stream=None, out=None):
    """Top-K expert ids [T][K] int32 and weights [T][K] fp32 (out: optional (idx, w) to fill)."""
    _need(x, "x")
    T, H = x.shape
    E = w_router.shape[0]
    _need(w_router, "w_router", torch.float32, (E, H))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    if logits_out is not None:
        _need(logits_out, "logits_out", torch.float32, (T, E))
    if out is not None:
        idx, w = out
        _need(idx, "topk_idx", torch.int32, (T, K))
        _need(w, "topk_w", torch.float32, (T, K))
    else:
        idx = torch.empty((T, K), dtype=torch.int32, device=x.device)
        w = torch.empty((T, K), dtype=torch.float32, device=x.device)
    nb = route_workspace_size(T, H, E, K, _act_dtype(x))
    ws = _workspace(nb, x.device, workspace)
    _chk(load().moe_route(_ptr(x), _act_dtype(x), _ptr(w_router), _ptr(bias), T, H, E, K, _ptr(idx), _ptr(w),
                          _ptr(logits_out), _ptr(ws), nb, _stream(stream)), "moe_route")
    return idx, w


# ------------------------------------------------------------------ moe_permute
def permute_workspace_size(T, K, E) -> int:
    return int(load().moe_permute_workspace_size(T, K, E))


def permute(topk_idx, E: int, workspace=None, stream=None, out=None):
    """(counts [E], offsets [E+1], perm [T*K], inv_perm [T*K]), all int32 (out: optional tuple to fill)."""
    _need(topk_idx, "topk_idx", torch.int32)
    T, K = topk_idx.shape
    dev = topk_idx.device
    if out is not None:
        counts, offsets, perm, inv = out
        for n, t, shp in (("counts", counts, (E,)), ("offsets", offsets, (E + 1,)), ("perm", perm, (T * K,)),
                          ("inv_perm", inv, (T * K,))):
            _need(t, n, torch.int32, shp)
    else:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
        offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(T * K, dtype=torch.int32, device=dev)
        inv = torch.empty(T * K, dtype=torch.int32, device=dev)
    nb = permute_workspace_size(T, K, E)
    ws = _workspace(nb, dev, workspace)
    _chk(load().moe_permute(_ptr(topk_idx), T, K, E, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(ws),
                            nb, _stream(stream)), "moe_permute")
    return counts, offsets, perm, inv


# ------------------------------------------------------------------ moe_route_group
def route_group_workspace_size(T, H, E, K, x_dtype=BF16) -> int:
    return int(load().moe_route_group_workspace_size(T, H, E, K, x_dtype))


def route_group(x, w_router, K: int, bias=None, workspace=None, stream=None, out=None):
    """moe_route then moe_permute in one call (one launch for selection and
    grouping when few tokens are routed).  Returns (idx, w, counts, offsets,
    perm, inv); out: optional 6-tuple to fill."""
    _need(x, "x")
    T, H = x.shape
    E = w_router.shape[0]
    _need(w_router, "w_router", torch.float32, (E, H))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    dev = x.device
    if out is not None:
        idx, w, counts, offsets, perm, inv = out
        for n, t, dt, shp in (("topk_idx", idx, torch.int32, (T, K)), ("topk_w", w, torch.float32, (T, K)),
                              ("counts", counts, torch.int32, (E,)), ("offsets", offsets, torch.int32, (E + 1,)),
                              ("perm", perm, torch.int32, (T * K,)), ("inv_perm", inv, torch.int32, (T * K,))):
            _need(t, n, dt, shp)
    else:
        i32 = dict(dtype=torch.int32, device=dev)
        idx, w = torch.empty((T, K), **i32), torch.empty((T, K), dtype=torch.float32, device=dev)
        counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        perm, inv = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
    nb = route_group_workspace_size(T, H, E, K, _act_dtype(x))
    ws = _workspace(nb, dev, workspace)
    _chk(load().moe_route_group(_ptr(x), _act_dtype(x), _ptr(w_router), _ptr(bias), T, H, E, K, _ptr(idx), _ptr(w),
                                _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(ws), nb, _stream(stream)),
         "moe_route_group")
    return idx, w, counts, offsets, perm, inv


def route_group_noalloc(x, w_router, K: int, bias=None, stream=None, out=None):
    """moe_route_group_noalloc: route_group on the library's own per-GPU
    scratch (no workspace argument, nothing allocated by the library).
    Returns (idx, w, counts, offsets, perm, inv); out: optional 6-tuple to fill."""
    _need(x, "x")
    T, H = x.shape
    E = w_router.shape[0]
    _need(w_router, "w_router", torch.float32, (E, H))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    dev = x.device
    if out is not None:
        idx, w, counts, offsets, perm, inv = out
        for n, t, dt, shp in (("topk_idx", idx, torch.int32, (T, K)), ("topk_w", w, torch.float32, (T, K)),
                              ("counts", counts, torch.int32, (E,)), ("offsets", offsets, torch.int32, (E + 1,)),
                              ("perm", perm, torch.int32, (T * K,)), ("inv_perm", inv, torch.int32, (T * K,))):
            _need(t, n, dt, shp)
    else:
        i32 = dict(dtype=torch.int32, device=dev)
        idx, w = torch.empty((T, K), **i32), torch.empty((T, K), dtype=torch.float32, device=dev)
        counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        perm, inv = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
    _chk(load().moe_route_group_noalloc(_ptr(x), _act_dtype(x), _ptr(w_router), _ptr(bias), T, H, E, K, _ptr(idx),
                                        _ptr(w), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv),
                                        _stream(stream)), "moe_route_group_noalloc")
    return idx, w, counts, offsets, perm, inv


# ------------------------------------------------------------------ moe_ffn
def weights_struct(wg, wu, wd, sg=None, su=None, sd=None) -> ExpertWeights:
    if wg.dtype == torch.uint8:
        # block-quantised: the bits per weight follow from the row lengths
        # (gate/up rows hold H inputs, H = the down matrix's row count)
        H, F = wd.shape[1], wg.shape[1]
        bits = wg.shape[2] * 8 // H
        if bits not in _QUANT_BY_BITS or wg.shape[2] * 8 != bits * H or wd.shape[2] * 8 != bits * F:
            raise ValueError(f"packed weights of shapes {tuple(wg.shape)} / {tuple(wd.shape)} are not int4, int3 or int2")
        dt = _QUANT_BY_BITS[bits]
        for n, s in (("s_gate", sg), ("s_up", su), ("s_down", sd)):
            _need(s, n, torch.float16)
    elif wg.dtype == torch.bfloat16:
        dt = BF16
    elif wg.dtype == torch.float32:
        dt = F32
    else:
        raise TypeError(f"expert weights must be float32, bfloat16 or uint8 (int4/int3/int2), not {wg.dtype}")
    for n, t in (("w_gate", wg), ("w_up", wu), ("w_down", wd)):
        _need(t, n, wg.dtype)
    return ExpertWeights(dt, wg.data_ptr(), wu.data_ptr(), wd.data_ptr(),
                         sg.data_ptr() if sg is not None else None, su.data_ptr() if su is not None else None,
                         sd.data_ptr() if sd is not None else None)


def ffn_workspace_size(T, K, E, H, F, x_dtype, w_dtype) -> int:
    return int(load().moe_ffn_workspace_size(T, K, E, H, F, x_dtype, w_dtype))


def ffn(x, wg, wu, wd, offsets, perm, K: int, sg=None, su=None, sd=None, y_dtype=None, out=None, workspace=None,
        stream=None):
    """y_perm [T*K][H] for the grouped rows."""
    _need(x, "x")
    T, H = x.shape
    E = wg.shape[0]
    F = wg.shape[1]
    _need(offsets, "offsets", torch.int32, (E + 1,))
    _need(perm, "perm", torch.int32, (T * K,))
    ws_struct = weights_struct(wg, wu, wd, sg, su, sd)
    if y_dtype is None:
        y_dtype = x.dtype
    y = out if out is not None else torch.empty((T * K, H), dtype=y_dtype, device=x.device)
    _need(y, "y_perm", y_dtype, (T * K, H))
    nb = ffn_workspace_size(T, K, E, H, F, _act_dtype(x), ws_struct.dtype)
    ws = _workspace(nb, x.device, workspace)
    _chk(load().moe_ffn(_ptr(x), _act_dtype(x), ctypes.byref(ws_struct), _ptr(offsets), _ptr(perm), T, K, H, F, E,
                        _ptr(y), _act_dtype(y), _ptr(ws), nb, _stream(stream)), "moe_ffn")
    return y


# ------------------------------------------------------------------ moe_combine
def combine(y_perm, inv_perm, topk_w, residual=None, out_dtype=None, out=None, stream=None, steer_v=None):
    """out [T][H] = sum_k w * y_perm[inv] (+ residual); with steer_v ([H] fp32
    unit vector) the row's component along it is removed before rounding
    (moe_combine_steer)."""
    _need(y_perm, "y_perm")
    _need(topk_w, "topk_w", torch.float32)
    T, K = topk_w.shape
    H = y_perm.shape[1]
    _need(inv_perm, "inv_perm", torch.int32, (T * K,))
    if out_dtype is None:
        out_dtype = residual.dtype if residual is not None else y_perm.dtype
    if residual is not None:
        _need(residual, "residual", out_dtype, (T, H))
    o = out if out is not None else torch.empty((T, H), dtype=out_dtype, device=y_perm.device)
    _need(o, "out", out_dtype, (T, H))
    if steer_v is not None:
        _need(steer_v, "steer_v", torch.float32, (H,))
        _chk(load().moe_combine_steer(_ptr(y_perm), _act_dtype(y_perm), _ptr(inv_perm), _ptr(topk_w), _ptr(residual),
                                      _ptr(steer_v), T, K, H, _ptr(o), _act_dtype(o), _stream(stream)),
             "moe_combine_steer")
        return o
    _chk(load().moe_combine(_ptr(y_perm), _act_dtype(y_perm), _ptr(inv_perm), _ptr(topk_w), _ptr(residual), T, K, H,
                            _ptr(o), _act_dtype(o), _stream(stream)), "moe_combine")
    return o


# ------------------------------------------------------------------ moe_expert_freq
def expert_freq(logits, K: int, keep: int = 0, counts=None, accumulate: bool = False, stream=None):
    """(counts [L][E] int64, rank_of [L][E] int32 | None, keep_map [L][keep] int32 | None)."""
    _need(logits, "logits", torch.float32)
    if logits.dim() == 2:
        logits = logits.unsqueeze(0)
    L, T, E = logits.shape
    dev = logits.device
    if counts is None:
        counts = torch.zeros((L, E), dtype=torch.int64, device=dev)
    _need(counts, "counts", torch.int64, (L, E))
    rank_of = torch.empty((L, E), dtype=torch.int32, device=dev) if keep else None
    keep_map = torch.empty((L, keep), dtype=torch.int32, device=dev) if keep else None
    _chk(load().moe_expert_freq(_ptr(logits), L, T, E, K, _ptr(counts), 1 if accumulate else 0, keep, _ptr(rank_of),
                                _ptr(keep_map), _stream(stream)), "moe_expert_freq")
    return counts, rank_of, keep_map


# ------------------------------------------------------------------ expert profile
def profile_rank(counts, workspace=None, stream=None):
    """counts [L][E] int64 (device) -> (rank [L][E] int32, pairs [L*E][2] int16 holding uint16 (layer, expert))."""
    _need(counts, "counts", torch.int64)
    L, E = counts.shape
    dev = counts.device
    rank = torch.empty((L, E), dtype=torch.int32, device=dev)
    pairs = torch.empty((L * E, 2), dtype=torch.int16, device=dev)
    nb = int(load().moe_profile_workspace_size(L, E))
    ws = _workspace(nb, dev, workspace)
    _chk(load().moe_profile_rank(_ptr(counts), L, E, _ptr(rank), _ptr(pairs), _ptr(ws), nb, _stream(stream)),
         "moe_profile_rank")
    return rank, pairs


def profile_hits(trace, rank, S: int, stream=None):
    """trace [L][T][K] int32, rank [L][E] int32 (device) -> hits (a 1-element int64 tensor, device)."""
    _need(trace, "trace", torch.int32)
    _need(rank, "rank", torch.int32)
    L, T, K = trace.shape
    E = rank.shape[1]
    hits = torch.empty(1, dtype=torch.int64, device=trace.device)   # the uint64 count, < 2^63
    _chk(load().moe_profile_hits(_ptr(trace), L, T, K, _ptr(rank), E, int(S), _ptr(hits), _stream(stream)),
         "moe_profile_hits")
    return hits


def _np_ptr(a):
    return ctypes.c_void_p(a.ctypes.data) if a is not None else None


def strp_write(pairs, L: int, E: int) -> bytes:
    """Host pairs [n][2] (uint16 (layer, expert) in rank order) -> the STRP v1 file's bytes."""
    import numpy as np
    p = np.ascontiguousarray(np.asarray(pairs, dtype=np.uint16).reshape(-1, 2))
    n = p.shape[0]
    nb = int(load().moe_strp_size(L, E, n))
    out = np.empty(nb, dtype=np.uint8)
    _chk(load().moe_strp_write(_np_ptr(p), n, L, E, _np_ptr(out), nb), "moe_strp_write")
    return out.tobytes()


def strp_read(buf: bytes):
    """STRP v1 bytes -> (L, E, pairs [n][2] uint16, inverse [L][E] int16)."""
    import numpy as np
    b = np.frombuffer(buf, dtype=np.uint8).copy()
    L, E, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _chk(load().moe_strp_read(_np_ptr(b), b.size, ctypes.byref(L), ctypes.byref(E), ctypes.byref(n), None, 0, None,
                              0), "moe_strp_read")
    pairs = np.empty((n.value, 2), dtype=np.uint16)
    inv = np.empty((L.value, E.value), dtype=np.int16)
    _chk(load().moe_strp_read(_np_ptr(b), b.size, ctypes.byref(L), ctypes.byref(E), ctypes.byref(n), _np_ptr(pairs),
                              n.value, _np_ptr(inv), inv.size), "moe_strp_read")
    return L.value, E.value, pairs, inv


def profile_remap(pairs, keep_map, E_old: int):
    """Host ranked pairs of an E_old-expert profile + keep_map [L][keep] -> the pruned model's ranked pairs."""
    import numpy as np
    p = np.ascontiguousarray(np.asarray(pairs, dtype=np.uint16).reshape(-1, 2))
    km = np.ascontiguousarray(np.asarray(keep_map, dtype=np.int32))
    L, keep = km.shape
    out = np.empty((max(p.shape[0], 1), 2), dtype=np.uint16)
    m = ctypes.c_int32()
    _chk(load().moe_profile_remap(_np_ptr(p), p.shape[0], L, E_old, _np_ptr(km), keep, _np_ptr(out),
                                  ctypes.byref(m)), "moe_profile_remap")
    return out[:m.value].copy()


# ------------------------------------------------------------------ one whole layer
def layer_workspace_size(T, H, E, K, F, x_dtype=BF16, w_dtype=BF16) -> int:
    return int(load().moe_layer_workspace_size(T, H, E, K, F, x_dtype, w_dtype))


class LayerWorkspace:
    """Preallocated workspaces and outputs for repeated calls of `layer` at one shape
    (and of the separate calls at that shape)."""

    def __init__(self, T, H, E, K, F, x_dtype=torch.bfloat16, w_dtype=BF16, y_dtype=None, device="cuda"):
        xd = F32 if x_dtype == torch.float32 else BF16
        self.y_dtype = y_dtype or x_dtype
        self.layer_ws = torch.empty(layer_workspace_size(T, H, E, K, F, xd, w_dtype), dtype=torch.uint8,
                                    device=device)
        self.route_ws = torch.empty(route_workspace_size(T, H, E, K, xd), dtype=torch.uint8, device=device)
        self.group_ws = torch.empty(route_group_workspace_size(T, H, E, K, xd), dtype=torch.uint8, device=device)
        self.perm_ws = torch.empty(permute_workspace_size(T, K, E), dtype=torch.uint8, device=device)
        self.ffn_ws = torch.empty(ffn_workspace_size(T, K, E, H, F, xd, w_dtype), dtype=torch.uint8, device=device)
        self.y = torch.empty((T * K, H), dtype=self.y_dtype, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.route_out = (torch.empty((T, K), **i32), torch.empty((T, K), dtype=torch.float32, device=device))
        self.perm_out = (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * K, **i32),
                         torch.empty(T * K, **i32))
        self.out = torch.empty((T, H), dtype=x_dtype, device=device)


def layer(x, w_router, wg, wu, wd, K: int, bias=None, sg=None, su=None, sd=None, residual=None, lw=None,
          stream=None, out=None, steer_v=None):
    """One MoE layer in one library call (moe_layer): routing + grouping, the
    experts and the combine (steered if steer_v is given).  Returns (out,
    routing dict)."""
    _need(x, "x")
    T, H = x.shape
    E, F = wg.shape[0], wg.shape[1]
    _need(w_router, "w_router", torch.float32, (E, H))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,))
    if residual is not None:
        _need(residual, "residual", x.dtype, (T, H))
    if steer_v is not None:
        _need(steer_v, "steer_v", torch.float32, (H,))
    ws_struct = weights_struct(wg, wu, wd, sg, su, sd)
    dev = x.device
    if lw is not None:
        idx, w = lw.route_out
        counts, offsets, perm, inv = lw.perm_out
        if out is None:
            out = lw.out
    else:
        i32 = dict(dtype=torch.int32, device=dev)
        idx, w = torch.empty((T, K), **i32), torch.empty((T, K), dtype=torch.float32, device=dev)
        counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        perm, inv = torch.empty(T * K, **i32), torch.empty(T * K, **i32)
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=dev)
    _need(out, "out", x.dtype, (T, H))
    nb = layer_workspace_size(T, H, E, K, F, _act_dtype(x), ws_struct.dtype)
    ws = _workspace(nb, dev, lw.layer_ws if lw is not None else None)
    _chk(load().moe_layer(_ptr(x), _act_dtype(x), _ptr(w_router), _ptr(bias), ctypes.byref(ws_struct), T, H, E, K, F,
                          _ptr(residual), _ptr(steer_v), _ptr(out), _ptr(idx), _ptr(w), _ptr(counts), _ptr(offsets),
                          _ptr(perm), _ptr(inv), _ptr(ws), nb, _stream(stream)), "moe_layer")
    return out, dict(idx=idx, w=w, counts=counts, offsets=offsets, perm=perm, inv=inv)


# ------------------------------------------------------------------ the attention half of a layer
_FP8 = torch.float8_e4m3fn


def _elsewhere(dev: int, stream) -> bool:
    """Whether a call has to switch to its tensors' device or to the given stream first (outputs and
    workspaces it allocates then belong to that stream)."""
    return stream is not None or (dev >= 0 and dev != torch._C._cuda_getDevice())


# the current stream of a device, as the library takes it
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(dev: int, t, name, dtype, shape):
    """t's address, after the checks (one pass over them where all hold)."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous() and dev >= 0:
        return t.data_ptr()
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, expected device {dev}")


def _opt(dev: int, t, name, dtype, shape):
    return None if t is None else _on(dev, t, name, dtype, shape)


def _bytes(dev: int, nbytes: int, ws):
    """A workspace of nbytes on the device: the given one where it is large enough, else a new one."""
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", dev))
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous on device {dev}")
    return ws


def _rows(t, name, dtype):
    """A [T][n] tensor whose rows are contiguous (they may lie apart)."""
    if t.dim() == 2 and t.is_cuda and t.dtype is dtype and t.is_contiguous():
        return t.shape[1]
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


class KVCache:
    """A paged key-value cache over tensors in the library's layout (include/moe.h, moe_kv_cache):
    k [pages][kv heads][head_dim / X][page size][X], X = 8 (bfloat16) or 16 (float8_e4m3fn),
    v [pages][kv heads][page size][head_dim], and for float8 the fp32 scales
    k_scale, v_scale [pages][kv heads][page size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in (torch.bfloat16, _FP8):
            raise TypeError(f"a cache holds bfloat16 or float8_e4m3fn, not {k.dtype}")
        _need(k, "k")
        if k.dim() != 5 or k.shape[4] != 16 // k.element_size():
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [pages][kv heads][head_dim / X][page size][X]")
        pages, heads, chunks, page, x = k.shape
        dev = k.get_device()
        _on(dev, v, "v", k.dtype, (pages, heads, page, chunks * x))
        if (k.dtype == _FP8) != (k_scale is not None) or (k.dtype == _FP8) != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to a float8 cache")
        if k_scale is not None:
            _on(dev, k_scale, "k_scale", torch.float32, (pages, heads, page))
            _on(dev, v_scale, "v_scale", torch.float32, (pages, heads, page))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.page_size, self.n_kv_heads, self.head_dim = pages, page, heads, chunks * x
        self.device = dev
        self.struct = KVCacheStruct(BF16 if k.dtype == torch.bfloat16 else FP8_E4M3, pages, page, heads, chunks * x,
                                    k.data_ptr(), v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
                                    None if v_scale is None else v_scale.data_ptr())
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def allocate(cls, num_pages, page_size, n_kv_heads, head_dim, dtype=torch.bfloat16, device="cuda"):
        if dtype not in (torch.bfloat16, _FP8):
            raise TypeError(f"a cache holds bfloat16 or float8_e4m3fn, not {dtype}")
        x = 8 if dtype == torch.bfloat16 else 16
        k = torch.empty((num_pages, n_kv_heads, head_dim // x, page_size, x), dtype=dtype, device=device)
        v = torch.empty((num_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=device)
        if dtype == torch.bfloat16:
            return cls(k, v)
        s = [torch.empty((num_pages, n_kv_heads, page_size), dtype=torch.float32, device=device) for _ in range(2)]
        return cls(k, v, *s)


class KVPlan:
    """The outputs of kv_plan for S requests and T rows: q_offsets [S+1], kv_len [S], positions [T], slots [T],
    counts [2], int32."""

    def __init__(self, q_offsets, kv_len, positions, slots, counts):
        dev, i32 = q_offsets.get_device(), torch.int32
        self.S, self.T, self.device = kv_len.numel(), slots.numel(), dev
        self.ptrs = (_on(dev, q_offsets, "q_offsets", i32, (self.S + 1,)), _on(dev, kv_len, "kv_len", i32, (self.S,)),
                     _on(dev, positions, "positions", i32, (self.T,)), _on(dev, slots, "slots", i32, (self.T,)),
                     _on(dev, counts, "counts", i32, (2,)))
        self.q_offsets, self.kv_len, self.positions, self.slots, self.counts = q_offsets, kv_len, positions, slots, counts

    @classmethod
    def allocate(cls, S, T, device="cuda"):
        return cls(*(torch.empty(n, dtype=torch.int32, device=device) for n in (S + 1, S, T, T, 2)))


def kv_plan(cached_len, new_len, free_pages, page_table, page_size: int, T: int, out=None, stream=None) -> KVPlan:
    """One step's page tables and slots from the requests' lengths (moe_kv_plan): new pages are taken from
    free_pages into page_table [S][W] (in place); out: optional KVPlan to fill."""
    dev, i32 = cached_len.get_device(), torch.int32
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return kv_plan(cached_len, new_len, free_pages, page_table, page_size, T, out=out)
    S, W = page_table.shape
    a, b = _on(dev, cached_len, "cached_len", i32, (S,)), _on(dev, new_len, "new_len", i32, (S,))
    n = free_pages.numel()
    f, t = _on(dev, free_pages, "free_pages", i32, (n,)), _on(dev, page_table, "page_table", i32, (S, W))
    p = out if out is not None else KVPlan.allocate(S, T, cached_len.device)
    if (p.S, p.T, p.device) != (S, T, dev):
        raise ValueError(f"out holds {p.S} requests and {p.T} rows on device {p.device}, expected {S}, {T} on {dev}")
    rc = load().moe_kv_plan(a, b, S, f, n, page_size, T, t, W, *p.ptrs, _current(dev))
    _chk(rc, "moe_kv_plan")
    return p


def qk_norm_rope(qkv, cache: KVCache, positions, slots, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None,
                 interleaved=False, rope_scale=1.0, out=None, stream=None):
    """Head norms, rotation and cache write of the fused projection's rows qkv [T][(n_heads + 2 n_kv_heads) *
    head_dim] (moe_qk_norm_rope).  The rotated part of a head is twice inv_freq's length.  Returns q
    [T][n_heads][head_dim] (out: optional tensor to fill)."""
    dev = qkv.get_device()
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return qk_norm_rope(qkv, cache, positions, slots, q_weight, k_weight, eps, inv_freq, interleaved,
                                rope_scale, out)
    f32, i32 = torch.float32, torch.int32
    stride = _rows(qkv, "qkv", torch.bfloat16)
    T, n = qkv.shape
    D = cache.head_dim
    Hq = n // D - 2 * cache.n_kv_heads
    if n % D or Hq <= 0:
        raise ValueError(f"qkv rows of {n} elements are not (n_heads + 2 * {cache.n_kv_heads}) heads of {D}")
    if cache.device != dev:
        raise ValueError(f"the cache is on device {cache.device}, expected {dev}")
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    q = out if out is not None else torch.empty((T, Hq, D), dtype=torch.bfloat16, device=qkv.device)
    _chk(load().moe_qk_norm_rope(qkv.data_ptr(), BF16, stride, T, Hq, cache.ref,
                                 _opt(dev, q_weight, "q_weight", f32, (D,)), _opt(dev, k_weight, "k_weight", f32, (D,)),
                                 eps, _opt(dev, inv_freq, "inv_freq", f32, (R // 2,)), R, 1 if interleaved else 0, rope_scale,
                                 _on(dev, positions, "positions", i32, (T,)), _on(dev, slots, "slots", i32, (T,)),
                                 _on(dev, q, "out", torch.bfloat16, (T, Hq, D)), _current(dev)), "moe_qk_norm_rope")
    return q


def paged_attention_workspace_size(T, n_heads, n_kv_heads, head_dim, S) -> int:
    return int(load().moe_paged_attn_workspace_size(T, n_heads, n_kv_heads, head_dim, S))


def paged_attention(q, cache: KVCache, page_table, q_offsets, kv_len, scale=None, softcap=0.0, window=0, out=None,
                    workspace=None, stream=None):
    """Attention of the rows q [T][n_heads][head_dim] over their requests' cached positions (moe_paged_attn);
    scale defaults to head_dim ** -0.5.  Rows of q may lie apart.  Returns out [T][n_heads][head_dim]."""
    dev = q.get_device()
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return paged_attention(q, cache, page_table, q_offsets, kv_len, scale, softcap, window, out, workspace)
    i32 = torch.int32
    if q.dim() != 3:
        raise ValueError("q must be [T][n_heads][head_dim]")
    T, Hq, D = q.shape
    stride = Hq * D
    if not q.is_contiguous():
        if q.stride(2) != 1 or (Hq > 1 and q.stride(1) != D):
            raise ValueError("a row of q must be contiguous")
        stride = q.stride(0)
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"q must be torch.bfloat16, not {q.dtype}")
    if cache.device != dev or cache.head_dim != D:
        raise ValueError(f"the cache has heads of {cache.head_dim} on device {cache.device}, q has {D} on {dev}")
    S, W = page_table.shape
    o = out if out is not None else torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    nb = paged_attention_workspace_size(T, Hq, cache.n_kv_heads, D, S)
    ws = _bytes(dev, nb, workspace)
    _chk(load().moe_paged_attn(q.data_ptr(), BF16, stride, T, Hq, cache.ref, _on(dev, page_table, "page_table", i32, (S, W)), W,
                               _on(dev, q_offsets, "q_offsets", i32, (S + 1,)), _on(dev, kv_len, "kv_len", i32, (S,)), S,
                               D ** -0.5 if scale is None else scale, softcap, window,
                               _on(dev, o, "out", torch.bfloat16, (T, Hq, D)), ws.data_ptr(), nb,
                               _current(dev)), "moe_paged_attn")
    return o


_ACT = {None: 0, "none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def linear_workspace_size(T, N, K) -> int:
    return int(load().moe_linear_workspace_size(T, N, K))


def linear(x, w, bias=None, act=None, residual=None, out_dtype=None, out=None, workspace=None, stream=None):
    """act(x w^T + bias) + residual in one rounding (moe_linear): x [T][K] (rows may lie apart) and w [N][K]
    bfloat16, bias [N] fp32, act None, "silu", "gelu", "gelu_tanh" or "relu", residual [T][N] in the output's
    dtype (bfloat16 or float32; out may be the residual)."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return linear(x, w, bias, act, residual, out_dtype, out, workspace)
    stride = _rows(x, "x", torch.bfloat16)
    T, K = x.shape
    N = w.shape[0]
    if act not in _ACT:
        raise ValueError(f"unknown activation {act!r}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else residual.dtype if residual is not None else torch.bfloat16
    o = out if out is not None else torch.empty((T, N), dtype=out_dtype, device=x.device)
    nb = linear_workspace_size(T, N, K)
    ws = _bytes(dev, nb, workspace).data_ptr() if nb else None
    _chk(load().moe_linear(x.data_ptr(), BF16, stride, _on(dev, w, "w", torch.bfloat16, (N, K)), BF16,
                           _opt(dev, bias, "bias", torch.float32, (N,)), _ACT[act],
                           _opt(dev, residual, "residual", out_dtype, (T, N)), T, N, K,
                           _on(dev, o, "out", out_dtype, (T, N)), _act_dtype(o), ws, nb, _current(dev)), "moe_linear")
    return o


class AttentionWorkspace:
    """Preallocated buffers for repeated calls of `attention_layer` at one shape (T rows of H elements, S requests)."""

    def __init__(self, T, H, n_heads, cache: KVCache, S, device="cuda"):
        bf, D, Hkv = torch.bfloat16, cache.head_dim, cache.n_kv_heads
        n = (n_heads + 2 * Hkv) * D
        self.qkv = torch.empty((T, n), dtype=bf, device=device)
        self.q = torch.empty((T, n_heads, D), dtype=bf, device=device)
        self.o = torch.empty((T, n_heads, D), dtype=bf, device=device)
        self.out = torch.empty((T, H), dtype=bf, device=device)
        self.attn_ws = torch.empty(paged_attention_workspace_size(T, n_heads, Hkv, D, S), dtype=torch.uint8,
                                   device=device)
        self.linear_ws = torch.empty(max(linear_workspace_size(T, n, H), linear_workspace_size(T, H, n_heads * D), 1),
                                     dtype=torch.uint8, device=device)


def attention_layer(x, w_qkv, w_out, cache: KVCache, plan: KVPlan, page_table, q_weight=None, k_weight=None, eps=1e-6,
                    inv_freq=None, interleaved=False, rope_scale=1.0, b_qkv=None, b_out=None, scale=None, softcap=0.0,
                    window=0, residual=None, ws=None, stream=None, out=None):
    """The attention half of a layer on the rows x [T][H] of one step (plan: kv_plan's outputs): the fused projection
    w_qkv [(n_heads + 2 n_kv_heads) * head_dim][H], head norms + rotation + cache write, attention over the paged
    cache and the output projection w_out [H][n_heads * head_dim], added to residual [T][H] (out may be it).  Rows
    behind the step's last come out undefined.  `layer` is the other half."""
    if _elsewhere(x.get_device(), stream):
        with torch.cuda.device(x.device), torch.cuda.stream(stream):
            return attention_layer(x, w_qkv, w_out, cache, plan, page_table, q_weight, k_weight, eps, inv_freq,
                                   interleaved, rope_scale, b_qkv, b_out, scale, softcap, window, residual, ws, out=out)
    if ws is None:
        n_heads = w_qkv.shape[0] // cache.head_dim - 2 * cache.n_kv_heads
        ws = AttentionWorkspace(x.shape[0], w_out.shape[0], n_heads, cache, page_table.shape[0], device=x.device)
    linear(x, w_qkv, bias=b_qkv, out=ws.qkv, workspace=ws.linear_ws)
    qk_norm_rope(ws.qkv, cache, plan.positions, plan.slots, q_weight, k_weight, eps, inv_freq, interleaved, rope_scale,
                 out=ws.q)
    paged_attention(ws.q, cache, page_table, plan.q_offsets, plan.kv_len, scale, softcap, window, out=ws.o,
                    workspace=ws.attn_ws)
    return linear(ws.o.view(ws.o.shape[0], -1), w_out, bias=b_out, residual=residual, out=ws.out if out is None else out,
                  workspace=ws.linear_ws)

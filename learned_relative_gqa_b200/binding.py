"""Thin Python binding of ``libinkling_rel_attn.so``.

Argument marshalling only: every step of the attention runs in the library's
CUDA kernels. The functions carry the C entry points' names; tensors are
PyTorch device tensors (PyTorch supplies device memory and streams), passed
to the library as raw pointers. There is no fallback: if the library is
missing or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libinkling_rel_attn.so")

INKLING_OK = 0
INKLING_ERR_INVALID_ARG = 1
INKLING_ERR_UNSUPPORTED = 2
INKLING_ERR_MALFORMED_POSITIONS = 3
INKLING_ERR_TIMEOUT = 4
INKLING_ERR_CUDA = 5


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seq_q", "seq_k", "heads_q", "heads_kv", "head_dim", "rel_extent", "window", "query_offset")]


class FlexDims(ctypes.Structure):
    """inkling_flex_attn_dims (include/inkling_flex_attn.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in (
        "batch", "seq", "heads_q", "heads_kv", "head_dim", "mask_type", "fixed_block_size", "sliding_window",
        "eos_id", "enable_gqa")] + [("scale", ctypes.c_double)]


FLEX_MASK_TYPES = {"causal": 0, "block_causal": 1}


class L2ClipDims(ctypes.Structure):
    """inkling_l2clip_dims (include/inkling_l2clip.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "seq", "heads", "head_dim")] + [("threshold", ctypes.c_double)]


class KVCacheDesc(ctypes.Structure):
    """inkling_kv_cache_desc (include/inkling_paged_attn.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in (
        "num_pages", "page_size", "heads_kv", "head_dim", "dtype", "page_stride", "token_stride", "head_stride")]


KV_DTYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


class KVPlanDims(ctypes.Structure):
    """inkling_kv_plan_dims (include/inkling_paged_attn.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("requests", "page_size", "max_pages", "num_pages", "max_tokens")]


class KVAppendDims(ctypes.Structure):
    """inkling_kv_append_dims (include/inkling_paged_attn.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("tokens", "k_row", "v_row", "clip_k")] + [("threshold", ctypes.c_double)]


class DecodeDims(ctypes.Structure):
    """inkling_rel_attn_decode_dims (include/inkling_paged_attn.h)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("requests", "heads_q", "rel_extent", "window", "max_pages")] + [
        ("scale", ctypes.c_double)]


class InklingError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {status_string(status)} (status {status})"
        if status == INKLING_ERR_CUDA:
            msg += f": {load().inkling_rel_attn_last_cuda_error().decode()}"
        super().__init__(msg)


_lib = None


def load(path: str = LIB_PATH):
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{os.path.basename(path)} is not built; run python -m learned_relative_gqa_b200.build")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    dp = ctypes.POINTER(Dims)
    lib.inkling_rel_attn_workspace_size.restype = sz
    lib.inkling_rel_attn_workspace_size.argtypes = [dp, ctypes.c_int]
    lib.inkling_rel_attn_validate.restype = ctypes.c_int
    lib.inkling_rel_attn_validate.argtypes = [dp, vp, vp, vp, vp, vp, sz, vp]
    lib.inkling_rel_attn_fwd.restype = ctypes.c_int
    lib.inkling_rel_attn_fwd.argtypes = [dp] + [vp] * 11 + [vp, sz, vp]
    lib.inkling_rel_attn_bwd.restype = ctypes.c_int
    lib.inkling_rel_attn_bwd.argtypes = [dp] + [vp] * 18 + [vp, sz, vp]
    lib.inkling_rel_attn_fwd_noalloc.restype = ctypes.c_int
    lib.inkling_rel_attn_fwd_noalloc.argtypes = [dp] + [vp] * 11 + [vp]
    lib.inkling_rel_attn_fwd_noalloc_last_device_error.restype = ctypes.c_int
    lib.inkling_rel_attn_fwd_noalloc_last_device_error.argtypes = [vp]
    lib.inkling_rel_attn_merge.restype = ctypes.c_int
    lib.inkling_rel_attn_merge.argtypes = [ctypes.c_int64, ctypes.c_int64, vp, vp, vp, vp, vp]
    lib.inkling_rel_attn_last_device_error.restype = ctypes.c_int
    lib.inkling_rel_attn_last_device_error.argtypes = [vp, vp]
    lib.inkling_rel_attn_selftest_exp2.restype = ctypes.c_int
    lib.inkling_rel_attn_selftest_exp2.argtypes = [vp, vp, ctypes.c_int64, vp]
    lib.inkling_rel_attn_selftest_wait_timeout.restype = ctypes.c_int
    lib.inkling_rel_attn_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp, sz, vp]
    lib.inkling_rel_attn_set_wait_timeout_ns.restype = ctypes.c_int
    lib.inkling_rel_attn_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.inkling_rel_attn_set_timing_events.restype = ctypes.c_int
    lib.inkling_rel_attn_set_timing_events.argtypes = [vp, ctypes.c_int]
    fd = ctypes.POINTER(FlexDims)
    lib.inkling_flex_attn_workspace_size.restype = sz
    lib.inkling_flex_attn_workspace_size.argtypes = [fd, ctypes.c_int]
    lib.inkling_flex_attn_fwd.restype = ctypes.c_int
    lib.inkling_flex_attn_fwd.argtypes = [fd] + [vp] * 7 + [vp, sz, vp]
    lib.inkling_flex_attn_bwd.restype = ctypes.c_int
    lib.inkling_flex_attn_bwd.argtypes = [fd] + [vp] * 12 + [vp, sz, vp]
    ld = ctypes.POINTER(L2ClipDims)
    lib.inkling_l2clip_workspace_size.restype = sz
    lib.inkling_l2clip_workspace_size.argtypes = [ld]
    lib.inkling_l2clip_fwd.restype = ctypes.c_int
    lib.inkling_l2clip_fwd.argtypes = [ld] + [vp] * 4 + [vp]
    lib.inkling_l2clip_bwd.restype = ctypes.c_int
    lib.inkling_l2clip_bwd.argtypes = [ld] + [vp] * 7 + [vp, sz, vp]
    lib.inkling_rel_attn_qclip_workspace_size.restype = sz
    lib.inkling_rel_attn_qclip_workspace_size.argtypes = [dp, ctypes.c_int]
    lib.inkling_rel_attn_fwd_qclip.restype = ctypes.c_int
    lib.inkling_rel_attn_fwd_qclip.argtypes = [dp, ctypes.c_double] + [vp] * 14 + [vp, sz, vp]
    lib.inkling_rel_attn_bwd_qclip.restype = ctypes.c_int
    lib.inkling_rel_attn_bwd_qclip.argtypes = [dp, ctypes.c_double] + [vp] * 23 + [vp, sz, vp]
    cd = ctypes.POINTER(KVCacheDesc)
    lib.inkling_kv_plan.restype = ctypes.c_int
    lib.inkling_kv_plan.argtypes = [ctypes.POINTER(KVPlanDims)] + [vp] * 10 + [vp]
    lib.inkling_kv_append.restype = ctypes.c_int
    lib.inkling_kv_append.argtypes = [cd, ctypes.POINTER(KVAppendDims)] + [vp] * 9 + [vp]
    ed = ctypes.POINTER(DecodeDims)
    lib.inkling_rel_attn_decode_workspace_size.restype = sz
    lib.inkling_rel_attn_decode_workspace_size.argtypes = [cd, ed]
    lib.inkling_rel_attn_decode.restype = ctypes.c_int
    lib.inkling_rel_attn_decode.argtypes = [cd, ed] + [vp] * 11 + [vp, sz, vp]
    lib.inkling_rel_attn_last_cuda_error.restype = ctypes.c_char_p
    lib.inkling_rel_attn_last_cuda_error.argtypes = []
    lib.inkling_status_string.restype = ctypes.c_char_p
    lib.inkling_status_string.argtypes = [ctypes.c_int]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().inkling_status_string(int(status)).decode()


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_dims(q: torch.Tensor, k: torch.Tensor, profiles: Optional[torch.Tensor], window: int,
              query_offset: int = 0, rel_extent: Optional[int] = None) -> Dims:
    B, S, Hq, D = q.shape
    Skv, Hkv = k.shape[1], k.shape[2]
    R = profiles.shape[3] if profiles is not None else int(rel_extent or 0)
    return Dims(B, S, Skv, Hq, Hkv, D, R, int(window), int(query_offset))


def inkling_rel_attn_workspace_size(dims: Dims, backward: bool) -> int:
    return int(load().inkling_rel_attn_workspace_size(ctypes.byref(dims), int(bool(backward))))


def alloc_workspace(dims: Dims, backward: bool, device) -> torch.Tensor:
    n = inkling_rel_attn_workspace_size(dims, backward)
    if n == 0:
        raise InklingError(INKLING_ERR_INVALID_ARG, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _u8(t):
    return None if t is None else (t if t.dtype == torch.uint8 else t.view(torch.uint8) if t.dtype == torch.bool
                                   else t.to(torch.uint8))


def _check(status: int, where: str):
    if status != INKLING_OK:
        raise InklingError(status, where)


def inkling_rel_attn_validate(dims: Dims, valid, key_valid, positions, key_positions, workspace,
                              stream=None) -> int:
    """Returns the library status (INKLING_OK or INKLING_ERR_MALFORMED_POSITIONS, ...)."""
    return int(load().inkling_rel_attn_validate(
        ctypes.byref(dims), _p(_u8(valid)), _p(_u8(key_valid)), _p(positions), _p(key_positions),
        _p(workspace), workspace.numel(), _stream(stream)))


def inkling_rel_attn_fwd(dims: Dims, q, k, v, profiles, sink, valid, key_valid, positions, key_positions,
                         out, lse, workspace, stream=None) -> None:
    st = load().inkling_rel_attn_fwd(
        ctypes.byref(dims), _p(q), _p(k), _p(v), _p(profiles), _p(sink), _p(_u8(valid)), _p(_u8(key_valid)),
        _p(positions), _p(key_positions), _p(out), _p(lse), _p(workspace), workspace.numel(), _stream(stream))
    _check(st, "inkling_rel_attn_fwd")


def inkling_rel_attn_bwd(dims: Dims, q, k, v, profiles, sink, valid, key_valid, positions, key_positions,
                         out, lse, dout, dlse, dq, dk, dv, dprofiles, dsink, workspace, stream=None) -> None:
    st = load().inkling_rel_attn_bwd(
        ctypes.byref(dims), _p(q), _p(k), _p(v), _p(profiles), _p(sink), _p(_u8(valid)), _p(_u8(key_valid)),
        _p(positions), _p(key_positions), _p(out), _p(lse), _p(dout), _p(dlse), _p(dq), _p(dk), _p(dv),
        _p(dprofiles), _p(dsink), _p(workspace), workspace.numel(), _stream(stream))
    _check(st, "inkling_rel_attn_bwd")


def inkling_rel_attn_fwd_noalloc(dims: Dims, q, k, v, profiles, sink, valid, key_valid, positions, key_positions,
                                 out, lse, stream=None) -> int:
    """Forward that uses the library's own static device scratch instead of a workspace.

    For callers that cannot allocate device memory. Returns the library status
    (INKLING_ERR_UNSUPPORTED when the problem needs more than the 4 MiB of scratch).
    """
    return int(load().inkling_rel_attn_fwd_noalloc(
        ctypes.byref(dims), _p(q), _p(k), _p(v), _p(profiles), _p(sink), _p(_u8(valid)), _p(_u8(key_valid)),
        _p(positions), _p(key_positions), _p(out), _p(lse), _stream(stream)))


def inkling_rel_attn_merge(out, lse, out_part, lse_part, stream=None) -> None:
    """Merges (out_part, lse_part), a result over a disjoint key set, into (out, lse) in place."""
    for t in (out, lse, out_part, lse_part):
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
            raise ValueError("inkling_rel_attn_merge: contiguous float32 CUDA tensors expected")
    if out.shape != out_part.shape or lse.shape != lse_part.shape or out.shape[:-1] != lse.shape:
        raise ValueError("inkling_rel_attn_merge: shape mismatch")
    _check(load().inkling_rel_attn_merge(int(lse.numel()), int(out.shape[-1]), _p(out), _p(lse), _p(out_part),
                                         _p(lse_part), _stream(stream)), "inkling_rel_attn_merge")


def inkling_rel_attn_fwd_noalloc_last_device_error(stream=None) -> int:
    """Reads and clears the device error word of the no-allocation forward (synchronous)."""
    return int(load().inkling_rel_attn_fwd_noalloc_last_device_error(_stream(stream)))


def inkling_rel_attn_last_device_error(workspace, stream=None) -> int:
    return int(load().inkling_rel_attn_last_device_error(_p(workspace), _stream(stream)))


def inkling_rel_attn_selftest_wait_timeout(timeout_us: int, workspace, stream=None) -> int:
    return int(load().inkling_rel_attn_selftest_wait_timeout(int(timeout_us), _p(workspace), workspace.numel(),
                                                             _stream(stream)))


def inkling_rel_attn_set_wait_timeout_ns(timeout_ns: int) -> None:
    """Limit of the attention kernels' pipeline waits for later calls (0 = default)."""
    _check(load().inkling_rel_attn_set_wait_timeout_ns(int(timeout_ns)), "inkling_rel_attn_set_wait_timeout_ns")


def inkling_rel_attn_selftest_exp2(t, out, stream=None) -> None:
    """t, out: contiguous float32 CUDA tensors of the same size."""
    _check(load().inkling_rel_attn_selftest_exp2(_p(t), _p(out), int(t.numel()), _stream(stream)),
           "inkling_rel_attn_selftest_exp2")


def inkling_rel_attn_set_timing_events(events, n_pairs: int) -> None:
    """events: a ctypes array of cudaEvent_t handles (or None to switch the hook off)."""
    _check(load().inkling_rel_attn_set_timing_events(events, int(n_pairs)), "inkling_rel_attn_set_timing_events")


# --------------------------------------------------------------------------
# convenience wrappers (allocate outputs with torch, then call the entry points)
# --------------------------------------------------------------------------
def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def forward(q, k, v, profiles, sink, valid, key_valid=None, positions=None, key_positions=None, *,
            window: int = 0, query_offset: int = 0, workspace=None, stream=None):
    """out [B,S,Hq,D] fp32 and lse [B,S,Hq] fp32 (see include/inkling_rel_attn.h)."""
    _contig(q, k, v, profiles, sink, valid, key_valid, positions, key_positions)
    dims = make_dims(q, k, profiles, window, query_offset)
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    ws = alloc_workspace(dims, False, q.device) if workspace is None else workspace
    inkling_rel_attn_fwd(dims, q, k, v, profiles, sink, valid, key_valid, positions, key_positions, out, lse, ws,
                         stream)
    return out, lse


def backward(q, k, v, profiles, sink, valid, key_valid, positions, key_positions, out, lse, dout, dlse=None, *,
             window: int = 0, query_offset: int = 0, workspace=None, stream=None):
    """dict dq, dk, dv, dprofiles, dsink (fp32)."""
    _contig(q, k, v, profiles, sink, valid, key_valid, positions, key_positions, out, lse, dout, dlse)
    dims = make_dims(q, k, profiles, window, query_offset)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty(q.shape, **f32)
    dk = torch.empty(k.shape, **f32)
    dv = torch.empty(v.shape, **f32)
    dprof = torch.empty(profiles.shape, **f32)
    dsink = torch.empty(sink.shape, **f32)
    ws = alloc_workspace(dims, True, q.device) if workspace is None else workspace
    inkling_rel_attn_bwd(dims, q, k, v, profiles, sink, valid, key_valid, positions, key_positions, out, lse, dout,
                         dlse, dq, dk, dv, dprof, dsink, ws, stream)
    return dict(dq=dq, dk=dk, dv=dv, dprofiles=dprof, dsink=dsink)


# --------------------------------------------------------------------------
# L2Clip of q fused into the attention (include/inkling_l2clip.h, *_qclip)
# --------------------------------------------------------------------------
def forward_qclip(x, k, v, profiles, sink, valid, key_valid=None, positions=None, key_positions=None, *,
                  threshold: float, clip_scale=None, tau=None, window: int = 0, query_offset: int = 0,
                  workspace=None, stream=None):
    """out [B,S,Hq,D] fp32, lse [B,S,Hq] fp32 and the clipped q [B,S,Hq,D] BF16 of the
    attention with q = L2Clip(x) computed inside the kernels."""
    _contig(x, k, v, profiles, sink, valid, key_valid, positions, key_positions, clip_scale, tau)
    dims = make_dims(x, k, profiles, window, query_offset)
    out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    lse = torch.empty(x.shape[:3], dtype=torch.float32, device=x.device)
    qc = torch.empty_like(x)
    if workspace is None:
        workspace = torch.empty(max(int(load().inkling_rel_attn_qclip_workspace_size(ctypes.byref(dims), 0)), 256),
                                dtype=torch.uint8, device=x.device)
    st = load().inkling_rel_attn_fwd_qclip(
        ctypes.byref(dims), float(threshold), _p(clip_scale), _p(tau), _p(x), _p(k), _p(v), _p(profiles), _p(sink),
        _p(_u8(valid)), _p(_u8(key_valid)), _p(positions), _p(key_positions), _p(qc), _p(out), _p(lse),
        _p(workspace), workspace.numel(), _stream(stream))
    _check(st, "inkling_rel_attn_fwd_qclip")
    return out, lse, qc


def backward_qclip(x, q_clipped, k, v, profiles, sink, valid, key_valid, positions, key_positions, out, lse, dout,
                   dlse=None, *, threshold: float, clip_scale=None, tau=None, window: int = 0, query_offset: int = 0,
                   workspace=None, stream=None):
    """dict dx (gradient of the unclipped q), dk, dv, dprofiles, dsink, dclip_scale, dtau (fp32;
    the last two None without their parameters)."""
    _contig(x, q_clipped, k, v, profiles, sink, valid, key_valid, positions, key_positions, out, lse, dout, dlse,
            clip_scale, tau)
    dims = make_dims(x, k, profiles, window, query_offset)
    f32 = dict(dtype=torch.float32, device=x.device)
    g = dict(dx=torch.empty(x.shape, **f32), dk=torch.empty(k.shape, **f32), dv=torch.empty(v.shape, **f32),
             dprofiles=torch.empty(profiles.shape, **f32), dsink=torch.empty(sink.shape, **f32),
             dclip_scale=None if clip_scale is None else torch.empty(clip_scale.shape, **f32),
             dtau=None if tau is None else torch.empty(tau.shape, **f32))
    if workspace is None:
        workspace = torch.empty(int(load().inkling_rel_attn_qclip_workspace_size(ctypes.byref(dims), 1)),
                                dtype=torch.uint8, device=x.device)
    st = load().inkling_rel_attn_bwd_qclip(
        ctypes.byref(dims), float(threshold), _p(clip_scale), _p(tau), _p(x), _p(q_clipped), _p(k), _p(v),
        _p(profiles), _p(sink), _p(_u8(valid)), _p(_u8(key_valid)), _p(positions), _p(key_positions), _p(out),
        _p(lse), _p(dout), _p(dlse), _p(g["dx"]), _p(g["dk"]), _p(g["dv"]), _p(g["dprofiles"]), _p(g["dsink"]),
        _p(g["dclip_scale"]), _p(g["dtau"]), _p(workspace), workspace.numel(), _stream(stream))
    _check(st, "inkling_rel_attn_bwd_qclip")
    return g


# --------------------------------------------------------------------------
# generic FlexAttention variant (include/inkling_flex_attn.h)
# --------------------------------------------------------------------------
def make_flex_dims(q: torch.Tensor, k: torch.Tensor, *, mask_type: str = "causal", eos_id: int = 0,
                   fixed_block_size: int = 0, sliding_window: int = 0, scale: Optional[float] = None,
                   enable_gqa: bool = False) -> FlexDims:
    B, Hq, S, D = q.shape
    if mask_type not in FLEX_MASK_TYPES:
        raise ValueError(f"mask_type must be one of {sorted(FLEX_MASK_TYPES)}")
    return FlexDims(B, S, Hq, k.shape[1], D, FLEX_MASK_TYPES[mask_type], int(fixed_block_size), int(sliding_window),
                    int(eos_id), int(bool(enable_gqa)), 0.0 if scale is None else float(scale))


def inkling_flex_attn_workspace_size(dims: FlexDims, backward: bool) -> int:
    return int(load().inkling_flex_attn_workspace_size(ctypes.byref(dims), int(bool(backward))))


def inkling_flex_attn_fwd(dims: FlexDims, q, k, v, sink_weights, tokens, out, lse, workspace, stream=None) -> None:
    st = load().inkling_flex_attn_fwd(ctypes.byref(dims), _p(q), _p(k), _p(v), _p(sink_weights), _p(tokens), _p(out),
                                      _p(lse), _p(workspace), workspace.numel(), _stream(stream))
    _check(st, "inkling_flex_attn_fwd")


def inkling_flex_attn_bwd(dims: FlexDims, q, k, v, sink_weights, tokens, out, lse, dout, dq, dk, dv, dsink_weights,
                          workspace, stream=None) -> None:
    st = load().inkling_flex_attn_bwd(ctypes.byref(dims), _p(q), _p(k), _p(v), _p(sink_weights), _p(tokens),
                                      _p(out), _p(lse), _p(dout), _p(dq), _p(dk), _p(dv), _p(dsink_weights),
                                      _p(workspace), workspace.numel(), _stream(stream))
    _check(st, "inkling_flex_attn_bwd")


def _flex_ws(dims: FlexDims, backward: bool, device) -> torch.Tensor:
    n = inkling_flex_attn_workspace_size(dims, backward)
    if n == 0:
        raise InklingError(INKLING_ERR_INVALID_ARG, "inkling_flex_attn_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def flex_forward(q, k, v, sink_weights=None, tokens=None, *, mask_type: str = "causal", eos_id: int = 0,
                 fixed_block_size: int = 0, sliding_window: int = 0, scale: Optional[float] = None,
                 enable_gqa: bool = False, workspace=None, stream=None):
    """out [B,Hq,S,D] BF16 and lse [B,Hq,S] FP32 (see include/inkling_flex_attn.h)."""
    _contig(q, k, v, sink_weights, tokens)
    dims = make_flex_dims(q, k, mask_type=mask_type, eos_id=eos_id, fixed_block_size=fixed_block_size,
                          sliding_window=sliding_window, scale=scale, enable_gqa=enable_gqa)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    ws = _flex_ws(dims, False, q.device) if workspace is None else workspace
    inkling_flex_attn_fwd(dims, q, k, v, sink_weights, tokens, out, lse, ws, stream)
    return out, lse


def flex_backward(q, k, v, out, lse, dout, sink_weights=None, tokens=None, *, mask_type: str = "causal",
                  eos_id: int = 0, fixed_block_size: int = 0, sliding_window: int = 0,
                  scale: Optional[float] = None, enable_gqa: bool = False, workspace=None, stream=None):
    """dict dq [B,Hq,S,D], dk / dv [B,Hkv,S,D] and dsink_weights [Hq] (None without sinks), FP32."""
    _contig(q, k, v, out, lse, dout, sink_weights, tokens)
    dims = make_flex_dims(q, k, mask_type=mask_type, eos_id=eos_id, fixed_block_size=fixed_block_size,
                          sliding_window=sliding_window, scale=scale, enable_gqa=enable_gqa)
    f32 = dict(dtype=torch.float32, device=q.device)
    dq = torch.empty(q.shape, **f32)
    dk = torch.empty(k.shape, **f32)
    dv = torch.empty(v.shape, **f32)
    dsw = None if sink_weights is None else torch.empty(sink_weights.shape, **f32)
    ws = _flex_ws(dims, True, q.device) if workspace is None else workspace
    inkling_flex_attn_bwd(dims, q, k, v, sink_weights, tokens, out, lse, dout, dq, dk, dv, dsw, ws, stream)
    return dict(dq=dq, dk=dk, dv=dv, dsink_weights=dsw)


# --------------------------------------------------------------------------
# L2Clip (include/inkling_l2clip.h)
# --------------------------------------------------------------------------
def make_l2clip_dims(x: torch.Tensor, threshold: float) -> L2ClipDims:
    B, S, H, D = x.shape
    return L2ClipDims(B, S, H, D, float(threshold))


def inkling_l2clip_workspace_size(dims: L2ClipDims) -> int:
    return int(load().inkling_l2clip_workspace_size(ctypes.byref(dims)))


def inkling_l2clip_fwd(dims: L2ClipDims, x, scale, tau, y, stream=None) -> None:
    _check(load().inkling_l2clip_fwd(ctypes.byref(dims), _p(x), _p(scale), _p(tau), _p(y), _stream(stream)),
           "inkling_l2clip_fwd")


def inkling_l2clip_bwd(dims: L2ClipDims, x, scale, tau, dy, dx, dscale, dtau, workspace, stream=None) -> None:
    _check(load().inkling_l2clip_bwd(ctypes.byref(dims), _p(x), _p(scale), _p(tau), _p(dy), _p(dx), _p(dscale),
                                     _p(dtau), _p(workspace), workspace.numel(), _stream(stream)),
           "inkling_l2clip_bwd")


def l2clip_forward(x, threshold: float, scale=None, tau=None, stream=None):
    """y [B,S,H,D] BF16: x (BF16) clipped per head vector (see include/inkling_l2clip.h)."""
    _contig(x, scale, tau)
    dims = make_l2clip_dims(x, threshold)
    y = torch.empty_like(x)
    inkling_l2clip_fwd(dims, x, scale, tau, y, stream)
    return y


def l2clip_backward(x, dy, threshold: float, scale=None, tau=None, stream=None):
    """dict dx [B,S,H,D], dscale [H,D] (None without scale), dtau [B,S] (None without tau), FP32."""
    _contig(x, dy, scale, tau)
    dims = make_l2clip_dims(x, threshold)
    f32 = dict(dtype=torch.float32, device=x.device)
    dx = torch.empty(x.shape, **f32)
    dscale = None if scale is None else torch.empty(scale.shape, **f32)
    dtau = None if tau is None else torch.empty(tau.shape, **f32)
    n = inkling_l2clip_workspace_size(dims)
    if n == 0:
        raise InklingError(INKLING_ERR_INVALID_ARG, "inkling_l2clip_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    inkling_l2clip_bwd(dims, x, scale, tau, dy, dx, dscale, dtau, ws, stream)
    return dict(dx=dx, dscale=dscale, dtau=dtau)


# --------------------------------------------------------------------------
# serving: paged key-value cache and single-token attention (include/inkling_paged_attn.h)
# --------------------------------------------------------------------------
def _on_device(device, **tensors):
    """ValueError unless every given (tensor, dtype) is contiguous, of that dtype and on `device`."""
    for name, (t, dtype) in tensors.items():
        if t is None:
            continue
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _shape(name, t, *want):
    if t is not None and tuple(t.shape) != want:
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")


def _allocating_on(stream):
    """Tensors allocated inside belong to `stream` (None: the current one), so that one that is
    dropped when a call returns is not reused before that stream is done with it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _stream_on(device, stream):
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"the stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def make_kv_cache_desc(k_cache: torch.Tensor, v_cache: torch.Tensor) -> KVCacheDesc:
    """Descriptor of two pools [num_pages, page_size, heads_kv, head_dim] (any strides, D contiguous)."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, heads_kv, head_dim] of one shape and dtype")
    if k_cache.dtype not in KV_DTYPES:
        raise ValueError(f"a cache is bfloat16 or float8_e4m3fn, got {k_cache.dtype}")
    if not k_cache.is_cuda or k_cache.device != v_cache.device:
        raise ValueError("k_cache and v_cache must be on one CUDA device")
    ks = k_cache.stride()
    if ks != v_cache.stride() or ks[3] != 1:
        raise ValueError("k_cache and v_cache must have the same strides, head_dim contiguous")
    return KVCacheDesc(*k_cache.shape, KV_DTYPES[k_cache.dtype], ks[0], ks[1], ks[2])


def _kv_scales(cache: torch.Tensor, k_scale, v_scale):
    quantised = cache.dtype == torch.float8_e4m3fn
    for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
        if (s is not None) != quantised:
            raise ValueError(f"{name}: an e4m3 cache needs its scales, a bfloat16 cache takes none")
        _shape(name, s, cache.shape[2])
    _on_device(cache.device, k_scale=(k_scale, torch.float32), v_scale=(v_scale, torch.float32))


def inkling_kv_plan(dims: KVPlanDims, old_lens, new_lens, block_table, free_pages, free_count, lens, query_start,
                    slots, positions, info, stream=None) -> None:
    with torch.cuda.device(block_table.device):
        st = load().inkling_kv_plan(
            ctypes.byref(dims), _p(old_lens), _p(new_lens), _p(block_table), _p(free_pages), _p(free_count), _p(lens),
            _p(query_start), _p(slots), _p(positions), _p(info), _stream_on(block_table.device, stream))
    _check(st, "inkling_kv_plan")


def inkling_kv_append(cache: KVCacheDesc, dims: KVAppendDims, k, v, slots, k_scale, v_scale, clip_scale, tau, k_cache,
                      v_cache, stream=None) -> None:
    with torch.cuda.device(k_cache.device):
        st = load().inkling_kv_append(
            ctypes.byref(cache), ctypes.byref(dims), _p(k), _p(v), _p(slots), _p(k_scale), _p(v_scale),
            _p(clip_scale), _p(tau), _p(k_cache), _p(v_cache), _stream_on(k_cache.device, stream))
    _check(st, "inkling_kv_append")


def inkling_rel_attn_decode_workspace_size(cache: KVCacheDesc, dims: DecodeDims) -> int:
    return int(load().inkling_rel_attn_decode_workspace_size(ctypes.byref(cache), ctypes.byref(dims)))


def alloc_decode_workspace(cache: KVCacheDesc, dims: DecodeDims, device) -> torch.Tensor:
    n = inkling_rel_attn_decode_workspace_size(cache, dims)
    if n == 0:
        raise InklingError(INKLING_ERR_INVALID_ARG, "inkling_rel_attn_decode_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def inkling_rel_attn_decode(cache: KVCacheDesc, dims: DecodeDims, q, k_cache, v_cache, k_scale, v_scale, profiles,
                            sink, block_table, lens, out, lse, workspace, stream=None) -> None:
    with torch.cuda.device(k_cache.device):
        st = load().inkling_rel_attn_decode(
            ctypes.byref(cache), ctypes.byref(dims), _p(q), _p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale),
            _p(profiles), _p(sink), _p(block_table), _p(lens), _p(out), _p(lse), _p(workspace), workspace.numel(),
            _stream_on(k_cache.device, stream))
    _check(st, "inkling_rel_attn_decode")


def kv_plan(old_lens, new_lens, block_table, free_pages, free_count, *, page_size: int, num_pages: int,
            max_tokens: int, stream=None):
    """Pages and slots of a serving step, from the requests' lengths before and after it.

    ``old_lens``, ``new_lens`` [N], ``block_table`` [N, M], ``free_pages`` [num_pages] and
    ``free_count`` [1] are int32 on one device; ``block_table`` and ``free_pages`` are updated
    in place. Returns a dict: ``lens`` [N] (tokens that have a page), ``query_start`` [N + 1],
    ``slots`` [max_tokens] int64, ``positions`` [max_tokens] and ``info`` [4] (pages free
    afterwards, new tokens, pages short, pages taken). ``info[:1]`` is the next call's
    ``free_count`` (see include/inkling_paged_attn.h).
    """
    device, i32 = block_table.device, torch.int32
    if block_table.dim() != 2 or not block_table.is_cuda:
        raise ValueError("block_table must be a CUDA tensor [requests, max_pages]")
    N, M = block_table.shape
    _on_device(device, block_table=(block_table, i32), old_lens=(old_lens, i32), new_lens=(new_lens, i32),
               free_pages=(free_pages, i32), free_count=(free_count, i32))
    _shape("old_lens", old_lens, N)
    _shape("new_lens", new_lens, N)
    _shape("free_pages", free_pages, int(num_pages))
    _shape("free_count", free_count, 1)
    dims = KVPlanDims(N, int(page_size), M, int(num_pages), int(max_tokens))
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    # one allocation for the four int32 outputs, each at a multiple of 16 bytes
    up = lambda n: (n + 3) // 4 * 4  # noqa: E731
    at = [0, up(N), up(N) + up(N + 1), up(N) + up(N + 1) + up(max_tokens)]
    with _allocating_on(stream):
        small = torch.empty(at[3] + 4, dtype=i32, device=device)
        slots = torch.empty(max_tokens, dtype=torch.int64, device=device)
    lens, query_start = small[:N], small[at[1]:at[1] + N + 1]
    positions, info = small[at[2]:at[2] + max_tokens], small[at[3]:]
    inkling_kv_plan(dims, old_lens, new_lens, block_table, free_pages, free_count, lens, query_start, slots, positions,
                    info, stream)
    return dict(lens=lens, query_start=query_start, slots=slots, positions=positions, info=info)


def kv_append(k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, threshold: Optional[float] = None,
              clip_scale=None, tau=None, stream=None) -> None:
    """Writes ``k``, ``v`` [T, Hkv, D] BF16 into the slots [T] (int64; outside the pool: skipped) of the pools.

    The rows may be slices of a wider projection (the token stride is free, heads and
    values dense). With a ``threshold``, k goes through L2Clip (``clip_scale`` [Hkv, D],
    ``tau`` [T]) on the way; an e4m3 cache takes ``k_scale``, ``v_scale`` [Hkv].
    """
    desc = make_kv_cache_desc(k_cache, v_cache)
    device = k_cache.device
    _, _, H, D = k_cache.shape
    T = slots.numel()
    for name, x in (("k", k), ("v", v)):
        _shape(name, x, T, H, D)
        if x.device != device or x.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16 on {device}")
        s = x.stride()
        if T > 0 and ((D > 1 and s[2] != 1) or (H > 1 and s[1] != D)):
            raise ValueError(f"{name} must have dense heads and values")
    _shape("slots", slots, T)
    _on_device(device, slots=(slots, torch.int64), clip_scale=(clip_scale, torch.float32), tau=(tau, torch.float32))
    _shape("clip_scale", clip_scale, H, D)
    _shape("tau", tau, T)
    _kv_scales(k_cache, k_scale, v_scale)
    if threshold is None and (clip_scale is not None or tau is not None):
        raise ValueError("clip_scale and tau need a threshold")
    one = H * D  # the stride of a single row means nothing
    dims = KVAppendDims(T, k.stride(0) if T > 1 else one, v.stride(0) if T > 1 else one, int(threshold is not None),
                        0.0 if threshold is None else float(threshold))
    inkling_kv_append(desc, dims, k, v, slots, k_scale, v_scale, clip_scale, tau, k_cache, v_cache, stream)


def paged_decode(q, k_cache, v_cache, block_table, lens, profiles=None, sink=None, *, window: int = 0,
                 scale: Optional[float] = None, k_scale=None, v_scale=None, workspace=None, stream=None):
    """out [N,Hq,D] and lse [N,Hq] (fp32) of each request's newest token over its cached tokens.

    ``q`` [N,Hq,D] BF16, pools [num_pages, page_size, Hkv, D] BF16 or e4m3 (then with
    ``k_scale``, ``v_scale`` [Hkv]), ``block_table`` [N,M] int32, ``lens`` [N] int32 with the
    new token counted (0: a padding row), ``profiles`` [N,Hq,R] BF16, ``sink`` [N,Hq] fp32
    (see include/inkling_paged_attn.h).
    """
    desc = make_kv_cache_desc(k_cache, v_cache)
    device = k_cache.device
    if q.dim() != 3 or q.shape[2] != k_cache.shape[3]:
        raise ValueError("q must be [requests, heads_q, head_dim] with the cache's head_dim")
    N, Hq, D = q.shape
    if block_table.dim() != 2:
        raise ValueError("block_table must be [requests, max_pages]")
    M = block_table.shape[1]
    R = 0
    if profiles is not None:
        if profiles.dim() != 3:
            raise ValueError("profiles must be [requests, heads_q, rel_extent]")
        R = profiles.shape[2]
        _shape("profiles", profiles, N, Hq, R)
    _shape("block_table", block_table, N, M)
    _shape("lens", lens, N)
    _shape("sink", sink, N, Hq)
    _on_device(device, q=(q, torch.bfloat16), block_table=(block_table, torch.int32), lens=(lens, torch.int32),
               profiles=(profiles, torch.bfloat16), sink=(sink, torch.float32),
               workspace=(workspace, torch.uint8))
    _kv_scales(k_cache, k_scale, v_scale)
    dims = DecodeDims(N, Hq, R, int(window), M, 0.0 if scale is None else float(scale))
    with _allocating_on(stream):
        if workspace is None:
            n = inkling_rel_attn_decode_workspace_size(desc, dims)
            workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
        out = torch.empty(q.shape, dtype=torch.float32, device=device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=device)
    inkling_rel_attn_decode(desc, dims, q, k_cache, v_cache, k_scale, v_scale, profiles if R else None, sink,
                            block_table, lens, out, lse, workspace, stream)
    return out, lse

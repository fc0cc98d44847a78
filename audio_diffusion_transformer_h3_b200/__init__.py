"""Python binding of libh3attn (include/h3attn.h).

Argument marshalling only: every step of the path runs in the CUDA library.
PyTorch supplies device memory and the current stream. The functions keep
the C names; the ``*_t`` helpers take torch tensors and call the same entry
points with their pointers.

The library is loaded from this directory (built in-tree by
``python audio_diffusion_transformer_h3_b200/build.py`` or
``__graft_entry__.build()``). There is no fallback: if it is missing or does
not load, importing this package raises.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libh3attn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python audio_diffusion_transformer_h3_b200/build.py` (nvcc, sm_100a)")
_lib = ctypes.CDLL(LIB_PATH)

# ----------------------------------------------------------------- C types

H3_OK = 0
H3_ERR_INVALID_ARG = 1
H3_ERR_UNSUPPORTED = 2
H3_ERR_MISALIGNED = 3
H3_ERR_WORKSPACE = 4
H3_ERR_CUDA = 5
H3_ERR_DEVICE_TIMEOUT = 6
H3_ERR_BAD_SEQLENS = 7


class h3_rope_cfg(ctypes.Structure):
    _fields_ = [("d_t", ctypes.c_int32), ("d_h", ctypes.c_int32), ("d_w", ctypes.c_int32),
                ("theta", ctypes.c_float)]


class h3_segment_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "image_refs", "image_h", "image_w", "audio_refs", "audio_ref_len", "audio_rate",
        "video_t", "video_h", "video_w", "audio_tail")]


class h3_rope_qk_cfg(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("attn_factor", ctypes.c_double)]


H3_BF16, H3_FP16, H3_FP32 = 0, 1, 2
H3_ROPE_INTERLEAVED, H3_ROPE_HALF = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "turns": 3, "yarn": 4}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
H3_ACT_GATED = 256

_c = ctypes
_P = _c.c_void_p
_lib.h3_segment_tokens.argtypes = [_c.POINTER(h3_segment_layout)]
_lib.h3_segment_tokens.restype = _c.c_int64
_lib.h3_build_positions.argtypes = [_c.POINTER(h3_segment_layout), _c.c_int32, _P, _c.c_int64, _P]
_lib.h3_build_positions.restype = _c.c_int
_lib.h3_build_positions_at.argtypes = [_c.POINTER(h3_segment_layout), _c.c_int32, _P, _P,
                                       _c.c_int64, _P]
_lib.h3_build_positions_at.restype = _c.c_int
_lib.h3_rope_apply.argtypes = [_P, _P, _P, _c.c_int64, _c.c_int32, _c.c_int32, h3_rope_cfg, _P]
_lib.h3_rope_apply.restype = _c.c_int
_lib.h3_workspace_size.argtypes = [_c.c_int64, _c.c_int32, _c.c_int32, _c.c_int32]
_lib.h3_workspace_size.restype = _c.c_size_t
_lib.h3_varlen_attn_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _c.c_int32, _c.c_int32, _P,
                                    h3_rope_cfg, _c.c_int64, _c.c_int32, _c.c_int32,
                                    _c.c_float, _P, _c.c_size_t, _P]
_lib.h3_varlen_attn_fwd.restype = _c.c_int
_lib.h3_varlen_attn_fwd_static.argtypes = [_P, _P, _P, _P, _P, _P, _c.c_int32, _c.c_int32, _P,
                                           h3_rope_cfg, _c.c_int64, _c.c_int32, _c.c_int32,
                                           _c.c_float, _P]
_lib.h3_varlen_attn_fwd_static.restype = _c.c_int
_lib.h3_varlen_attn_fwd_skip.argtypes = [_P, _P, _P, _P, _P, _P, _c.c_int32, _c.c_int32, _P,
                                         h3_rope_cfg, _c.c_int64, _c.c_int32, _c.c_int32,
                                         _c.c_float, _c.c_float, _P, _c.c_size_t, _P]
_lib.h3_varlen_attn_fwd_skip.restype = _c.c_int
_lib.h3_sage_workspace_size.argtypes = [_c.c_int64, _c.c_int32, _c.c_int32, _c.c_int32]
_lib.h3_sage_workspace_size.restype = _c.c_size_t
_lib.h3_varlen_attn_fwd_sage.argtypes = [_P, _P, _P, _P, _P, _P, _c.c_int32, _c.c_int32, _P,
                                         h3_rope_cfg, _c.c_int64, _c.c_int32, _c.c_int32,
                                         _c.c_float, _P, _c.c_size_t, _P]
_lib.h3_varlen_attn_fwd_sage.restype = _c.c_int
_lib.h3_qkv_rope_gemm.argtypes = [_P, _P, _P, _P, _P, _P, h3_rope_cfg, _c.c_int64, _c.c_int32,
                                  _c.c_int32, _c.c_int32, _P, _c.c_size_t, _P]
_lib.h3_qkv_rope_gemm.restype = _c.c_int
_lib.h3_qkv_rope_attn_fwd.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _c.c_int32, _c.c_int32,
                                      _P, h3_rope_cfg, _c.c_int64, _c.c_int32, _c.c_int32,
                                      _c.c_int32, _c.c_float, _P, _c.c_size_t, _P]
_lib.h3_qkv_rope_attn_fwd.restype = _c.c_int
_i32, _i64, _size = _c.c_int32, _c.c_int64, _c.c_size_t
_lib.h3_rope_qk_freqs.argtypes = [_c.POINTER(h3_rope_qk_cfg), _P]
_lib.h3_rope_qk_freqs.restype = _c.c_int
_lib.h3_rope_qk_apply.argtypes = [_P, _i64, _P, _i64, _P, _i64, _P, _i64, _P,
                                  _c.POINTER(h3_rope_qk_cfg), _i64, _i32, _i32, _i32, _i32, _P]
_lib.h3_rope_qk_apply.restype = _c.c_int
_lib.h3_linear_workspace_size.argtypes = [_i64, _i32, _i32, _i32]
_lib.h3_linear_workspace_size.restype = _size
_lib.h3_linear_fwd.argtypes = [_P, _i64, _P, _i64, _P, _P, _i64, _P, _i64, _i64, _i32, _i32,
                               _i32, _i32, _P, _size, _P]
_lib.h3_linear_fwd.restype = _c.c_int
_lib.h3_cross_workspace_size.argtypes = [_i64, _i32, _i32, _i32, _i32, _i32, _i32]
_lib.h3_cross_workspace_size.restype = _size
_lib.h3_cross_attn_fwd.argtypes = [_P, _i64, _P, _i64, _P, _i64, _P, _i64, _P, _P, _P, _i32,
                                   _i32, _i32, _P, _i64, _i64, _i32, _i32, _i32, _c.c_float,
                                   _i32, _P, _size, _P]
_lib.h3_cross_attn_fwd.restype = _c.c_int
_lib.h3_read_skip_count.argtypes = [_P, _P, _c.POINTER(_c.c_uint64)]
_lib.h3_read_skip_count.restype = _c.c_int
_lib.h3_selftest_bounded_wait.argtypes = [_P, _c.c_size_t, _c.c_int64, _P]
_lib.h3_selftest_bounded_wait.restype = _c.c_int
_lib.h3_read_device_status.argtypes = [_P, _P]
_lib.h3_read_device_status.restype = _c.c_int
_lib.h3_status_string.argtypes = [_c.c_int]
_lib.h3_status_string.restype = _c.c_char_p
_lib.h3_last_cuda_error.argtypes = []
_lib.h3_last_cuda_error.restype = _c.c_int32

EXPORTED = ("h3_segment_tokens", "h3_build_positions", "h3_build_positions_at", "h3_rope_apply", "h3_workspace_size",
            "h3_varlen_attn_fwd", "h3_varlen_attn_fwd_skip", "h3_read_skip_count",
            "h3_qkv_rope_gemm", "h3_qkv_rope_attn_fwd", "h3_sage_workspace_size",
            "h3_varlen_attn_fwd_sage",
            "h3_rope_qk_freqs", "h3_rope_qk_apply", "h3_linear_workspace_size", "h3_linear_fwd",
            "h3_cross_workspace_size", "h3_cross_attn_fwd",
            "h3_varlen_attn_fwd_static", "h3_selftest_bounded_wait",
            "h3_read_device_status", "h3_status_string", "h3_last_cuda_error")

# Scratch bytes compiled into the library for h3_varlen_attn_fwd_static
# (H3_STATIC_WORKSPACE_BYTES in include/h3attn.h).
H3_STATIC_WORKSPACE_BYTES = 256 + (64 << 20)


class H3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        msg = h3_status_string(status)
        if status == H3_ERR_CUDA:
            msg += f" (cudaError {h3_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


def _check(status: int, where: str) -> None:
    if status != H3_OK:
        raise H3Error(status, where)


def rope_cfg(split: Sequence[int], theta: float) -> h3_rope_cfg:
    return h3_rope_cfg(int(split[0]), int(split[1]), int(split[2]), float(theta))


# -------------------------------------------------------- raw C entry points

def h3_status_string(status: int) -> str:
    return _lib.h3_status_string(int(status)).decode()


def h3_last_cuda_error() -> int:
    return int(_lib.h3_last_cuda_error())


def h3_segment_tokens(layout: h3_segment_layout) -> int:
    return int(_lib.h3_segment_tokens(ctypes.byref(layout)))


def h3_workspace_size(N: int, H: int, D: int, nseg: int) -> int:
    return int(_lib.h3_workspace_size(N, H, D, nseg))


def h3_rope_apply(x: int, out: int, pos: int, N: int, H: int, D: int,
                  rope: h3_rope_cfg, stream: int) -> int:
    return int(_lib.h3_rope_apply(x, out, pos, N, H, D, rope, stream))


def h3_varlen_attn_fwd(q: int, k: int, v: int, o: int, lse: int, cu_seqlens: int, nseg: int,
                       max_seqlen: int, pos: int, rope: h3_rope_cfg, N: int, H: int, D: int,
                       softmax_scale: float, workspace: int, workspace_bytes: int,
                       stream: int) -> int:
    return int(_lib.h3_varlen_attn_fwd(q, k, v, o, lse, cu_seqlens, nseg, max_seqlen, pos, rope,
                                       N, H, D, softmax_scale, workspace, workspace_bytes,
                                       stream))


def h3_varlen_attn_fwd_skip(q: int, k: int, v: int, o: int, lse: int, cu_seqlens: int,
                            nseg: int, max_seqlen: int, pos: int, rope: h3_rope_cfg, N: int,
                            H: int, D: int, softmax_scale: float, skip_threshold: float,
                            workspace: int, workspace_bytes: int, stream: int) -> int:
    return int(_lib.h3_varlen_attn_fwd_skip(q, k, v, o, lse, cu_seqlens, nseg, max_seqlen, pos,
                                            rope, N, H, D, softmax_scale, skip_threshold,
                                            workspace, workspace_bytes, stream))


def h3_sage_workspace_size(N: int, H: int, D: int, nseg: int) -> int:
    return int(_lib.h3_sage_workspace_size(N, H, D, nseg))


def h3_varlen_attn_fwd_sage(q: int, k: int, v: int, o: int, lse: int, cu_seqlens: int,
                            nseg: int, max_seqlen: int, pos: int, rope: h3_rope_cfg, N: int,
                            H: int, D: int, softmax_scale: float, workspace: int,
                            workspace_bytes: int, stream: int) -> int:
    return int(_lib.h3_varlen_attn_fwd_sage(q, k, v, o, lse, cu_seqlens, nseg, max_seqlen, pos,
                                            rope, N, H, D, softmax_scale, workspace,
                                            workspace_bytes, stream))


def h3_qkv_rope_gemm(x: int, w: int, q: int, k: int, v: int, pos: int, rope: h3_rope_cfg,
                     N: int, K: int, H: int, D: int, workspace: int, workspace_bytes: int,
                     stream: int) -> int:
    return int(_lib.h3_qkv_rope_gemm(x, w, q, k, v, pos, rope, N, K, H, D, workspace,
                                     workspace_bytes, stream))


def h3_qkv_rope_attn_fwd(x: int, w: int, q: int, k: int, v: int, o: int, lse: int,
                         cu_seqlens: int, nseg: int, max_seqlen: int, pos: int,
                         rope: h3_rope_cfg, N: int, K: int, H: int, D: int,
                         softmax_scale: float, workspace: int, workspace_bytes: int,
                         stream: int) -> int:
    return int(_lib.h3_qkv_rope_attn_fwd(x, w, q, k, v, o, lse, cu_seqlens, nseg, max_seqlen,
                                         pos, rope, N, K, H, D, softmax_scale, workspace,
                                         workspace_bytes, stream))


def h3_read_skip_count(workspace: int, stream: int) -> int:
    n = ctypes.c_uint64(0)
    _check(_lib.h3_read_skip_count(workspace, stream, ctypes.byref(n)), "h3_read_skip_count")
    return int(n.value)


def h3_varlen_attn_fwd_static(q: int, k: int, v: int, o: int, lse: int, cu_seqlens: int,
                              nseg: int, max_seqlen: int, pos: int, rope: h3_rope_cfg, N: int,
                              H: int, D: int, softmax_scale: float, stream: int) -> int:
    """h3_varlen_attn_fwd without a caller workspace: for hosts that cannot
    allocate device memory, the library's own compiled-in scratch is used
    (N*H*D <= 2^25; calls on one device must not overlap on the GPU)."""
    return int(_lib.h3_varlen_attn_fwd_static(q, k, v, o, lse, cu_seqlens, nseg, max_seqlen,
                                              pos, rope, N, H, D, softmax_scale, stream))


# ctypes cuts integers off to 32 bits where the C calls take that many. The bits of
# several sizes together, shifted by 31, are 0 where all fit, and -1 where one is
# negative, which the calls refuse themselves.
_FITS = (0, -1)


def h3_rope_qk_freqs(cfg: h3_rope_qk_cfg):
    """Angle per position of each pair, NumPy float64 [rot_dim/2] (host only)."""
    import numpy as np
    f = np.zeros(max(1, min(256, cfg.rot_dim // 2)), dtype=np.float64)
    _check(_lib.h3_rope_qk_freqs(ctypes.byref(cfg), f.ctypes.data), "h3_rope_qk_freqs")
    return f


def h3_rope_qk_apply(q: int, ldq: int, q_out: int, ldq_out: int, k: int, ldk: int, k_out: int,
                     ldk_out: int, positions: int, cfg: h3_rope_qk_cfg, N: int, Hq: int, Hk: int,
                     D: int, dtype: int, stream: int) -> int:
    if (Hq | Hk | D | dtype) >> 31 not in _FITS:
        return H3_ERR_INVALID_ARG
    return _lib.h3_rope_qk_apply(q, ldq, q_out, ldq_out, k, ldk, k_out, ldk_out, positions,
                                 ctypes.byref(cfg), N, Hq, Hk, D, dtype, stream)


def h3_linear_workspace_size(M: int, N: int, K: int, act: int) -> int:
    return _lib.h3_linear_workspace_size(M, N, K, act) if (N | K | act) >> 31 in _FITS else 0


def h3_linear_fwd(x: int, ldx: int, w: int, ldw: int, bias: int, residual: int, ldr: int, y: int,
                  ldy: int, M: int, N: int, K: int, act: int, dtype: int, workspace: int,
                  workspace_bytes: int, stream: int) -> int:
    if (N | K | act | dtype) >> 31 not in _FITS:
        return H3_ERR_INVALID_ARG
    return _lib.h3_linear_fwd(x, ldx, w, ldw, bias, residual, ldr, y, ldy, M, N, K, act, dtype,
                              workspace, workspace_bytes, stream)


def h3_cross_workspace_size(Nq: int, Hq: int, Hk: int, D: int, nseg: int, max_q: int,
                            max_k: int) -> int:
    if (Hq | Hk | D | nseg | max_q | max_k) >> 31 not in _FITS:
        return 0
    return _lib.h3_cross_workspace_size(Nq, Hq, Hk, D, nseg, max_q, max_k)


def h3_cross_attn_fwd(q: int, ldq: int, k: int, ldk: int, v: int, ldv: int, o: int, ldo: int,
                      lse: int, cu_q: int, cu_k: int, nseg: int, max_q: int, max_k: int,
                      key_mask: int, Nq: int, Nk: int, Hq: int, Hk: int, D: int,
                      softmax_scale: float, dtype: int, workspace: int, workspace_bytes: int,
                      stream: int) -> int:
    if (nseg | max_q | max_k | Hq | Hk | D | dtype) >> 31 not in _FITS:
        return H3_ERR_INVALID_ARG
    return _lib.h3_cross_attn_fwd(q, ldq, k, ldk, v, ldv, o, ldo, lse, cu_q, cu_k, nseg, max_q,
                                  max_k, key_mask, Nq, Nk, Hq, Hk, D, softmax_scale, dtype,
                                  workspace, workspace_bytes, stream)


def h3_selftest_bounded_wait(workspace: int, workspace_bytes: int, limit_cycles: int,
                             stream: int) -> int:
    return int(_lib.h3_selftest_bounded_wait(workspace, workspace_bytes, limit_cycles, stream))


def h3_read_device_status(workspace: int, stream: int) -> int:
    return int(_lib.h3_read_device_status(workspace, stream))


def h3_build_positions(layouts, t_origins=None):
    """Host position build. ``layouts``: objects with the attributes of
    ``h3_segment_layout`` (or of a segment description with ``video``,
    ``audio_tail``, ``image_refs``, ``image_grid``, ``audio_refs``,
    ``audio_ref_len``, ``audio_rate``); ``t_origins``: optional clock origin
    per segment (h3_build_positions_at). Returns (pos float32 [N, 3],
    cu_seqlens int32 [nseg + 1]) as NumPy arrays."""
    import numpy as np
    segs = (h3_segment_layout * max(1, len(layouts)))()
    for i, l in enumerate(layouts):
        segs[i] = to_c_layout(l)
    total = sum(max(0, h3_segment_tokens(segs[i])) for i in range(len(layouts)))
    pos = np.zeros((max(total, 1), 3), dtype=np.float32)
    cu = np.zeros(len(layouts) + 1, dtype=np.int32)
    if t_origins is None:
        st = _lib.h3_build_positions(segs, len(layouts), pos.ctypes.data, total,
                                     cu.ctypes.data)
    else:
        org = np.ascontiguousarray(t_origins, dtype=np.float64)
        if org.shape != (len(layouts),):
            raise ValueError("one clock origin per segment")
        st = _lib.h3_build_positions_at(segs, len(layouts), org.ctypes.data,
                                        pos.ctypes.data, total, cu.ctypes.data)
    _check(st, "h3_build_positions")
    return pos[:total], cu


def to_c_layout(l) -> h3_segment_layout:
    if isinstance(l, h3_segment_layout):
        return l
    T, Hg, Wg = l.video
    ih, iw = l.image_grid
    return h3_segment_layout(l.image_refs, ih, iw, l.audio_refs, l.audio_ref_len, l.audio_rate,
                             T, Hg, Wg, l.audio_tail)


# ------------------------------------------------------ torch tensor helpers

def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _thd(x, name):
    import torch
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 3 and x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor [N, H, D]")
    return x


def rope_apply_t(x, pos, split, theta: float = 10000.0, out=None, stream=None):
    """out = RoPE(x, pos) through h3_rope_apply. x bf16 [N, H, D], pos fp32 [N, 3]."""
    import torch
    _thd(x, "x")
    if out is None:
        out = torch.empty_like(x)
    N, H, D = x.shape
    _check(h3_rope_apply(x.data_ptr(), out.data_ptr(), pos.data_ptr(), N, H, D,
                         rope_cfg(split, theta), _stream(stream)), "h3_rope_apply")
    return out


def workspace_for(N: int, H: int, D: int, nseg: int, device=None):
    import torch
    n = h3_workspace_size(N, H, D, nseg)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def varlen_attn_fwd_t(q, k, v, cu_seqlens, max_seqlen: int, pos=None, split=None,
                      theta: float = 10000.0, softmax_scale: Optional[float] = None,
                      out=None, return_lse: bool = False, workspace=None, stream=None):
    """O (and LSE [H, N] if asked) through h3_varlen_attn_fwd."""
    import torch
    _thd(q, "q"); _thd(k, "k"); _thd(v, "v")
    N, H, D = q.shape
    nseg = int(cu_seqlens.numel()) - 1
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((H, N), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        workspace = workspace_for(N, H, D, nseg, q.device)
    scale = (1.0 / math.sqrt(D)) if softmax_scale is None else float(softmax_scale)
    rope = rope_cfg(split, theta) if pos is not None else h3_rope_cfg(0, 0, 0, 0.0)
    st = h3_varlen_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                            lse.data_ptr() if lse is not None else 0,
                            cu_seqlens.data_ptr(), nseg, int(max_seqlen),
                            pos.data_ptr() if pos is not None else 0, rope, N, H, D, scale,
                            workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(st, "h3_varlen_attn_fwd")
    return (out, lse) if return_lse else out


def varlen_attn_fwd_skip_t(q, k, v, cu_seqlens, max_seqlen: int, skip_threshold: float,
                           pos=None, split=None, theta: float = 10000.0,
                           softmax_scale: Optional[float] = None, out=None,
                           return_lse: bool = False, workspace=None, stream=None):
    """Skip-softmax variant through h3_varlen_attn_fwd_skip; the number of
    skipped (32-row block, key tile) pairs is read with skip_count_t(workspace)."""
    import torch
    _thd(q, "q"); _thd(k, "k"); _thd(v, "v")
    N, H, D = q.shape
    nseg = int(cu_seqlens.numel()) - 1
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((H, N), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        workspace = workspace_for(N, H, D, nseg, q.device)
    scale = (1.0 / math.sqrt(D)) if softmax_scale is None else float(softmax_scale)
    rope = rope_cfg(split, theta) if pos is not None else h3_rope_cfg(0, 0, 0, 0.0)
    st = h3_varlen_attn_fwd_skip(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 lse.data_ptr() if lse is not None else 0,
                                 cu_seqlens.data_ptr(), nseg, int(max_seqlen),
                                 pos.data_ptr() if pos is not None else 0, rope, N, H, D, scale,
                                 float(skip_threshold), workspace.data_ptr(), workspace.numel(),
                                 _stream(stream))
    _check(st, "h3_varlen_attn_fwd_skip")
    return (out, lse) if return_lse else out


def qkv_rope_gemm_t(x, w, heads: int, head_dim: int, pos=None, split=None,
                    theta: float = 10000.0, out=None, workspace=None, stream=None):
    """(q, k, v) [N, H, D] bf16 through h3_qkv_rope_gemm: the projection
    x [N, K] @ w[3*H*D, K]^T with RoPE applied to q and k in its epilogue."""
    import torch
    for t, name in ((x, "x"), (w, "w")):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.dim() == 2 and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA bfloat16 matrix")
    N, K = x.shape
    if tuple(w.shape) != (3 * heads * head_dim, K):
        raise ValueError(f"w must be [3*H*D, K] = [{3 * heads * head_dim}, {K}]")
    if out is None:
        out = tuple(torch.empty((N, heads, head_dim), dtype=torch.bfloat16, device=x.device)
                    for _ in range(3))
    q, k, v = out
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=x.device)
    rope = rope_cfg(split, theta) if pos is not None else h3_rope_cfg(0, 0, 0, 0.0)
    st = h3_qkv_rope_gemm(x.data_ptr(), w.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                          pos.data_ptr() if pos is not None else 0, rope, N, K, heads,
                          head_dim, workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(st, "h3_qkv_rope_gemm")
    return q, k, v


def qkv_rope_attn_fwd_t(x, w, heads: int, head_dim: int, cu_seqlens, max_seqlen: int,
                        pos=None, split=None, theta: float = 10000.0,
                        softmax_scale: Optional[float] = None, qkv=None, out=None,
                        return_lse: bool = False, workspace=None, stream=None):
    """O (and LSE [H, N] if asked) of attention over the projection x w^T,
    through h3_qkv_rope_attn_fwd: q and k are rotated in the projection's
    epilogue and the attention reads them as they are. ``qkv`` receives the
    projection ([N, H, D] bf16 each; allocated if None)."""
    import torch
    for t, name in ((x, "x"), (w, "w")):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.dim() == 2 and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA bfloat16 matrix")
    N, K = x.shape
    if tuple(w.shape) != (3 * heads * head_dim, K):
        raise ValueError(f"w must be [3*H*D, K] = [{3 * heads * head_dim}, {K}]")
    if qkv is None:
        qkv = tuple(torch.empty((N, heads, head_dim), dtype=torch.bfloat16, device=x.device)
                    for _ in range(3))
    q, k, v = qkv
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _thd(t, name)
    if out is None:
        out = torch.empty_like(q)
    lse = (torch.empty((heads, N), dtype=torch.float32, device=x.device) if return_lse
           else None)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=x.device)
    nseg = int(cu_seqlens.numel()) - 1
    scale = (1.0 / math.sqrt(head_dim)) if softmax_scale is None else float(softmax_scale)
    rope = rope_cfg(split, theta) if pos is not None else h3_rope_cfg(0, 0, 0, 0.0)
    st = h3_qkv_rope_attn_fwd(x.data_ptr(), w.data_ptr(), q.data_ptr(), k.data_ptr(),
                              v.data_ptr(), out.data_ptr(),
                              lse.data_ptr() if lse is not None else 0, cu_seqlens.data_ptr(),
                              nseg, int(max_seqlen), pos.data_ptr() if pos is not None else 0,
                              rope, N, K, heads, head_dim, scale, workspace.data_ptr(),
                              workspace.numel(), _stream(stream))
    _check(st, "h3_qkv_rope_attn_fwd")
    return (out, lse) if return_lse else out


def sage_workspace_for(N: int, H: int, D: int, nseg: int, device=None):
    import torch
    n = h3_sage_workspace_size(N, H, D, nseg)
    if n == 0:
        raise ValueError("the SAGE variant supports head dim 128 only")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def sage_workspace_views(workspace, N: int, H: int, nseg: int) -> dict:
    """Views of the regions h3_varlen_attn_fwd_sage leaves in its workspace
    (layout of h3_sage_workspace_size in include/h3attn.h): q8, k8, v8 uint8
    [N, H, 128]; s_q, s_k float32 [H, N]; v_amax, s_v float32 [nseg, H, 128]."""
    import torch

    def up(x):
        return (x + 255) // 256 * 256
    codes, scales, vsc = up(N * H * 128), up(N * H * 4), up(nseg * H * 128 * 4)
    off = {"q8": 256}
    off["k8"] = off["q8"] + codes
    off["v8"] = off["k8"] + codes
    off["s_q"] = off["v8"] + codes
    off["s_k"] = off["s_q"] + scales
    off["v_amax"] = off["s_k"] + scales
    off["s_v"] = off["v_amax"] + vsc
    out = {}
    for name in ("q8", "k8", "v8"):
        out[name] = workspace[off[name]:off[name] + N * H * 128].view(N, H, 128)
    for name in ("s_q", "s_k"):
        out[name] = workspace[off[name]:off[name] + N * H * 4].view(torch.float32).view(H, N)
    for name in ("v_amax", "s_v"):
        out[name] = workspace[off[name]:off[name] + nseg * H * 512].view(torch.float32) \
            .view(nseg, H, 128)
    return out


def varlen_attn_fwd_sage_t(q, k, v, cu_seqlens, max_seqlen: int, pos=None, split=None,
                           theta: float = 10000.0, softmax_scale: Optional[float] = None,
                           out=None, return_lse: bool = False, workspace=None, stream=None):
    """SAGE-style FP8 variant through h3_varlen_attn_fwd_sage (head dim 128)."""
    import torch
    _thd(q, "q"); _thd(k, "k"); _thd(v, "v")
    N, H, D = q.shape
    nseg = int(cu_seqlens.numel()) - 1
    if out is None:
        out = torch.empty_like(q)
    lse = torch.empty((H, N), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        workspace = sage_workspace_for(N, H, D, nseg, q.device)
    scale = (1.0 / math.sqrt(D)) if softmax_scale is None else float(softmax_scale)
    rope = rope_cfg(split, theta) if pos is not None else h3_rope_cfg(0, 0, 0, 0.0)
    st = h3_varlen_attn_fwd_sage(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 lse.data_ptr() if lse is not None else 0,
                                 cu_seqlens.data_ptr(), nseg, int(max_seqlen),
                                 pos.data_ptr() if pos is not None else 0, rope, N, H, D, scale,
                                 workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(st, "h3_varlen_attn_fwd_sage")
    return (out, lse) if return_lse else out


def skip_count_t(workspace, stream=None) -> int:
    """Skipped (32-row block, key tile) pairs of the last skip call on ``workspace`` (syncs)."""
    return h3_read_skip_count(workspace.data_ptr(), _stream(stream))


def device_status_t(workspace, stream=None) -> int:
    """Device status word of the last call that used ``workspace`` (syncs)."""
    return h3_read_device_status(workspace.data_ptr(), _stream(stream))


# -------------------------------------------- layers around the attention (torch)

_DTYPE_CODES: dict = {}
_torch = _forward_ad = None


def _load_torch():
    """torch, kept: an import statement in every helper costs these short calls
    a tenth of their time."""
    global _torch, _forward_ad
    import torch
    _torch, _forward_ad = torch, torch.autograd.forward_ad
    return torch


def _dtype_code(dtype, fp32: bool = False) -> int:
    if not _DTYPE_CODES:
        torch = _torch or _load_torch()
        _DTYPE_CODES.update({torch.bfloat16: H3_BF16, torch.float16: H3_FP16,
                             torch.float32: H3_FP32})
    code = _DTYPE_CODES.get(dtype, -1)
    if code < 0 or (code == H3_FP32 and not fp32):
        raise ValueError(f"dtype {dtype} is not supported")
    return code


def _same(device, *tensors):
    """Every given tensor is on ``device``; none asks for a gradient or carries a
    tangent (these calls are forward only, so either would be lost in silence)."""
    torch = _torch or _load_torch()
    grad = torch.is_grad_enabled()
    dual = _forward_ad._current_level >= 0
    cuda = device.type == "cuda"
    for t in tensors:
        if t is None:
            continue
        if t.device != device or not cuda:
            raise ValueError(f"all tensors must be on one CUDA device: {t.device}, {device}")
        if grad and t.requires_grad:
            raise ValueError("forward only: call under torch.no_grad() or detach the inputs")
        if dual and _forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError("forward only: a tangent would be lost")


def _on(device, stream, *tensors):
    """Context in which a call on ``stream`` (None: the device's current one)
    allocates and launches: that device is current, and what the call allocates
    belongs to that stream. The memory of ``tensors`` is not given out again
    before a given stream has done what is on it by the time they are dropped,
    unless it is the caller's (a raw handle, an ExternalStream): that one may end
    before they do, and its caller keeps them."""
    torch = _torch or _load_torch()
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):   # (ExternalStream takes 0 for "a new one")
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    if isinstance(stream, torch.cuda.ExternalStream):
        tensors = ()
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, not on {device}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _current_stream(device) -> int:
    """Handle of the device's current stream, without building a stream object."""
    torch = _torch or _load_torch()
    return torch._C._cuda_getCurrentRawStream(device.index)


def _like(x):
    """A contiguous tensor of x's shape and type."""
    return _torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _bytes(workspace) -> int:
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.nbytes


def _changed(*outs):
    """Tells autograd that these tensors have been written into."""
    _torch.autograd.graph.increment_version([t for t in outs if t is not None])


def _heads(x, name):
    """(token stride) of a [N, H, D] tensor whose heads are contiguous."""
    if x.dim() != 3:
        raise ValueError(f"{name} must be [N, H, D]")
    N, H, D = x.shape
    s = x.stride()
    if N > 0 and ((s[2] != 1 and D > 1) or (s[1] != D and H > 1)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return H * D if N <= 1 else s[0]


def _rows(x, name):
    if x.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if x.shape[0] > 0 and x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    # of a single row the stride says nothing
    return x.stride(0) if x.shape[0] > 1 else (x.shape[1] + 7) // 8 * 8


def _int32(x, name, shape=None):
    torch = _torch or _load_torch()
    if x.dtype != torch.int32 or not x.is_contiguous() or (shape is not None and x.shape != shape):
        raise ValueError(f"{name} must be contiguous int32" + (f" {list(shape)}" if shape else ""))


def rope_qk_cfg(rot_dim: int, theta: float = 10000.0, layout: str = "interleaved",
                scaling: Optional[dict] = None) -> h3_rope_qk_cfg:
    """``scaling``: None or a dict with ``kind`` ("linear", "ntk", "turns",
    "yarn") and the fields of h3_rope_qk_cfg it reads (``factor``,
    ``original_len``, ``beta_fast``, ``beta_slow``, ``attn_factor``)."""
    s = dict(scaling or {})
    kind = s.pop("kind", "none")
    if kind not in ROPE_SCALINGS or layout not in ("interleaved", "half"):
        raise ValueError(f"unknown scaling {kind!r} or layout {layout!r}")
    if int(rot_dim) >> 31 not in _FITS:
        raise ValueError(f"rot_dim {rot_dim} is out of range")
    values = {"factor": 1.0, "original_len": 0.0, "beta_fast": 0.0, "beta_slow": 0.0,
              "attn_factor": 1.0}
    for key, value in s.items():
        if key not in values:
            raise ValueError(f"unknown scaling field {key!r}")
        values[key] = float(value)
    return h3_rope_qk_cfg(int(rot_dim), H3_ROPE_HALF if layout == "half" else H3_ROPE_INTERLEAVED,
                          ROPE_SCALINGS[kind], 0, float(theta), values["factor"],
                          values["original_len"], values["beta_fast"], values["beta_slow"],
                          values["attn_factor"])


_PLAIN = frozenset((float, int, str))


def _by_value(scaling):
    """A scaling's items as plain numbers: what a cfg is kept under."""
    if _PLAIN.issuperset(map(type, scaling.values())):
        return tuple(scaling.items())
    return tuple((k, v if isinstance(v, str) else float(v)) for k, v in scaling.items())


@functools.lru_cache(maxsize=64)
def _rope_qk_cfg(rot_dim, theta, layout, scaling) -> h3_rope_qk_cfg:
    return rope_qk_cfg(rot_dim, theta, layout, dict(scaling))


def rope_qk_t(q, k, positions, rot_dim: Optional[int] = None, theta: float = 10000.0,
              layout: str = "interleaved", scaling: Optional[dict] = None, out=None, stream=None):
    """(q, k) rotated by whole-number positions through h3_rope_qk_apply. q
    [N, Hq, D], k [N, Hk, D] or None, bf16, fp16 or fp32, heads contiguous (a
    token stride is free); positions int32 [N]. ``out``: (q_out, k_out), which
    may be (q, k). The gradient of q and k is this call on the outputs'
    gradients with negated positions. The tensors of a call on a raw handle or an
    ExternalStream are the caller's to keep until that stream has done it."""
    torch = _torch or _load_torch()
    device = q.device
    given = out or ()
    _same(device, q, k, positions, *given)
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream, q, k, positions, *given):
            return rope_qk_t(q, k, positions, rot_dim, theta, layout, scaling, out)
    code = _dtype_code(q.dtype, fp32=True)
    N, Hq, D = q.shape
    ldq = _heads(q, "q")
    _int32(positions, "positions", (N,))
    cfg = _rope_qk_cfg(D if rot_dim is None else int(rot_dim), float(theta), layout,
                       _by_value(scaling) if scaling else ())
    Hk, ldk, kp = 0, 0, 0
    if k is not None:
        if k.dtype != q.dtype or k.dim() != 3 or k.shape[0] != N or k.shape[2] != D:
            raise ValueError("k must be [N, Hk, D] of q's type")
        Hk, ldk, kp = k.shape[1], _heads(k, "k"), k.data_ptr()
    if out is None:
        qo, ko = _like(q), None if k is None else _like(k)
        ldqo, ldko = Hq * D, Hk * D
    else:
        qo, ko = out
        if qo.shape != q.shape or qo.dtype != q.dtype or (k is None) != (ko is None) or (
                k is not None and (ko.shape != k.shape or ko.dtype != q.dtype)):
            raise ValueError("out must have the shapes and type of (q, k)")
        ldqo, ldko = _heads(qo, "q_out"), 0 if ko is None else _heads(ko, "k_out")
    _check(h3_rope_qk_apply(q.data_ptr(), ldq, qo.data_ptr(), ldqo, kp, ldk,
                            0 if ko is None else ko.data_ptr(), ldko, positions.data_ptr(), cfg,
                            N, Hq, Hk, D, code, _current_stream(device)),
           "h3_rope_qk_apply")
    if given:
        _changed(*given)
    return qo, ko


def linear_workspace_for(M: int, N: int, K: int, gated: bool = False, device=None):
    """Workspace of linear_t for x [M, K] and N output features."""
    torch = _torch or _load_torch()
    n = h3_linear_workspace_size(M, N, K, H3_ACT_GATED if gated else 0)
    if n == 0:
        raise ValueError("sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def linear_t(x, w, bias=None, act: str = "none", gated: bool = False, residual=None, out=None,
             workspace=None, stream=None):
    """act(x w^T + bias) + residual through h3_linear_fwd. x [M, K], w [N, K],
    bf16 or fp16, rows 16-byte aligned (row strides a multiple of 8: where K is
    not, x and w are views of wider rows; what lies behind K is not read).
    ``gated``: w [2N, K], act(first half) * (second half). ``out`` may be
    ``residual``. Without a ``workspace`` the call makes its own, and what it
    reports there (device_status_t) cannot be asked for. The tensors of a call on
    a raw handle or an ExternalStream are the caller's to keep until that stream
    has done it."""
    torch = _torch or _load_torch()
    device = x.device
    _same(device, x, w, bias, residual, out, workspace)
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream, x, w, bias, residual, out, workspace):
            return linear_t(x, w, bias, act, gated, residual, out, workspace)
    code = _dtype_code(x.dtype)
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}")
    ldx, ldw = _rows(x, "x"), _rows(w, "w")
    M, K = x.shape
    N = w.shape[0]
    if w.dtype != x.dtype or w.shape[1] != K or (gated and N % 2):
        raise ValueError(f"w must be [{'2N' if gated else 'N'}, {K}] of x's type")
    if bias is not None and (bias.dtype != x.dtype or bias.shape != (N,) or
                             not bias.is_contiguous()):
        raise ValueError(f"bias must be contiguous [{N}] of x's type")
    a = ACTIVATIONS[act]
    if gated:
        N //= 2
        a += H3_ACT_GATED
    ldr = 0
    if residual is not None:
        if residual.shape != (M, N) or residual.dtype != x.dtype:
            raise ValueError(f"residual must be [{M}, {N}] of x's type")
        ldr = _rows(residual, "residual")
    given = out
    if out is None:
        out = x.new_empty((M, N))
    elif out.shape != (M, N) or out.dtype != x.dtype:
        raise ValueError(f"out must be [{M}, {N}] of x's type")
    if workspace is None:
        workspace = linear_workspace_for(M, N, K, gated, device)
    _check(h3_linear_fwd(x.data_ptr(), ldx, w.data_ptr(), ldw,
                         0 if bias is None else bias.data_ptr(),
                         0 if residual is None else residual.data_ptr(), ldr, out.data_ptr(),
                         _rows(out, "out"), M, N, K, a, code, workspace.data_ptr(),
                         _bytes(workspace), _current_stream(device)),
           "h3_linear_fwd")
    if given is not None:
        _changed(given)
    return out


def cross_workspace_for(Nq: int, Hq: int, Hk: int, D: int, nseg: int, max_q: int, max_k: int,
                        device=None):
    """Workspace of cross_attn_fwd_t for these sizes."""
    torch = _torch or _load_torch()
    n = h3_cross_workspace_size(Nq, Hq, Hk, D, nseg, max_q, max_k)
    if n == 0:
        raise ValueError("sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def cross_attn_fwd_t(q, k, v, cu_q, cu_k, max_q: int, max_k: int, key_mask=None,
                     softmax_scale: Optional[float] = None, out=None, return_lse: bool = False,
                     workspace=None, stream=None):
    """O (and LSE [Hq, Nq] if asked) through h3_cross_attn_fwd: the queries of
    each segment attend to its keys in another packed sequence. q [Nq, Hq, D],
    k, v [Nk, Hk, D], bf16 or fp16, heads contiguous, token strides a multiple
    of 8; cu_q, cu_k int32 [nseg + 1]; key_mask bool or uint8 [Nk], False: no
    query attends to this key. A row without keys gets 0 (LSE -inf). Rows
    behind cu_q[-1] are not written, and none is where the lengths are not as
    said: a caller who cannot vouch for them passes a ``workspace`` and asks
    device_status_t for it. The tensors of a call on a raw handle or an
    ExternalStream are the caller's to keep until that stream has done it."""
    torch = _torch or _load_torch()
    device = q.device
    _same(device, q, k, v, cu_q, cu_k, key_mask, out, workspace)
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        with _on(device, stream, q, k, v, cu_q, cu_k, key_mask, out, workspace):
            return cross_attn_fwd_t(q, k, v, cu_q, cu_k, max_q, max_k, key_mask, softmax_scale,
                                    out, return_lse, workspace)
    code = _dtype_code(q.dtype)
    ldq, ldk, ldv = _heads(q, "q"), _heads(k, "k"), _heads(v, "v")
    Nq, Hq, D = q.shape
    Nk, Hk, _ = k.shape
    if k.dtype != q.dtype or v.dtype != q.dtype or k.shape != v.shape or k.shape[2] != D:
        raise ValueError("k and v must be [Nk, Hk, D] of q's type")
    nseg = cu_q.numel() - 1
    _int32(cu_q, "cu_q", (nseg + 1,))
    _int32(cu_k, "cu_k", (nseg + 1,))
    if key_mask is not None and (key_mask.shape != (Nk,) or not key_mask.is_contiguous() or
                                 key_mask.dtype not in (torch.bool, torch.uint8)):
        raise ValueError(f"key_mask must be contiguous bool or uint8 [{Nk}]")
    given = out
    if out is None:
        out = _like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and type")
    lse = q.new_empty((Hq, Nq), dtype=torch.float32) if return_lse else None
    if workspace is None:
        workspace = cross_workspace_for(Nq, Hq, Hk, D, nseg, int(max_q), int(max_k), device)
    scale = (1.0 / math.sqrt(D)) if softmax_scale is None else float(softmax_scale)
    _check(h3_cross_attn_fwd(q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
                             out.data_ptr(), _heads(out, "out"),
                             0 if lse is None else lse.data_ptr(), cu_q.data_ptr(),
                             cu_k.data_ptr(), nseg, int(max_q), int(max_k),
                             0 if key_mask is None else key_mask.data_ptr(), Nq, Nk, Hq, Hk, D,
                             scale, code, workspace.data_ptr(), _bytes(workspace),
                             _current_stream(device)),
           "h3_cross_attn_fwd")
    if given is not None:
        _changed(given)
    return (out, lse) if return_lse else out

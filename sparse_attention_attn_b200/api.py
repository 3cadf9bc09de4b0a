"""PyTorch-facing calls of the S2-Attn library (device memory and streams only).

Each function checks tensor placement, dtype, layout and shape, then calls the
C ABI through ctypes on torch's current CUDA stream.  The arithmetic happens
only in the CUDA kernels of libs2attn.so; a missing library or a non-B200
device raises instead of falling back to anything else.

Shift rule (LongQLoRA community post, section 03, Shift Short Attention; the
LongLoRA abstract): with group size G < N, query heads h >= H/2 attend inside
groups of the sequence rolled by G/2 rows (wrap-around); G == N is dense causal
attention.  Training uses the shifted groups, inference the dense path.
"""
from __future__ import annotations

import ctypes
import warnings
from typing import NamedTuple, Optional

import torch

from . import _lib


class _Binding:
    """The calls of _s2torch.so (csrc/s2_torch.cpp: the usual case of the smallest
    calls in one step, None for any other), bound at the first use to the library
    the ctypes binding loaded; where it is not built, does not load, or was
    compiled for another interface of the library or another torch (it calls the
    one by address and reads the other's tensors by their layout), functions that
    leave every call to the Python path."""

    _NAMES = ("qknorm_fwd", "qknorm_bwd", "cache_append", "cache_plan", "cache_attention")

    def __getattr__(self, name):
        if name not in self._NAMES:
            raise AttributeError(name)
        lib = _lib.load()
        self.__dict__.update({n: lambda *args: None for n in self._NAMES})
        try:
            from . import _s2torch
        except ImportError:
            return self.__dict__[name]
        ours = (lib.s2attn_header_hash().decode(), f"{torch.version.__version__} {torch.version.git_version}")
        its = (getattr(_s2torch, "header_hash", None), getattr(_s2torch, "torch_version", None))
        if its != ours:
            warnings.warn(f"_s2torch.so was built for {its}, not for {ours}: its calls take the Python way until "
                          "`python -m sparse_attention_attn_b200.build` is run", RuntimeWarning, stacklevel=3)
            return self.__dict__[name]
        _s2torch.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in
                        ("s2attn_qknorm_rope_fwd", "s2attn_qknorm_rope_bwd",
                         "s2attn_qknorm_rope_bwd_workspace_bytes", "s2attn_cache_append", "s2attn_cache_plan",
                         "s2attn_cache_attn", "s2attn_cache_attn_workspace_bytes")))
        self.__dict__.update({n: getattr(_s2torch, n) for n in self._NAMES})
        return self.__dict__[name]


_fast = _Binding()


def _stream(device=None) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(name: str, t: torch.Tensor, shape, dtype=torch.bfloat16, device=None) -> None:
    try:  # the usual case in as few steps as it takes; what fails is named below
        if (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()
                and (device is None or t.device == device)):
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device} (all operands on one device)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims(q: torch.Tensor, k: torch.Tensor):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, N, H, D] and k [B, N, Hkv, D]")
    B, N, H, D = q.shape
    return B, N, H, k.shape[2], D


def s2attn_forward(q, k, v, group_size: int, out=None, lse=None):
    """S2-Attn forward.  q [B,N,H,D], k/v [B,N,Hkv,D] bf16 CUDA tensors.

    Returns (o [B,N,H,D] bf16, lse [B,H,N] fp32 natural-log log-sum-exp).
    """
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    _need("k", k, (B, N, Hkv, D), device=dev)
    _need("v", v, (B, N, Hkv, D), device=dev)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    _need("out", out, (B, N, H, D), device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    with torch.cuda.device(dev):  # the C ABI launches on the current device
        st = _lib.s2attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                             B, H, Hkv, N, D, int(group_size), _stream(dev))
    _lib._check("s2attn_fwd", st)
    return out, lse


def bwd_workspace_bytes(B, H, Hkv, N, D, group_size) -> int:
    n = _lib.s2attn_bwd_workspace_bytes(B, H, Hkv, N, D, int(group_size))
    if n == 0:
        raise _lib.S2AttnError("s2attn_bwd_workspace_bytes", _lib.S2ATTN_ERR_INVALID_ARG)
    return n


def s2attn_backward(q, k, v, o, lse, do, group_size: int, dq=None, dk=None, dv=None,
                    workspace=None):
    """S2-Attn backward.  Returns (dq, dk, dv); dk/dv summed over shared query heads."""
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    for name, t, shp in (("k", k, (B, N, Hkv, D)), ("v", v, (B, N, Hkv, D)),
                         ("o", o, (B, N, H, D)), ("do", do, (B, N, H, D))):
        _need(name, t, shp, device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _need("dq", dq, (B, N, H, D), device=dev)
    _need("dk", dk, (B, N, Hkv, D), device=dev)
    _need("dv", dv, (B, N, Hkv, D), device=dev)
    wsb = bwd_workspace_bytes(B, H, Hkv, N, D, group_size)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    if workspace.numel() * workspace.element_size() < wsb:
        raise _lib.S2AttnError("s2attn_bwd", _lib.S2ATTN_ERR_WORKSPACE)
    with torch.cuda.device(dev):  # the C ABI launches on the current device
        st = _lib.s2attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                             do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                             B, H, Hkv, N, D, int(group_size), workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), _stream(dev))
    _lib._check("s2attn_bwd", st)
    return dq, dk, dv


def device_status(workspace=None) -> int:
    """Synchronise the current stream and return (and clear) the device status."""
    ptr = workspace.data_ptr() if workspace is not None else None
    return _lib.s2attn_device_status(ptr, _stream())


def rope_table(N: int, D: int, pos_scale: float, rope_base: float = 10000.0, device=None):
    """fp32 (cos, sin) table [N, D/2, 2] of RoPE with Position Interpolation:
    pair i at token t turns by t * pos_scale * rope_base^(-2i/D) (LongQLoRA
    post section 04: Position Interpolation shrinks RoPE's angles; pos_scale =
    L_train / L_target).  Built on the GPU; reuse it across layers and steps."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    nbytes = _lib.s2attn_rope_table_bytes(N, D)
    if nbytes == 0:
        raise _lib.S2AttnError("s2attn_rope_table_bytes", _lib.S2ATTN_ERR_UNSUPPORTED)
    table = torch.empty((N, D // 2, 2), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_rope_table(table.data_ptr(), N, D, float(pos_scale), float(rope_base), _stream(dev))
    _lib._check("s2attn_rope_table", st)
    return table


def rope_apply(x, table, inverse: bool = False, out=None):
    """x [B, N, heads, D] bf16 rotated by the table (the opposite way when
    `inverse`); out may be x (in place)."""
    B, N, Hx, D = x.shape
    _need("x", x, (B, N, Hx, D))
    _need("table", table, (N, D // 2, 2), torch.float32, device=x.device)
    out = torch.empty_like(x) if out is None else out
    _need("out", out, (B, N, Hx, D), device=x.device)
    with torch.cuda.device(x.device):
        st = _lib.s2attn_rope_apply(x.data_ptr(), out.data_ptr(), table.data_ptr(), B, N, Hx, D, int(inverse),
                                    _stream(x.device))
    _lib._check("s2attn_rope_apply", st)
    return out


def s2attn_forward_rope(q, k, v, group_size: int, table, out=None, lse=None, q_rot=None, k_rot=None):
    """S2 attention on RoPE-rotated q and k.  Returns (o, lse, q_rot, k_rot);
    q_rot and k_rot are what the backward takes."""
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    _need("k", k, (B, N, Hkv, D), device=dev)
    _need("v", v, (B, N, Hkv, D), device=dev)
    _need("table", table, (N, D // 2, 2), torch.float32, device=dev)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=dev) if lse is None else lse
    q_rot = torch.empty_like(q) if q_rot is None else q_rot
    k_rot = torch.empty_like(k) if k_rot is None else k_rot
    _need("out", out, (B, N, H, D), device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    _need("q_rot", q_rot, (B, N, H, D), device=dev)
    _need("k_rot", k_rot, (B, N, Hkv, D), device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_fwd_rope(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                  q_rot.data_ptr(), k_rot.data_ptr(), table.data_ptr(), B, H, Hkv, N, D,
                                  int(group_size), _stream(dev))
    _lib._check("s2attn_fwd_rope", st)
    return out, lse, q_rot, k_rot


def s2attn_backward_rope(q_rot, k_rot, v, o, lse, do, group_size: int, table, dq=None, dk=None, dv=None,
                         workspace=None):
    """Backward of s2attn_forward_rope: gradients with respect to the
    unrotated q and k, and v.  Returns (dq, dk, dv)."""
    B, N, H, Hkv, D = _dims(q_rot, k_rot)
    _need("q_rot", q_rot, (B, N, H, D))
    dev = q_rot.device
    for name, t, shp in (("k_rot", k_rot, (B, N, Hkv, D)), ("v", v, (B, N, Hkv, D)),
                         ("o", o, (B, N, H, D)), ("do", do, (B, N, H, D))):
        _need(name, t, shp, device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    _need("table", table, (N, D // 2, 2), torch.float32, device=dev)
    dq = torch.empty_like(q_rot) if dq is None else dq
    dk = torch.empty_like(k_rot) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t, shp in (("dq", dq, (B, N, H, D)), ("dk", dk, (B, N, Hkv, D)), ("dv", dv, (B, N, Hkv, D))):
        _need(name, t, shp, device=dev)
    wsb = bwd_workspace_bytes(B, H, Hkv, N, D, group_size)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if workspace.numel() * workspace.element_size() < wsb:
        raise _lib.S2AttnError("s2attn_bwd_rope", _lib.S2ATTN_ERR_WORKSPACE)
    with torch.cuda.device(dev):
        st = _lib.s2attn_bwd_rope(q_rot.data_ptr(), k_rot.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                  do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), table.data_ptr(),
                                  B, H, Hkv, N, D, int(group_size), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream(dev))
    _lib._check("s2attn_bwd_rope", st)
    return dq, dk, dv


class S2RopeAttention(torch.autograd.Function):
    """Autograd wrapper: RoPE with Position Interpolation, then S2 attention."""

    @staticmethod
    def forward(ctx, q, k, v, group_size, table):
        o, lse, q_rot, k_rot = s2attn_forward_rope(q, k, v, group_size, table)
        ctx.save_for_backward(q_rot, k_rot, v, o, lse, table)
        ctx.group_size = group_size
        return o

    @staticmethod
    def backward(ctx, do):
        q_rot, k_rot, v, o, lse, table = ctx.saved_tensors
        dq, dk, dv = s2attn_backward_rope(q_rot, k_rot, v, o, lse, do.contiguous(), ctx.group_size, table)
        return dq, dk, dv, None, None


def seg_forward(q, k, v, causal: bool = True, out=None, lse=None):
    """Attention of a chunk's queries q [B, N, H, D] over keys k, v [B, Nk, Hkv, D]:
    causal -- row i sees keys [0, Nk - N + i] (the earlier keys, then its own
    chunk causally); not causal -- every key (a detached segment as a piece).
    Returns (o, lse) of that attention."""
    B, N, H, Hkv, D = _dims(q, k)
    Nk = k.shape[1]
    _need("q", q, (B, N, H, D))
    dev = q.device
    _need("k", k, (B, Nk, Hkv, D), device=dev)
    _need("v", v, (B, Nk, Hkv, D), device=dev)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=dev) if lse is None else lse
    _need("out", out, (B, N, H, D), device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_seg_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                 B, H, Hkv, N, Nk, D, int(causal), _stream(dev))
    _lib._check("s2attn_seg_fwd", st)
    return out, lse


def seg_backward(q, k, v, o, lse, do, causal: bool = True, dq=None, dk=None, dv=None, dq_accumulate=False,
                 workspace=None):
    """Backward of seg_forward given the chunk rows' final o and lse: dq, and
    (causal) dk, dv of the chunk's own keys -- the last N key rows.  Not
    causal: dq only (dk, dv returned as None).  dq_accumulate adds into dq."""
    B, N, H, Hkv, D = _dims(q, k)
    Nk = k.shape[1]
    _need("q", q, (B, N, H, D))
    dev = q.device
    for name, t, shp in (("k", k, (B, Nk, Hkv, D)), ("v", v, (B, Nk, Hkv, D)), ("o", o, (B, N, H, D)),
                         ("do", do, (B, N, H, D))):
        _need(name, t, shp, device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    if dq is None:
        if dq_accumulate:
            raise ValueError("dq_accumulate needs dq")
        dq = torch.empty_like(q)
    _need("dq", dq, (B, N, H, D), device=dev)
    if causal:
        dk = torch.empty((B, N, Hkv, D), dtype=k.dtype, device=dev) if dk is None else dk
        dv = torch.empty((B, N, Hkv, D), dtype=v.dtype, device=dev) if dv is None else dv
        _need("dk", dk, (B, N, Hkv, D), device=dev)
        _need("dv", dv, (B, N, Hkv, D), device=dev)
    else:
        dk = dv = None
    wsb = _lib.s2attn_seg_bwd_workspace_bytes(B, H, Hkv, N, Nk, D)
    if wsb == 0:
        raise _lib.S2AttnError("s2attn_seg_bwd_workspace_bytes", _lib.S2ATTN_ERR_INVALID_ARG)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_seg_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 do.data_ptr(), dq.data_ptr(), None if dk is None else dk.data_ptr(),
                                 None if dv is None else dv.data_ptr(), B, H, Hkv, N, Nk, D, int(causal),
                                 int(dq_accumulate), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(dev))
    _lib._check("s2attn_seg_bwd", st)
    return dq, dk, dv


def lse_merge(o_a, lse_a, o_b, lse_b, out=None, lse=None):
    """Attention over the union of two disjoint key sets from the two pieces'
    (o, lse); out / lse may be o_a / lse_a (in place)."""
    B, N, H, D = o_a.shape
    dev = o_a.device
    _need("o_a", o_a, (B, N, H, D))
    _need("o_b", o_b, (B, N, H, D), device=dev)
    _need("lse_a", lse_a, (B, H, N), torch.float32, device=dev)
    _need("lse_b", lse_b, (B, H, N), torch.float32, device=dev)
    out = torch.empty_like(o_a) if out is None else out
    lse = torch.empty_like(lse_a) if lse is None else lse
    _need("out", out, (B, N, H, D), device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_lse_merge(o_a.data_ptr(), lse_a.data_ptr(), o_b.data_ptr(), lse_b.data_ptr(),
                                   out.data_ptr(), lse.data_ptr(), B, H, N, D, _stream(dev))
    _lib._check("s2attn_lse_merge", st)
    return out, lse


def _need_hist(hist, B, N, dev):
    if not isinstance(hist, torch.Tensor) or hist.dtype != torch.int32 or hist.dim() != 3:
        raise ValueError("hist must be an int32 tensor [B, N/256, S]")
    if hist.device != dev or not hist.is_contiguous() or tuple(hist.shape[:2]) != (B, N // 256):
        raise ValueError(f"hist must be a contiguous [B, N/256, S] tensor on {dev}")


def hga_forward(q, k, v, group_size: int, hist, out=None, lse=None):
    """HGA-style block-sparse attention: each row attends its own segment
    (group_size rows, no shift) causally and the historical key tiles listed
    for its 256-row query block in hist (int32 [B, N/256, S], tile indices of
    earlier segments; a list ends at its first other entry, e.g. -1)."""
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    _need("k", k, (B, N, Hkv, D), device=dev)
    _need("v", v, (B, N, Hkv, D), device=dev)
    _need_hist(hist, B, N, dev)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=dev) if lse is None else lse
    _need("out", out, (B, N, H, D), device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_hga_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                 hist.data_ptr(), hist.shape[2], B, H, Hkv, N, D, int(group_size), _stream(dev))
    _lib._check("s2attn_hga_fwd", st)
    return out, lse


def hga_backward(q, k, v, o, lse, do, group_size: int, hist, dq=None, dk=None, dv=None, workspace=None):
    """Backward of hga_forward: dq through every attended key; dk, dv through
    the local attention only (the historical keys are detached)."""
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    for name, t, shp in (("k", k, (B, N, Hkv, D)), ("v", v, (B, N, Hkv, D)), ("o", o, (B, N, H, D)),
                         ("do", do, (B, N, H, D))):
        _need(name, t, shp, device=dev)
    _need("lse", lse, (B, H, N), torch.float32, device=dev)
    _need_hist(hist, B, N, dev)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    wsb = _lib.s2attn_hga_bwd_workspace_bytes(B, H, Hkv, N, D, int(group_size))
    if wsb == 0:
        raise _lib.S2AttnError("s2attn_hga_bwd_workspace_bytes", _lib.S2ATTN_ERR_INVALID_ARG)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_hga_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), hist.data_ptr(),
                                 hist.shape[2], B, H, Hkv, N, D, int(group_size), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(dev))
    _lib._check("s2attn_hga_bwd", st)
    return dq, dk, dv


class ChunkAttention(torch.autograd.Function):
    """Chunk-wise training step: the chunk's queries attend its own keys
    causally and the detached earlier keys fully; the two pieces are merged by
    log-sum-exp and only q, k_act, v_act receive gradients."""

    @staticmethod
    def forward(ctx, q, k_act, v_act, k_past, v_past):
        o_a, lse_a = seg_forward(q, k_past, v_past, causal=False)
        o_b, lse_b = seg_forward(q, k_act, v_act, causal=True)
        o, lse = lse_merge(o_a, lse_a, o_b, lse_b, out=o_a, lse=lse_a)
        ctx.save_for_backward(q, k_act, v_act, k_past, v_past, o, lse)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k_act, v_act, k_past, v_past, o, lse = ctx.saved_tensors
        do = do.contiguous()
        dq, _, _ = seg_backward(q, k_past, v_past, o, lse, do, causal=False)
        dq, dk, dv = seg_backward(q, k_act, v_act, o, lse, do, causal=True, dq=dq, dq_accumulate=True)
        return dq, dk, dv, None, None


class S2Attention(torch.autograd.Function):
    """Autograd wrapper: the drop-in attention call of a training step."""

    @staticmethod
    def forward(ctx, q, k, v, group_size):
        o, lse = s2attn_forward(q, k, v, group_size)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.group_size = group_size
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = s2attn_backward(q, k, v, o, lse, do.contiguous(), ctx.group_size)
        return dq, dk, dv, None


def s2_attn(q, k, v, group_size: int):
    """Shifted sparse attention with autograd (training path)."""
    return S2Attention.apply(q, k, v, group_size)


def dense_causal_attn(q, k, v):
    """Dense causal attention through the same kernels (G = N, no shift)."""
    return S2Attention.apply(q, k, v, q.shape[1])


# ---------------------------------------------------------------- NF4 QKV projection

def _need_nf4(codes, scale_codes, c2, rows: int, K: int, dev) -> None:
    _need("codes", codes, (rows, K // 2), torch.uint8, device=dev)
    _need("scale_codes", scale_codes, (rows * (K // 64),), torch.int8, device=dev)
    _need("c2", c2, ((rows * (K // 64) + 255) // 256,), torch.float32, device=dev)


def nf4_levels():
    """The 16 NF4 levels the kernels use (ascending; index = 4-bit code)."""
    return _lib.s2attn_nf4_levels()


def nf4_qkv(x, codes, scale_codes, c2, n_heads: int, n_kv_heads: int, head_dim: int, q=None, k=None, v=None):
    """q, k, v = the QKV projection of x (bf16 [B, N, K]) through NF4 weights
    with double quantization, dequantized inside the tensor-core GEMM.  The
    weight is [(H + 2 Hkv) D, K]: codes uint8 [rows, K/2] (two 4-bit codes a
    byte, the even element in the low nibble), scale_codes int8 [rows K/64],
    c2 fp32 [ceil(rows K/64 / 256)].  Returns bf16 [B, N, H, D], [B, N, Hkv, D],
    [B, N, Hkv, D]."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, N, K] tensor")
    B, N, K = x.shape
    H, Hkv, D = int(n_heads), int(n_kv_heads), int(head_dim)
    dev = x.device
    _need("x", x, (B, N, K))
    rows = (H + 2 * Hkv) * D
    _need_nf4(codes, scale_codes, c2, rows, K, dev)
    q = torch.empty((B, N, H, D), dtype=torch.bfloat16, device=dev) if q is None else q
    k = torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device=dev) if k is None else k
    v = torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device=dev) if v is None else v
    _need("q", q, (B, N, H, D), device=dev)
    _need("k", k, (B, N, Hkv, D), device=dev)
    _need("v", v, (B, N, Hkv, D), device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_nf4_qkv(x.data_ptr(), codes.data_ptr(), scale_codes.data_ptr(), c2.data_ptr(), q.data_ptr(),
                                 k.data_ptr(), v.data_ptr(), B * N, K, H, Hkv, D, _stream(dev))
    _lib._check("s2attn_nf4_qkv", st)
    return q, k, v


def nf4_dequantize(codes, scale_codes, c2, out=None):
    """The dequantized weight W' (bf16 [rows, K]) of NF4 codes [rows, K/2]."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be a [rows, K/2] tensor")
    rows, K = codes.shape[0], 2 * codes.shape[1]
    dev = codes.device
    _need_nf4(codes, scale_codes, c2, rows, K, dev)
    out = torch.empty((rows, K), dtype=torch.bfloat16, device=dev) if out is None else out
    _need("out", out, (rows, K), device=dev)
    with torch.cuda.device(dev):
        st = _lib.s2attn_nf4_dequant(codes.data_ptr(), scale_codes.data_ptr(), c2.data_ptr(), out.data_ptr(), rows, K,
                                     _stream(dev))
    _lib._check("s2attn_nf4_dequant", st)
    return out


def _run(dev, fn: str, *args) -> None:
    """One C call with `dev` current, on its current stream.  The device guard
    is entered only where it changes something: the smallest calls take a few
    microseconds on the GPU, and the guard as long on the host."""
    if torch._C._cuda_getDevice() == dev.index:
        st = getattr(_lib.load(), fn)(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = getattr(_lib.load(), fn)(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st != _lib.S2ATTN_OK:
        _lib._check(fn, st)


# ---------------------------------------------------------------- query/key norm with rotation

def _need_norm_weights(w_q, w_k, D: int, dev) -> int:
    """Checks the two [D] norm weights; 1 for fp32, 0 for bf16."""
    dtype = getattr(w_q, "dtype", None)
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise ValueError(f"w_q must be a torch.float32 or torch.bfloat16 tensor, got {dtype}")
    shape = (D,)
    _need("w_q", w_q, shape, dtype, dev)
    _need("w_k", w_k, shape, dtype, dev)
    return 1 if dtype is torch.float32 else 0


def qknorm_rope_forward(q, k, w_q, w_k, table, eps: float = 1e-6, q_out=None, k_out=None):
    """Root-mean-square norm of every query and key head, weighted by w_q and
    w_k ([D], fp32 or bf16), and the rotation by the table, in one pass.
    q [B, N, H, D], k [B, N, Hkv, D] bf16; any N.  Returns (q_out, k_out), which
    s2attn_forward takes; q_out may be q and k_out may be k (in place)."""
    if q_out is None and k_out is None:
        r = _fast.qknorm_fwd(q, k, w_q, w_k, table, eps)
        if r is not None:
            return r
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    _need("k", k, (B, N, Hkv, D), device=dev)
    w32 = _need_norm_weights(w_q, w_k, D, dev)
    _need("table", table, (N, D // 2, 2), torch.float32, dev)
    q_out = _out("q_out", q_out, q)
    k_out = _out("k_out", k_out, k)
    _run(dev, "s2attn_qknorm_rope_fwd", q.data_ptr(), k.data_ptr(), w_q.data_ptr(), w_k.data_ptr(), table.data_ptr(),
         q_out.data_ptr(), k_out.data_ptr(), B, N, H, Hkv, D, w32, float(eps))
    return q_out, k_out


def qknorm_rope_backward(q, k, w_q, w_k, dq_out, dk_out, table, eps: float = 1e-6, dq=None, dk=None, dw_q=None,
                         dw_k=None, workspace=None):
    """Backward of qknorm_rope_forward from its inputs and the gradients of its
    outputs.  Returns (dq, dk, dw_q, dw_k); the weight gradients have the
    weights' type.  dq may be dq_out and dk may be dk_out (in place)."""
    if dq is None and dk is None and dw_q is None and dw_k is None and workspace is None:
        r = _fast.qknorm_bwd(q, k, w_q, w_k, dq_out, dk_out, table, eps)
        if r is not None:
            return r
    B, N, H, Hkv, D = _dims(q, k)
    _need("q", q, (B, N, H, D))
    dev = q.device
    _need("k", k, (B, N, Hkv, D), device=dev)
    _need("dq_out", dq_out, (B, N, H, D), device=dev)
    _need("dk_out", dk_out, (B, N, Hkv, D), device=dev)
    w32 = _need_norm_weights(w_q, w_k, D, dev)
    _need("table", table, (N, D // 2, 2), torch.float32, dev)
    dq, dk = _out("dq", dq, q), _out("dk", dk, k)
    dw_q, dw_k = _out("dw_q", dw_q, w_q), _out("dw_k", dw_k, w_k)
    workspace, wsb = _workspace("s2attn_qknorm_rope_bwd", workspace, _lib.s2attn_qknorm_rope_bwd_workspace_bytes(D),
                                dev)
    _run(dev, "s2attn_qknorm_rope_bwd", q.data_ptr(), k.data_ptr(), w_q.data_ptr(), w_k.data_ptr(), table.data_ptr(),
         dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), dw_q.data_ptr(), dw_k.data_ptr(), B, N,
         H, Hkv, D, w32, float(eps), workspace.data_ptr(), wsb)
    return dq, dk, dw_q, dw_k


def _optional(name: str, t):
    """Address of an optional operand, None without it.  The C calls take a null
    address for its absence, so a tensor without memory (inside
    torch.func.functionalize) is refused."""
    if t is None:
        return None
    p = t.data_ptr()
    if p == 0 and t.numel() > 0:
        raise ValueError(f"{name} has no memory")
    return p


def _out(name: str, t, like):
    """The caller's output checked against the tensor it is shaped like, or a new one."""
    if t is None:
        return torch.empty_like(like)
    _need(name, t, like.shape, like.dtype, device=like.device)
    return t


def _workspace(fn: str, workspace, need: int, dev):
    """The caller's workspace checked, or a new one; and its size."""
    if need == 0:
        raise _lib.S2AttnError(fn, _lib.S2ATTN_ERR_UNSUPPORTED)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    have = workspace.numel() * workspace.element_size()
    if have < need:
        raise _lib.S2AttnError(fn, _lib.S2ATTN_ERR_WORKSPACE)
    return workspace, have


class QKNormRope(torch.autograd.Function):
    """Autograd wrapper of the query/key norm with rotation: gradients for q,
    k and both norm weights (once: the gradient itself has none).  To capture a
    training step into a CUDA graph, call qknorm_rope_forward / _backward, or
    capture with torch.autograd.grad while no eager graph of the same leaves is
    alive: a leaf's gradient accumulation stays on the stream that first used
    it."""

    @staticmethod
    def forward(ctx, q, k, w_q, w_k, table, eps=1e-6):
        q_out, k_out = qknorm_rope_forward(q, k, w_q, w_k, table, eps)
        ctx.save_for_backward(q, k, w_q, w_k, table)
        ctx.eps = eps
        return q_out, k_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, w_q, w_k, table = ctx.saved_tensors
        dq, dk, dw_q, dw_k = qknorm_rope_backward(q, k, w_q, w_k, dq_out.contiguous(), dk_out.contiguous(), table,
                                                  ctx.eps)
        return dq, dk, dw_q, dw_k, None, None


def s2_qknorm_attn(q, k, v, w_q, w_k, group_size: int, table, eps: float = 1e-6):
    """Shifted sparse attention on normed and rotated q and k, with autograd
    (training path of layers with query/key norm)."""
    q_rot, k_rot = QKNormRope.apply(q, k, w_q, w_k, table, eps)
    return S2Attention.apply(q_rot, k_rot, v, group_size)


# ---------------------------------------------------------------- decoding over a paged cache

class CachePlan(NamedTuple):
    """Where the new tokens of a step go (int32 CUDA tensors, mask int64)."""
    cu_seqlens: torch.Tensor          # [R + 1] first token of each request, and the total
    positions: torch.Tensor           # [T] position for the rotation
    slots: torch.Tensor               # [T] slot in the cache, -1: none
    mask: Optional[torch.Tensor]      # [T] visible drafts of a tree, None without parents
    counts: torch.Tensor              # [4] free blocks taken (the first ones), needed, new tokens, those without a block


def cache_plan(ctx_lens, new_lens, block_tables, free_blocks, block_size: int, num_tokens: int, parents=None):
    """Blocks, slots and positions for the new tokens of a ragged batch, on the
    GPU.  ctx_lens, new_lens int32 [R]: tokens in the cache and tokens to add;
    block_tables int32 [R, max_blocks]: the requests' blocks, extended in place
    by blocks of free_blocks (int32, taken from its front in request order: drop
    its first counts[0] entries before the next step); num_tokens: size of the
    token arrays, at least sum(new_lens) (tokens behind it are dropped).  parents
    int32 [num_tokens]: the new tokens of each request are a tree of drafts,
    parents[t] the index in the request of the draft before it, -1 for the
    context.  Returns a CachePlan."""
    r = _fast.cache_plan(ctx_lens, new_lens, block_tables, free_blocks, block_size, num_tokens, parents)
    if r is not None:
        return CachePlan(*r)
    if not isinstance(ctx_lens, torch.Tensor) or ctx_lens.dim() != 1:
        raise ValueError("ctx_lens must be an int32 tensor [R]")
    R, T = ctx_lens.shape[0], int(num_tokens)
    _need("ctx_lens", ctx_lens, (R,), torch.int32)
    dev = ctx_lens.device
    _need("new_lens", new_lens, (R,), torch.int32, dev)
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise ValueError("block_tables must be an int32 tensor [R, max_blocks]")
    _need("block_tables", block_tables, (R, block_tables.shape[1]), torch.int32, dev)
    if not isinstance(free_blocks, torch.Tensor) or free_blocks.dim() != 1:
        raise ValueError("free_blocks must be an int32 tensor [num_free]")
    _need("free_blocks", free_blocks, (free_blocks.shape[0],), torch.int32, dev)
    if parents is not None:
        _need("parents", parents, (T,), torch.int32, dev)
    if T <= 0:
        raise _lib.S2AttnError("s2attn_cache_plan", _lib.S2ATTN_ERR_INVALID_ARG)
    mask = None if parents is None else torch.empty(T, dtype=torch.int64, device=dev)
    buf = torch.empty(2 * T + R + 5, dtype=torch.int32, device=dev)  # one allocation
    positions, slots, cu_seqlens, counts = buf.split_with_sizes((T, T, R + 1, 4))
    p = buf.data_ptr()
    _run(dev, "s2attn_cache_plan", ctx_lens.data_ptr(), new_lens.data_ptr(), block_tables.data_ptr(),
         free_blocks.data_ptr(), _optional("parents", parents), p + 8 * T, p, p + 4 * T, None if
         mask is None else mask.data_ptr(), p + 4 * (2 * T + R + 1), R, block_tables.shape[1], free_blocks.shape[0],
         int(block_size), T)
    return CachePlan(cu_seqlens, positions, slots, mask, counts)


def _need_cache(k_cache, v_cache, Hkv, D, dev):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a [num_blocks, block_size, Hkv, D] tensor")
    nb, bs, heads, _ = k_cache.shape
    shape = (nb, bs, heads if Hkv is None else Hkv, D)
    _need("k_cache", k_cache, shape, torch.bfloat16, dev)
    _need("v_cache", v_cache, shape, torch.bfloat16, dev)
    return nb, bs, heads


def cache_append(q, k, v, table, positions, slots, k_cache, v_cache, w_q=None, w_k=None, eps: float = 1e-6,
                 q_out=None):
    """The serving form of qknorm_rope_forward: q [T, H, D], k and v
    [T, Hkv, D] bf16, the new tokens of a ragged batch, are rotated by the
    table's rows at positions (int32 [T]) -- after the norm where w_q and w_k
    are given -- and k and v written to the caches ([num_blocks, block_size,
    Hkv, D] bf16) at slots (int32 [T]).  Tokens with a negative slot are
    padding: nothing is written for them.  No two tokens may share a slot.
    Returns q_out (may be q)."""
    r = _fast.cache_append(q, k, v, table, positions, slots, k_cache, v_cache, w_q, w_k, eps, q_out)
    if r is not None:
        return r
    if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor) or q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, H, D] and k [T, Hkv, D]")
    T, H, D = q.shape
    Hkv = k.shape[1]
    _need("q", q, (T, H, D))
    dev = q.device
    _need("k", k, (T, Hkv, D), device=dev)
    _need("v", v, (T, Hkv, D), device=dev)
    _need("positions", positions, (T,), torch.int32, dev)
    _need("slots", slots, (T,), torch.int32, dev)
    nb, bs, _ = _need_cache(k_cache, v_cache, Hkv, D, dev)
    if not isinstance(table, torch.Tensor) or table.dim() != 3:
        raise ValueError("table must be a [rows, D/2, 2] tensor (rope_table)")
    rows = table.shape[0]
    _need("table", table, (rows, D // 2, 2), torch.float32, dev)
    if (w_q is None) != (w_k is None):
        raise ValueError("w_q and w_k go together")
    w32 = 0 if w_q is None else _need_norm_weights(w_q, w_k, D, dev)
    q_out = _out("q_out", q_out, q)
    _run(dev, "s2attn_cache_append", q.data_ptr(), k.data_ptr(), v.data_ptr(), _optional("w_q", w_q),
         _optional("w_k", w_k), table.data_ptr(), positions.data_ptr(), slots.data_ptr(), q_out.data_ptr(),
         k_cache.data_ptr(), v_cache.data_ptr(), T, H, Hkv, D, rows, nb * bs, w32, float(eps))
    return q_out


def cache_attention(q, k_cache, v_cache, block_tables, ctx_lens, cu_seqlens, mask=None, out=None, lse=None,
                    workspace=None):
    """Attention of the new tokens of a ragged batch over a paged cache that
    already holds their keys and values.  q [T, H, D] bf16; request i owns rows
    cu_seqlens[i] .. cu_seqlens[i+1] of q (int32 [R + 1]), has ctx_lens[i]
    earlier keys (int32 [R]) and the blocks of row i of block_tables (int32
    [R, max_blocks]).  Every row attends the earlier keys and, of the request's
    new ones, those its mask (int64 [T], bit j = new token j) names -- without
    mask those up to its own.  Returns (o [T, H, D] bf16, lse [H, T] fp32); rows
    that see no key get 0 and -inf, rows of no request are left as they are.  The
    softmax weights are rounded to bf16 for the product with V, all else is fp32.
    The number of tokens, of requests and the tables' width choose the kernel:
    tables no wider than the step's longest request, and no idle requests or
    padding, are the fastest."""
    if out is None and lse is None and workspace is None:
        r = _fast.cache_attention(q, k_cache, v_cache, block_tables, ctx_lens, cu_seqlens, mask)
        if r is not None:
            return r
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [T, H, D] tensor")
    T, H, D = q.shape
    _need("q", q, (T, H, D))
    dev = q.device
    nb, bs, Hkv = _need_cache(k_cache, v_cache, None, D, dev)
    if not isinstance(block_tables, torch.Tensor) or block_tables.dim() != 2:
        raise ValueError("block_tables must be an int32 tensor [R, max_blocks]")
    R, maxb = block_tables.shape
    _need("block_tables", block_tables, (R, maxb), torch.int32, dev)
    _need("ctx_lens", ctx_lens, (R,), torch.int32, dev)
    _need("cu_seqlens", cu_seqlens, (R + 1,), torch.int32, dev)
    if mask is not None:
        _need("mask", mask, (T,), torch.int64, device=dev)
    out = _out("out", out, q)
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=dev)
    else:
        _need("lse", lse, (H, T), torch.float32, device=dev)
    workspace, wsb = _workspace("s2attn_cache_attn", workspace, _lib.s2attn_cache_attn_workspace_bytes(D), dev)
    _run(dev, "s2attn_cache_attn", q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
         ctx_lens.data_ptr(), cu_seqlens.data_ptr(), _optional("mask", mask), out.data_ptr(),
         lse.data_ptr(), T, R, H, Hkv, D, nb, bs, maxb, workspace.data_ptr(), wsb)
    return out, lse

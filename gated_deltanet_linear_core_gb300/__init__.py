"""Gated DeltaNet (GDN) linear-attention layer core for GB300 (sm_103a).

A thin binding of the C ABI in include/gdn.h (libgdn.so, hand-written CUDA
kernels).  The functions below only marshal arguments: they check tensor
placement and layout, allocate outputs with torch when the caller passes none,
and call the library on the current CUDA stream.  Every step of the layer runs
in the library's kernels; if libgdn.so is missing, every call raises.

Layer core (cortex commit "feat(stage-8c): linear-attention layer (Qwen3-Next
GatedDeltaNet)"): conv1d(k=4)+SiLU -> split [q|k|v] -> l2norm(q,k), gates
g = -exp(A_log) softplus(a+dt_bias), beta = sigmoid(b) -> gated delta rule
(chunked prefill or per-token decode) -> RMSNormGated(o, z).
"""
from __future__ import annotations

from dataclasses import dataclass
from functools import lru_cache

import torch

from . import _lib
from ._lib import GDNError, GDN_QK_L2NORM, GDN_SOLVE_NEUMANN, GDN_CHUNK  # noqa: F401

__all__ = [
    "GDNDims", "GDNError", "gdn_conv1d_fwd", "gdn_conv1d_update", "gdn_chunk_prefill",
    "gdn_chunk_prefill_workspace_size", "gdn_chunk_prefill_launches", "gdn_chunk_prefill_noalloc", "gdn_recurrent_decode", "gdn_rmsnorm_gated",
    "gdn_ckpt_count", "gdn_check_cu_seqlens", "gdn_sync_status", "gdn_selftest_bounded_wait",
    "gdn_layer_prefill_host", "gdn_decode_step", "gdn_decode_verify", "gdn_layer_prefill",
    "gdn_layer_prefill_workspace_size", "gdn_layer_prefill_launches", "gdn_chunk_prefill_norm",
    "HeadShard", "head_shard",
    "gdn_layer_decode", "gdn_kv_append", "gdn_rope", "gdn_rope_kv_append", "gdn_attn_decode", "gdn_attn_decode_workspace_size",
    "gdn_attn_decode_shared", "gdn_attn_decode_shared_workspace_size", "gdn_draft_accept",
    "library_path",
]

RMSNORM_EPS = 1e-6


@dataclass(frozen=True)
class GDNDims:
    """H_k query/key heads, H_v value heads, head dims d_k = d_v, conv width 4."""
    H_k: int
    H_v: int
    d_k: int
    d_v: int
    conv_k: int = 4

    @property
    def conv_dim(self) -> int:
        return 2 * self.H_k * self.d_k + self.H_v * self.d_v


def library_path() -> str:
    return _lib.LIB_PATH


def _dims(d) -> _lib.Dims:
    return _lib.Dims(int(d.H_k), int(d.H_v), int(d.d_k), int(d.d_v), int(getattr(d, "conv_k", 4)))


def _conv_dim(d) -> int:
    return 2 * int(d.H_k) * int(d.d_k) + int(d.H_v) * int(d.d_v)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _lib.GDN_BF16
    if t.dtype == torch.float32:
        return _lib.GDN_F32
    raise TypeError(f"unsupported activation dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t, name, dtype=None, shape=None):
    """Device pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr() if t.numel() else None


def _stream(t: torch.Tensor, stream):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.current_stream(t.device).cuda_stream


def _nseq(cu_seqlens):
    return 1 if cu_seqlens is None else int(cu_seqlens.numel()) - 1


def gdn_ckpt_count(cu_seqlens, every: int) -> int:
    """Checkpoint rows for packed sequences (host offsets: list, numpy or CPU tensor)."""
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int32, device="cpu").contiguous()
    r = _lib.load().gdn_ckpt_count(cu.data_ptr(), int(cu.numel()) - 1, int(every))
    if r < 0:
        raise ValueError("invalid cu_seqlens or checkpoint interval")
    return int(r)


def gdn_check_cu_seqlens(cu_seqlens: torch.Tensor, T_tot: int, stream=None) -> None:
    """Validates device offsets (synchronises the stream)."""
    p = _ptr(cu_seqlens, "cu_seqlens", torch.int32)
    _lib.check(_lib.load().gdn_check_cu_seqlens(p, _nseq(cu_seqlens), int(T_tot),
                                               _stream(cu_seqlens, stream)),
               "gdn_check_cu_seqlens")


def gdn_sync_status(device=None, stream=None) -> None:
    """Synchronises the stream and raises GDNError if a kernel gave up a
    bounded device-side wait (GDN_ERR_TIMEOUT) or the stream holds a CUDA error."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _lib.check(_lib.load().gdn_sync_status(s), "gdn_sync_status")


def gdn_selftest_bounded_wait(limit_ns: int = 1_000_000, device=None, stream=None) -> None:
    """Enqueues one kernel whose bounded wait runs out after limit_ns (nothing
    arrives at its barrier); the next gdn_sync_status raises GDN_ERR_TIMEOUT."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _lib.check(_lib.load().gdn_selftest_bounded_wait(int(limit_ns), s), "gdn_selftest_bounded_wait")


def gdn_conv1d_fwd(x, w, dims, cu_seqlens=None, conv_state_in=None, conv_state_out=None,
                   ckpt_every=0, conv_ckpt_out=None, apply_silu=True, y=None, stream=None):
    """Prefill depthwise causal conv1d(k=4) with state prepend (+SiLU).
    x [T, conv_dim]; w [conv_dim, 4]; states [n_seq, conv_dim, 3];
    checkpoints [rows, conv_dim, 3].  Returns y [T, conv_dim]."""
    dt = x.dtype
    T, C = x.shape
    if C != _conv_dim(dims):
        raise ValueError(f"x has {C} channels, dims give {_conv_dim(dims)}")
    if y is None:
        y = torch.empty_like(x)
    rows = 0 if conv_ckpt_out is None else int(conv_ckpt_out.shape[0])
    st = _lib.load().gdn_conv1d_fwd(
        _ptr(x, "x", dt), _ptr(w, "w", dt, (C, 4)), _ptr(cu_seqlens, "cu_seqlens", torch.int32),
        _nseq(cu_seqlens), T, _ptr(conv_state_in, "conv_state_in", dt),
        _ptr(conv_state_out, "conv_state_out", dt), int(ckpt_every),
        _ptr(conv_ckpt_out, "conv_ckpt_out", dt), rows, int(bool(apply_silu)),
        _ptr(y, "y", dt, (T, C)), _dims(dims), _dtype_code(x), _stream(x, stream))
    _lib.check(st, "gdn_conv1d_fwd")
    return y


def gdn_conv1d_update(x, w, conv_state, dims, apply_silu=True, y=None, stream=None):
    """Decode conv for B sequences; conv_state [B, conv_dim, 3] shifted in place."""
    dt = x.dtype
    B, C = x.shape
    if y is None:
        y = torch.empty_like(x)
    st = _lib.load().gdn_conv1d_update(
        _ptr(x, "x", dt), _ptr(w, "w", dt, (C, 4)), _ptr(conv_state, "conv_state", dt, (B, C, 3)),
        B, int(bool(apply_silu)), _ptr(y, "y", dt, (B, C)), _dims(dims), _dtype_code(x),
        _stream(x, stream))
    _lib.check(st, "gdn_conv1d_update")
    return y


def gdn_chunk_prefill_workspace_size(n_seq: int, T_tot: int, dims, dtype) -> int:
    code = _lib.GDN_BF16 if dtype == torch.bfloat16 else _lib.GDN_F32
    return int(_lib.load().gdn_chunk_prefill_workspace_size(int(n_seq), int(T_tot), _dims(dims),
                                                            code))


def gdn_chunk_prefill_launches(n_seq: int, T_tot: int, dims, dtype, cu_seqlens=True, chunk=64) -> int:
    """Kernel launches of one gdn_chunk_prefill call; cu_seqlens: whether the
    call passes cu_seqlens (a truthy value) or not (None / False); chunk: its
    chunk size (16, 32 or 64)."""
    code = _lib.GDN_BF16 if dtype == torch.bfloat16 else _lib.GDN_F32
    has_cu = 0 if cu_seqlens is None or cu_seqlens is False else 1
    return int(_lib.load().gdn_chunk_prefill_launches(int(n_seq), int(T_tot), has_cu, _dims(dims), code,
                                                      _flags(False, "direct", chunk)))


def _flags(l2norm_qk, solve, chunk) -> int:
    if solve not in ("direct", "neumann"):
        raise ValueError(f"solve must be 'direct' or 'neumann', not {solve!r}")
    return ((_lib.GDN_QK_L2NORM if l2norm_qk else 0) | (_lib.GDN_SOLVE_NEUMANN if solve == "neumann" else 0) |
            (0 if chunk == 64 else _lib.GDN_CHUNK(chunk)))


def _gate_ptrs(a, b, A_log, dt_bias, g, beta, dt):
    return (_ptr(a, "a", dt), _ptr(b, "b", dt), _ptr(A_log, "A_log", torch.float32),
            _ptr(dt_bias, "dt_bias", torch.float32), _ptr(g, "g", torch.float32),
            _ptr(beta, "beta", torch.float32))


def gdn_chunk_prefill(qkv, dims, a=None, b=None, A_log=None, dt_bias=None, g=None, beta=None,
                      cu_seqlens=None, initial_state=None, final_state=None, ckpt_every=0,
                      state_ckpt_out=None, scale=0.0, l2norm_qk=True, o=None, workspace=None,
                      stream=None, solve="direct", chunk=64):
    """Chunked gated delta rule over packed sequences.  qkv [T, conv_dim]
    (post-conv); states [n_seq, H_v, d_k, d_v] f32; returns o [T, H_v, d_v].
    solve="neumann" forms each chunk's (I + A)^-1 as the Neumann-style product
    (GDN_SOLVE_NEUMANN; tensor-core path only).  chunk: 16, 32 or 64 tokens
    (GDN_CHUNK; on the tensor-core path 16 and 32 need final_state)."""
    if solve not in ("direct", "neumann"):
        raise ValueError(f"solve must be 'direct' or 'neumann', not {solve!r}")
    dt = qkv.dtype
    T = int(qkv.shape[0])
    if o is None:
        o = torch.empty((T, dims.H_v, dims.d_v), dtype=dt, device=qkv.device)
    rows = 0 if state_ckpt_out is None else int(state_ckpt_out.shape[0])
    lib = _lib.load()
    if workspace is None:
        need = lib.gdn_chunk_prefill_workspace_size(_nseq(cu_seqlens), T, _dims(dims),
                                                    _dtype_code(qkv))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=qkv.device)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.gdn_chunk_prefill(
        _ptr(qkv, "qkv", dt), *_gate_ptrs(a, b, A_log, dt_bias, g, beta, dt),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _nseq(cu_seqlens), T,
        _ptr(initial_state, "initial_state", torch.float32),
        _ptr(final_state, "final_state", torch.float32), int(ckpt_every),
        _ptr(state_ckpt_out, "state_ckpt_out", torch.float32), rows, float(scale),
        _flags(l2norm_qk, solve, chunk), _ptr(o, "o", dt), _ptr(workspace, "workspace"),
        ws, _dims(dims), _dtype_code(qkv), _stream(qkv, stream))
    _lib.check(st, "gdn_chunk_prefill")
    return o


def gdn_chunk_prefill_norm(qkv, z, norm_w, dims, a=None, b=None, A_log=None, dt_bias=None, g=None,
                           beta=None, cu_seqlens=None, initial_state=None, final_state=None, ckpt_every=0,
                           state_ckpt_out=None, scale=0.0, l2norm_qk=True, norm_eps=RMSNORM_EPS, out=None,
                           workspace=None, stream=None, solve="direct", chunk=64):
    """gdn_chunk_prefill followed by RMSNormGated(o, z): returns out [T, H_v*d_v]
    (the rule's output is normalised in place in `out`)."""
    if solve not in ("direct", "neumann"):
        raise ValueError(f"solve must be 'direct' or 'neumann', not {solve!r}")
    dt = qkv.dtype
    T = int(qkv.shape[0])
    if out is None:
        out = torch.empty((T, dims.H_v * dims.d_v), dtype=dt, device=qkv.device)
    rows = 0 if state_ckpt_out is None else int(state_ckpt_out.shape[0])
    lib = _lib.load()
    if workspace is None:
        need = lib.gdn_chunk_prefill_workspace_size(_nseq(cu_seqlens), T, _dims(dims), _dtype_code(qkv))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=qkv.device)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.gdn_chunk_prefill_norm(
        _ptr(qkv, "qkv", dt), *_gate_ptrs(a, b, A_log, dt_bias, g, beta, dt),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _nseq(cu_seqlens), T,
        _ptr(initial_state, "initial_state", torch.float32),
        _ptr(final_state, "final_state", torch.float32), int(ckpt_every),
        _ptr(state_ckpt_out, "state_ckpt_out", torch.float32), rows, float(scale),
        _flags(l2norm_qk, solve, chunk), _ptr(z, "z", dt, (T, dims.H_v * dims.d_v)), _ptr(norm_w, "norm_w", dt, (dims.d_v,)), float(norm_eps),
        _ptr(out, "out", dt, (T, dims.H_v * dims.d_v)), _ptr(workspace, "workspace"), ws, _dims(dims),
        _dtype_code(qkv), _stream(qkv, stream))
    _lib.check(st, "gdn_chunk_prefill_norm")
    return out


def gdn_chunk_prefill_noalloc(qkv, dims, o, final_state, a=None, b=None, A_log=None,
                              dt_bias=None, g=None, beta=None, cu_seqlens=None,
                              initial_state=None, ckpt_every=0, state_ckpt_out=None, scale=0.0,
                              l2norm_qk=True, stream=None):
    """gdn_chunk_prefill for callers that cannot allocate device memory: its
    scratch is a fixed array inside the library, and this binding allocates
    nothing either -- the caller passes every output (o [T, H_v, d_v] and
    final_state [n_seq, H_v, d_k, d_v] f32, plus state_ckpt_out when
    checkpointing).  bf16, d = 128 only.  Calls that overlap on the GPU share
    the array and race; the first call on a device should precede any stream
    capture."""
    dt = qkv.dtype
    T = int(qkv.shape[0])
    rows = 0 if state_ckpt_out is None else int(state_ckpt_out.shape[0])
    st = _lib.load().gdn_chunk_prefill_noalloc(
        _ptr(qkv, "qkv", dt), *_gate_ptrs(a, b, A_log, dt_bias, g, beta, dt),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), _nseq(cu_seqlens), T,
        _ptr(initial_state, "initial_state", torch.float32),
        _ptr(final_state, "final_state", torch.float32), int(ckpt_every),
        _ptr(state_ckpt_out, "state_ckpt_out", torch.float32), rows, float(scale),
        _lib.GDN_QK_L2NORM if l2norm_qk else 0, _ptr(o, "o", dt, (T, dims.H_v, dims.d_v)),
        _dims(dims), _dtype_code(qkv), _stream(qkv, stream))
    _lib.check(st, "gdn_chunk_prefill_noalloc")
    return o


def gdn_recurrent_decode(qkv, state, dims, a=None, b=None, A_log=None, dt_bias=None, g=None,
                         beta=None, scale=0.0, l2norm_qk=True, o=None, stream=None):
    """One decode step for B sequences; state [B, H_v, d_k, d_v] f32 in place.
    Returns o [B, H_v, d_v]."""
    dt = qkv.dtype
    B = int(qkv.shape[0])
    if o is None:
        o = torch.empty((B, dims.H_v, dims.d_v), dtype=dt, device=qkv.device)
    st = _lib.load().gdn_recurrent_decode(
        _ptr(qkv, "qkv", dt), *_gate_ptrs(a, b, A_log, dt_bias, g, beta, dt),
        _ptr(state, "state", torch.float32, (B, dims.H_v, dims.d_k, dims.d_v)), B, float(scale),
        _lib.GDN_QK_L2NORM if l2norm_qk else 0, _ptr(o, "o", dt), _dims(dims), _dtype_code(qkv),
        _stream(qkv, stream))
    _lib.check(st, "gdn_recurrent_decode")
    return o


def gdn_rmsnorm_gated(o, z, w, dims, eps=RMSNORM_EPS, out=None, stream=None):
    """RMSNormGated per value head: o [T, H_v, d_v], z [T, H_v*d_v] -> out [T, H_v*d_v]."""
    dt = o.dtype
    T = int(o.shape[0])
    if out is None:
        out = torch.empty((T, dims.H_v * dims.d_v), dtype=dt, device=o.device)
    st = _lib.load().gdn_rmsnorm_gated(
        _ptr(o, "o", dt), _ptr(z, "z", dt), _ptr(w, "w", dt, (dims.d_v,)), float(eps), T,
        _ptr(out, "out", dt), _dims(dims), _dtype_code(o), _stream(o, stream))
    _lib.check(st, "gdn_rmsnorm_gated")
    return out


def gdn_layer_prefill_workspace_size(n_seq: int, T_tot: int, dims, dtype) -> int:
    code = _lib.GDN_BF16 if dtype == torch.bfloat16 else _lib.GDN_F32
    return int(_lib.load().gdn_layer_prefill_workspace_size(int(n_seq), int(T_tot), _dims(dims), code))


def gdn_layer_prefill_launches(n_seq: int, T_tot: int, dims, dtype, cu_seqlens=True, chunk=64) -> int:
    """Kernel launches of one gdn_layer_prefill call (cu_seqlens and chunk as
    in gdn_chunk_prefill_launches)."""
    code = _lib.GDN_BF16 if dtype == torch.bfloat16 else _lib.GDN_F32
    has_cu = 0 if cu_seqlens is None or cu_seqlens is False else 1
    return int(_lib.load().gdn_layer_prefill_launches(int(n_seq), int(T_tot), has_cu, _dims(dims), code,
                                                      _flags(False, "direct", chunk)))


def gdn_layer_prefill(mixed_qkv, z, a, b, conv_w, A_log, dt_bias, norm_w, dims, cu_seqlens=None,
                      initial_state=None, conv_state=None, ckpt_every=0, scale=0.0,
                      return_intermediates=False, stream=None, norm_eps=RMSNORM_EPS, out=None,
                      final_state=None, conv_state_out=None, workspace=None, solve="direct", chunk=64,
                      state_ckpt_out=None, conv_ckpt_out=None):
    """Whole layer core over packed sequences: conv1d+SiLU -> chunked delta rule
    -> RMSNormGated, as one gdn_layer_prefill call (bf16, d = 128: the conv
    inside the chunk kernels).  Returns a dict with out
    [T, H_v*d_v], final_state [n_seq, H_v, d_k, d_v] f32, conv_state
    [n_seq, conv_dim, 3] and, when ckpt_every > 0, state_ckpt / conv_ckpt.
    return_intermediates=True runs the three calls one by one instead and adds
    the conv output y and the rule's output o to the dict.  state_ckpt_out and
    conv_ckpt_out may pass preallocated checkpoint buffers."""
    if solve not in ("direct", "neumann"):
        raise ValueError(f"solve must be 'direct' or 'neumann', not {solve!r}")
    dev, dt = mixed_qkv.device, mixed_qkv.dtype
    T = int(mixed_qkv.shape[0])
    n_seq = _nseq(cu_seqlens)
    C = _conv_dim(dims)
    rows = 0
    if ckpt_every:
        host_cu = (cu_seqlens.to("cpu") if cu_seqlens is not None
                   else torch.tensor([0, T], dtype=torch.int32))
        rows = gdn_ckpt_count(host_cu, ckpt_every)
    if conv_state_out is None:
        conv_state_out = torch.empty((n_seq, C, 3), dtype=dt, device=dev)
    conv_ck = conv_ckpt_out
    if conv_ck is None and rows:
        conv_ck = torch.empty((rows, C, 3), dtype=dt, device=dev)
    if final_state is None:
        final_state = torch.empty((n_seq, dims.H_v, dims.d_k, dims.d_v), dtype=torch.float32, device=dev)
    S_ck = state_ckpt_out
    if S_ck is None and rows:
        S_ck = torch.empty((rows, dims.H_v, dims.d_k, dims.d_v), dtype=torch.float32, device=dev)
    if rows and (tuple(S_ck.shape) != (rows, dims.H_v, dims.d_k, dims.d_v) or
                 tuple(conv_ck.shape) != (rows, C, 3)):
        raise ValueError(f"checkpoint buffers must hold {rows} rows")
    if return_intermediates:
        y = gdn_conv1d_fwd(mixed_qkv, conv_w, dims, cu_seqlens, conv_state, conv_state_out, ckpt_every,
                           conv_ck, True, stream=stream)
        o = gdn_chunk_prefill(y, dims, a, b, A_log, dt_bias, cu_seqlens=cu_seqlens,
                              initial_state=initial_state, final_state=final_state, ckpt_every=ckpt_every,
                              state_ckpt_out=S_ck, scale=scale, stream=stream, solve=solve, chunk=chunk)
        out = gdn_rmsnorm_gated(o, z, norm_w, dims, eps=norm_eps, out=out, stream=stream)
        return {"out": out, "final_state": final_state, "conv_state": conv_state_out, "state_ckpt": S_ck,
                "conv_ckpt": conv_ck, "y": y, "o": o}
    if out is None:
        out = torch.empty((T, dims.H_v * dims.d_v), dtype=dt, device=dev)
    lib = _lib.load()
    if workspace is None:
        need = lib.gdn_layer_prefill_workspace_size(n_seq, T, _dims(dims), _dtype_code(mixed_qkv))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.gdn_layer_prefill(
        _ptr(mixed_qkv, "mixed_qkv", dt, (T, C)), _ptr(z, "z", dt), _ptr(a, "a", dt), _ptr(b, "b", dt),
        _ptr(conv_w, "conv_w", dt, (C, 4)), _ptr(A_log, "A_log", torch.float32),
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(norm_w, "norm_w", dt, (dims.d_v,)), float(norm_eps),
        _ptr(cu_seqlens, "cu_seqlens", torch.int32), n_seq, T,
        _ptr(initial_state, "initial_state", torch.float32),
        _ptr(final_state, "final_state", torch.float32, (n_seq, dims.H_v, dims.d_k, dims.d_v)),
        _ptr(conv_state, "conv_state", dt), _ptr(conv_state_out, "conv_state_out", dt, (n_seq, C, 3)),
        int(ckpt_every), _ptr(S_ck, "state_ckpt", torch.float32), _ptr(conv_ck, "conv_ckpt", dt), rows,
        float(scale),
        _flags(True, solve, chunk),
        _ptr(out, "out", dt, (T, dims.H_v * dims.d_v)), _ptr(workspace, "workspace"), ws, _dims(dims),
        _dtype_code(mixed_qkv), _stream(mixed_qkv, stream))
    _lib.check(st, "gdn_layer_prefill")
    return {"out": out, "final_state": final_state, "conv_state": conv_state_out, "state_ckpt": S_ck,
            "conv_ckpt": conv_ck}


def _hptr(t, name, dtype=None, shape=None):
    """Address of a contiguous page-locked CPU tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.device.type != "cpu" or not t.is_pinned():
        raise ValueError(f"{name}: must be a page-locked (pinned) CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr() if t.numel() else None


def gdn_layer_prefill_host(h_qkv, h_z, h_a, h_b, conv_w, A_log, dt_bias, norm_w, dims,
                           initial_state=None, conv_state_in=None, scale=0.0, l2norm=True,
                           norm_eps=1e-6, h_out=None, final_state=None, conv_state_out=None,
                           workspace=None, stream=None):
    """The layer core for one sequence whose activations (h_qkv [T, conv_dim],
    h_z [T, H_v*d_v], h_a, h_b [T, H_v]) and output h_out are pinned CPU tensors;
    parameters and states are CUDA tensors.  Copies in, kernels and copies out
    overlap piece by piece inside the library.  Returns a dict with out (the
    pinned host tensor; complete once the stream reaches this point),
    final_state [1, H_v, d_k, d_v] f32 and conv_state [1, conv_dim, 3]."""
    dt = h_qkv.dtype
    dev = conv_w.device
    T = int(h_qkv.shape[0])
    C, O = _conv_dim(dims), int(dims.H_v) * int(dims.d_v)
    code = _dtype_code(h_qkv)
    if h_out is None:
        h_out = torch.empty((T, O), dtype=dt).pin_memory()
    if final_state is None:
        final_state = torch.empty((1, dims.H_v, dims.d_k, dims.d_v), dtype=torch.float32, device=dev)
    if conv_state_out is None:
        conv_state_out = torch.empty((1, C, 3), dtype=dt, device=dev)
    lib = _lib.load()
    need = lib.gdn_layer_prefill_host_workspace_size(T, _dims(dims), code)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib.gdn_layer_prefill_host(
        _hptr(h_qkv, "h_qkv", dt, (T, C)), _hptr(h_z, "h_z", dt, (T, O)),
        _hptr(h_a, "h_a", dt, (T, dims.H_v)), _hptr(h_b, "h_b", dt, (T, dims.H_v)),
        _ptr(conv_w, "conv_w", dt, (C, 4)), _ptr(A_log, "A_log", torch.float32),
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(norm_w, "norm_w", dt), T,
        _ptr(initial_state, "initial_state", torch.float32), _ptr(final_state, "final_state", torch.float32),
        _ptr(conv_state_in, "conv_state_in", dt), _ptr(conv_state_out, "conv_state_out", dt),
        float(scale), _lib.GDN_QK_L2NORM if l2norm else 0, float(norm_eps),
        _hptr(h_out, "h_out", dt, (T, O)), _ptr(workspace, "workspace", torch.uint8),
        workspace.numel() if workspace is not None else 0, _dims(dims), code, _stream(conv_w, stream))
    _lib.check(st, "gdn_layer_prefill_host")
    return {"out": h_out, "final_state": final_state, "conv_state": conv_state_out}


def gdn_decode_step(x, z, a, b, conv_w, A_log, dt_bias, norm_w, dims, state, conv_state,
                    slots=None, scale=0.0, l2norm=True, norm_eps=1e-6, out=None, stream=None):
    """One fused decode step (conv update, gates, recurrence, RMSNormGated) in
    one kernel for B sequences; x [B, conv_dim], z [B, H_v*d_v], a, b [B, H_v];
    state [n_slots, H_v, d_k, d_v] f32 and conv_state [n_slots, conv_dim, 3]
    are updated in place at slots[b] (int32 [B], distinct) or at b.  Returns
    out [B, H_v*d_v]."""
    dt = x.dtype
    B = int(x.shape[0])
    C, O = _conv_dim(dims), int(dims.H_v) * int(dims.d_v)
    if out is None:
        out = torch.empty((B, O), dtype=dt, device=x.device)
    if state.dim() != 4 or tuple(state.shape[1:]) != (dims.H_v, dims.d_k, dims.d_v):
        raise ValueError("state: expected [n_slots, H_v, d_k, d_v]")
    if conv_state.dim() != 3 or tuple(conv_state.shape[1:]) != (C, 3):
        raise ValueError("conv_state: expected [n_slots, conv_dim, 3]")
    if slots is None and (state.shape[0] < B or conv_state.shape[0] < B):
        raise ValueError("state/conv_state: fewer slots than sequences")
    st = _lib.load().gdn_decode_step(
        _ptr(x, "x", dt, (B, C)), _ptr(conv_w, "conv_w", dt, (C, 4)), _ptr(conv_state, "conv_state", dt),
        _ptr(z, "z", dt, (B, O)), _ptr(a, "a", dt, (B, dims.H_v)), _ptr(b, "b", dt, (B, dims.H_v)),
        _ptr(A_log, "A_log", torch.float32), _ptr(dt_bias, "dt_bias", torch.float32),
        _ptr(state, "state", torch.float32), _ptr(norm_w, "norm_w", dt), float(norm_eps),
        _ptr(slots, "slots", torch.int32, (B,)) if slots is not None else None, B, float(scale),
        _lib.GDN_QK_L2NORM if l2norm else 0, _ptr(out, "out", dt, (B, O)), _dims(dims),
        _dtype_code(x), _stream(x, stream))
    _lib.check(st, "gdn_decode_step")
    return out


def gdn_decode_verify(x, z, a, b, conv_w, A_log, dt_bias, norm_w, dims, state, conv_state,
                      slots, scale=0.0, l2norm=True, norm_eps=1e-6, out=None, stream=None):
    """Speculative-decoding verification: K draft tokens of B sequences
    (x [B, K, conv_dim], z [B, K, H_v*d_v], a, b [B, K, H_v]) through the fused
    decode step in one kernel.  States are read from slot slots[b, 0] of
    state [n_slots, H_v, d_k, d_v] f32 / conv_state [n_slots, conv_dim, 3]; the
    states after draft token t are written to slot slots[b, t + 1] (slots int32
    [B, K + 1]).  Returns out [B, K, H_v*d_v]."""
    dt = x.dtype
    if x.dim() != 3:
        raise ValueError("x: expected [B, K, conv_dim]")
    B, K = int(x.shape[0]), int(x.shape[1])
    C, O = _conv_dim(dims), int(dims.H_v) * int(dims.d_v)
    if out is None:
        out = torch.empty((B, K, O), dtype=dt, device=x.device)
    if state.dim() != 4 or tuple(state.shape[1:]) != (dims.H_v, dims.d_k, dims.d_v):
        raise ValueError("state: expected [n_slots, H_v, d_k, d_v]")
    if conv_state.dim() != 3 or tuple(conv_state.shape[1:]) != (C, 3):
        raise ValueError("conv_state: expected [n_slots, conv_dim, 3]")
    st = _lib.load().gdn_decode_verify(
        _ptr(x, "x", dt, (B, K, C)), _ptr(conv_w, "conv_w", dt, (C, 4)),
        _ptr(conv_state, "conv_state", dt), _ptr(z, "z", dt, (B, K, O)),
        _ptr(a, "a", dt, (B, K, dims.H_v)), _ptr(b, "b", dt, (B, K, dims.H_v)),
        _ptr(A_log, "A_log", torch.float32), _ptr(dt_bias, "dt_bias", torch.float32),
        _ptr(state, "state", torch.float32), _ptr(norm_w, "norm_w", dt), float(norm_eps),
        _ptr(slots, "slots", torch.int32, (B, K + 1)), B, K, float(scale),
        _lib.GDN_QK_L2NORM if l2norm else 0, _ptr(out, "out", dt, (B, K, O)), _dims(dims),
        _dtype_code(x), _stream(x, stream))
    _lib.check(st, "gdn_decode_verify")
    return out


def gdn_layer_decode(x, z, a, b, conv_w, A_log, dt_bias, norm_w, dims, state, conv_state,
                     scale=0.0, stream=None):
    """One decode step of the layer core for B sequences (x [B, conv_dim]);
    state and conv_state are updated in place.  Returns out [B, H_v*d_v]."""
    y = gdn_conv1d_update(x, conv_w, conv_state, dims, True, stream=stream)
    o = gdn_recurrent_decode(y, state, dims, a, b, A_log, dt_bias, scale=scale, stream=stream)
    return gdn_rmsnorm_gated(o, z, norm_w, dims, stream=stream)


def _dptr(t, name, dev, dtype, shape=None):
    """_ptr for a tensor that must lie on CUDA device number `dev`.  One pass of
    cheap checks; what fails them goes through _ptr's for its message (a call's
    tensors are looked at in about 0.3 us each, and a decode step has a dozen)."""
    if t is None:
        return None
    try:
        if (t.get_device() == dev and (t.dtype is dtype or dtype is None) and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()  # 0, that is NULL, without elements
    except AttributeError:
        pass
    if isinstance(t, torch.Tensor) and t.get_device() != dev:
        raise ValueError(f"{name}: tensors on different devices (cuda:{dev} and {t.device})")
    return _ptr(t, name, dtype, shape)


def _elsewhere(dev, stream) -> bool:
    """Whether a call on device number `dev` needs _on_stream: it names a stream,
    or its device is not the current one (or no CUDA device)."""
    return stream is not None or dev < 0 or torch._C._cuda_getDevice() != dev


def _on_stream(dev, stream, used, body):
    """body() with device number `dev` current and, where the caller names a
    stream, that stream current too, so that outputs and workspaces allocated in
    body belong to the stream that uses them; the tensors `used` are then marked as
    in use there, so that a caller may drop them at once."""
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != dev:
        raise ValueError(f"stream: on {stream.device}, the tensors are on cuda:{dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return body()
        if not isinstance(stream, torch.cuda.Stream):
            raw = int(getattr(stream, "cuda_stream", stream))
            stream = torch.cuda.ExternalStream(raw, dev) if raw else torch.cuda.default_stream(dev)
        with torch.cuda.stream(stream):
            res = body()
        for t in used:
            if t is not None:
                t.record_stream(stream)
        return res


def _cache_dims(k_cache, v_cache, page_table, seq_lens):
    cs, ts = k_cache.shape, page_table.shape
    if len(cs) != 4 or v_cache.shape != cs:
        raise ValueError("k_cache, v_cache: expected [n_pages, H_kv, page_size, D], both alike")
    if len(ts) != 2 or seq_lens.shape != ts[:1]:
        raise ValueError("page_table: expected [B, max_pages]; seq_lens: [B]")
    return (*cs, *ts)


def gdn_kv_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens=None, stream=None):
    """Writes new tokens' keys and values k, v [T, H_kv, D] into the pages of
    k_cache, v_cache [n_pages, H_kv, page_size, D] (in place).  The L_b new tokens
    of sequence b (cu_seqlens int32 [B + 1], or T / B each) end at position
    seq_lens[b] (int32 [B], new tokens counted); page_table int32 [B, max_pages].
    Returns (k_cache, v_cache)."""
    dt, i32, dev = k.dtype, torch.int32, k.get_device()
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, (k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens),
                          lambda: gdn_kv_append(k, v, k_cache, v_cache, page_table, seq_lens, cu_seqlens))
    n_pages, H, ps, D, B, mp = _cache_dims(k_cache, v_cache, page_table, seq_lens)
    if k.dim() != 3:
        raise ValueError("k: expected [T, H_kv, D]")
    T = k.shape[0]
    st = _lib.load().gdn_kv_append(
        _dptr(k, "k", dev, dt, (T, H, D)), _dptr(v, "v", dev, dt, (T, H, D)), _dptr(k_cache, "k_cache", dev, dt),
        _dptr(v_cache, "v_cache", dev, dt), _dptr(page_table, "page_table", dev, i32),
        _dptr(seq_lens, "seq_lens", dev, i32), _dptr(cu_seqlens, "cu_seqlens", dev, i32, (B + 1,)), B, T, H, D, ps,
        n_pages, mp, _dtype_code(k), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _lib.check(st, "gdn_kv_append")
    return k_cache, v_cache


def _rows(t, name, dev, dtype, T, D, H=None):
    """Pointer and strides (tokens, heads) of a [T, H, D] tensor on CUDA device number
    `dev` whose heads' dims are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    shape = t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or (H is not None and shape[1] != H):
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [{T}, {'H' if H is None else H}, {D}]")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensors on different devices (cuda:{dev} and {t.device})")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    token, head, dim = t.stride()
    if dim != 1:
        raise ValueError(f"{name}: the dims of a head must be contiguous")
    return t.data_ptr(), token, head


def _rotation(inv_freq, positions, axes, T, D, dev):
    """Checked pointers of a rotation: (positions, n_axes, axes, inv_freq, R)."""
    shape, n_axes = inv_freq.shape, 1
    if len(shape) != 1 or not 1 <= shape[0] <= D // 2:
        raise ValueError(f"inv_freq: shape {tuple(shape)}, expected [R / 2] with 2 <= R <= {D}")
    half = shape[0]
    if positions is not None:
        shape = positions.shape
        if len(shape) not in (1, 2) or shape[-1] != T:
            raise ValueError(f"positions: shape {tuple(shape)}, expected [{T}] or [n_axes, {T}]")
        n_axes = shape[0] if len(shape) == 2 else 1
    return (_dptr(positions, "positions", dev, torch.int32), n_axes, _dptr(axes, "axes", dev, torch.int32, (half,)),
            _dptr(inv_freq, "inv_freq", dev, torch.float32), 2 * half)


def gdn_rope(x, inv_freq, positions, axes=None, norm_w=None, norm_eps=RMSNORM_EPS, mscale=1.0, interleaved=False,
             out=None, stream=None):
    """Rotary positions of x [T, H, D] (strided between tokens and heads at will, as a
    slice of a fused projection is): the pairs (j, j + R/2) of a head's first R dims,
    with interleaved (2j, 2j + 1), turn by positions[axes[j]][t] * inv_freq[j].
    inv_freq f32 [R/2]; positions int32 [T] or [n_axes, T]; axes int32 [R/2] (None:
    axis 0).  norm_w f32 [D]: the head's RMS norm with that weight comes first.
    mscale multiplies the rotated dims.  Returns out (dense unless given; x for in place)."""
    dt, dev = x.dtype, x.get_device()
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, (x, inv_freq, positions, axes, norm_w, out),
                          lambda: gdn_rope(x, inv_freq, positions, axes, norm_w, norm_eps, mscale, interleaved, out))
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x: expected [T, H, D]")
    if positions is None:
        raise ValueError("positions: needed")
    T, H, D = shape
    code = _dtype_code(x)
    p_x, x_tok, x_head = _rows(x, "x", dev, dt, T, D, H)
    p_pos, n_axes, p_axes, p_freq, R = _rotation(inv_freq, positions, axes, T, D, dev)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=x.device)
        p_out, o_tok, o_head = out.data_ptr(), H * D, D
    else:
        p_out, o_tok, o_head = _rows(out, "out", dev, dt, T, D, H)
    st = _lib.load().gdn_rope(
        p_x, x_tok, x_head, p_pos, n_axes, p_axes, p_freq, _dptr(norm_w, "norm_w", dev, torch.float32, (D,)), norm_eps,
        mscale, _lib.GDN_ROPE_INTERLEAVED if interleaved else 0, p_out, o_tok, o_head, T, H, D, R, code,
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _lib.check(st, "gdn_rope")
    return out


def gdn_rope_kv_append(q, k, v, k_cache, v_cache, page_table, seq_lens, inv_freq, positions=None, axes=None,
                       q_norm_w=None, k_norm_w=None, norm_eps=RMSNORM_EPS, mscale=1.0, interleaved=False,
                       cu_seqlens=None, q_out=None, stream=None):
    """gdn_rope of the new tokens' queries q [T, H_q, D] and keys k [T, H_kv, D], and
    gdn_kv_append of the keys and the values v, in one pass.  positions None: each
    token's place in its sequence.  q, k, v may be slices of a fused projection (see
    gdn_rope); the other arguments as gdn_rope's and gdn_kv_append's.  Returns q_out
    [T, H_q, D] (dense; may be q); the caches are written in place."""
    dt, i32, f32, dev = q.dtype, torch.int32, torch.float32, q.get_device()
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, (q, k, v, k_cache, v_cache, page_table, seq_lens, inv_freq, positions, axes,
                                        q_norm_w, k_norm_w, cu_seqlens, q_out),
                          lambda: gdn_rope_kv_append(q, k, v, k_cache, v_cache, page_table, seq_lens, inv_freq, positions,
                                                     axes, q_norm_w, k_norm_w, norm_eps, mscale, interleaved, cu_seqlens,
                                                     q_out))
    n_pages, H, ps, D, B, mp = _cache_dims(k_cache, v_cache, page_table, seq_lens)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q: expected [T, H_q, D]")
    T, H_q = shape[0], shape[1]
    code = _dtype_code(q)
    p_q, q_tok, q_head = _rows(q, "q", dev, dt, T, D)
    p_k, k_tok, k_head = _rows(k, "k", dev, dt, T, D, H)
    p_v, v_tok, v_head = _rows(v, "v", dev, dt, T, D, H)
    p_pos, n_axes, p_axes, p_freq, R = _rotation(inv_freq, positions, axes, T, D, dev)
    if q_out is None:
        q_out = torch.empty(shape, dtype=dt, device=q.device)
        p_o = q_out.data_ptr()
    else:
        p_o = _dptr(q_out, "q_out", dev, dt, (T, H_q, D))
    st = _lib.load().gdn_rope_kv_append(
        p_q, q_tok, q_head, p_k, k_tok, k_head, p_v, v_tok, v_head, p_o, _dptr(k_cache, "k_cache", dev, dt),
        _dptr(v_cache, "v_cache", dev, dt), _dptr(page_table, "page_table", dev, i32),
        _dptr(seq_lens, "seq_lens", dev, i32), _dptr(cu_seqlens, "cu_seqlens", dev, i32, (B + 1,)), p_pos, n_axes, p_axes,
        p_freq, _dptr(q_norm_w, "q_norm_w", dev, f32, (D,)), _dptr(k_norm_w, "k_norm_w", dev, f32, (D,)), norm_eps, mscale,
        _lib.GDN_ROPE_INTERLEAVED if interleaved else 0, B, T, H_q, H, D, R, ps, n_pages, mp, code,
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _lib.check(st, "gdn_rope_kv_append")
    return q_out


@lru_cache(maxsize=256)
def _attn_workspace(B, K, H_q, H_kv, D, page_size, code):
    return int(_lib.load().gdn_attn_decode_workspace_size(B, K, H_q, H_kv, D, page_size, code))


def gdn_attn_decode_workspace_size(B: int, K: int, H_q: int, H_kv: int, D: int, page_size: int, dtype) -> int:
    return _attn_workspace(int(B), int(K), int(H_q), int(H_kv), int(D), int(page_size),
                           _lib.GDN_BF16 if dtype == torch.bfloat16 else _lib.GDN_F32)


def gdn_attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale=0.0, gate=None, out=None, lse=None,
                    return_lse=False, workspace=None, stream=None):
    """Softmax attention of the K newest tokens (q [B, K, H_q, D], causal among
    themselves) over the paged cache, their own keys and values included
    (gdn_kv_append); K = 1 is a decode step, K up to 16 a verification pass.
    gate [B, K, H_q, D]: out = attention * sigmoid(gate).  Returns out
    [B, K, H_q, D], with return_lse also lse [B, K, H_q] f32."""
    dt, i32, dev = q.dtype, torch.int32, q.get_device()
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, (q, k_cache, v_cache, page_table, seq_lens, gate, out, lse, workspace),
                          lambda: gdn_attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, gate, out, lse,
                                                  return_lse, workspace))
    n_pages, H, ps, D, B, mp = _cache_dims(k_cache, v_cache, page_table, seq_lens)
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != D:
        raise ValueError(f"q: shape {tuple(shape)}, expected [{B}, K, H_q, {D}]")
    K, H_q = shape[1], shape[2]
    code = _dtype_code(q)
    # what the caller passes is checked, what is allocated here is not
    p_q = _dptr(q, "q", dev, dt)
    if out is None:
        out = torch.empty_like(q)
        p_o = out.data_ptr()
    else:
        p_o = _dptr(out, "out", dev, dt, shape)
    if lse is None and return_lse:
        lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device)
        p_e = lse.data_ptr()
    else:
        p_e = _dptr(lse, "lse", dev, torch.float32, shape[:3])
    if workspace is None:  # one batch size stands for all: the size goes by the head layout and K
        nws = _attn_workspace(1 if B else 0, K, H_q, H, D, ps, code)
        workspace = torch.empty(nws, dtype=torch.uint8, device=q.device)
        p_w = workspace.data_ptr()
    else:
        p_w, nws = _dptr(workspace, "workspace", dev, None), workspace.numel() * workspace.element_size()
    st = _lib.load().gdn_attn_decode(
        p_q, _dptr(k_cache, "k_cache", dev, dt), _dptr(v_cache, "v_cache", dev, dt),
        _dptr(page_table, "page_table", dev, i32), _dptr(seq_lens, "seq_lens", dev, i32), scale,
        _dptr(gate, "gate", dev, dt, shape), p_o, p_e, B, K, H_q, H, D, ps, n_pages, mp, p_w, nws, code,
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _lib.check(st, "gdn_attn_decode")
    return (out, lse) if return_lse else out


@lru_cache(maxsize=256)
def _shared_workspace(B, K, H_q, H_kv, D, page_size, G, code):
    return int(_lib.load().gdn_attn_decode_shared_workspace_size(B, K, H_q, H_kv, D, page_size, G, code))


def gdn_attn_decode_shared_workspace_size(B: int, K: int, H_q: int, H_kv: int, D: int, page_size: int, dtype,
                                          groups: int = 1) -> int:
    return _shared_workspace(int(B), int(K), int(H_q), int(H_kv), int(D), int(page_size), int(groups),
                             _lib.GDN_BF16 if dtype == torch.bfloat16 else _lib.GDN_F32)


def gdn_attn_decode_shared(q, k_cache, v_cache, page_table, seq_lens, prefix_lens, cu_groups=None, scale=0.0, gate=None,
                           out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """gdn_attn_decode of sequences in groups that share their first tokens, which are
    attended to once per group: sequences cu_groups[g] .. cu_groups[g + 1] - 1 (int32
    [G + 1]; None: one group of all) hold the same keys and values at their first
    prefix_lens[g] (int32 [G]) positions.  seq_lens counts the prefix too, and the
    page table holds its pages in every row; results are gdn_attn_decode's up to rounding."""
    dt, i32, dev = q.dtype, torch.int32, q.get_device()
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, (q, k_cache, v_cache, page_table, seq_lens, prefix_lens, cu_groups, gate, out, lse,
                                        workspace),
                          lambda: gdn_attn_decode_shared(q, k_cache, v_cache, page_table, seq_lens, prefix_lens, cu_groups,
                                                         scale, gate, out, lse, return_lse, workspace))
    n_pages, H, ps, D, B, mp = _cache_dims(k_cache, v_cache, page_table, seq_lens)
    shape = q.shape
    if len(shape) != 4 or shape[0] != B or shape[3] != D:
        raise ValueError(f"q: shape {tuple(shape)}, expected [{B}, K, H_q, {D}]")
    ps_shape = prefix_lens.shape
    if len(ps_shape) != 1 or ps_shape[0] < 1 or (cu_groups is None and ps_shape[0] != 1):
        raise ValueError(f"prefix_lens: shape {tuple(ps_shape)}, expected [G], [1] without cu_groups")
    K, H_q, G = shape[1], shape[2], ps_shape[0]
    code = _dtype_code(q)
    p_q = _dptr(q, "q", dev, dt)
    if out is None:
        out = torch.empty_like(q)
        p_o = out.data_ptr()
    else:
        p_o = _dptr(out, "out", dev, dt, shape)
    if lse is None and return_lse:
        lse = torch.empty(shape[:3], dtype=torch.float32, device=q.device)
        p_e = lse.data_ptr()
    else:
        p_e = _dptr(lse, "lse", dev, torch.float32, shape[:3])
    if workspace is None:
        nws = _shared_workspace(B, K, H_q, H, D, ps, G, code)
        workspace = torch.empty(nws, dtype=torch.uint8, device=q.device)
        p_w = workspace.data_ptr()
    else:
        p_w, nws = _dptr(workspace, "workspace", dev, None), workspace.numel() * workspace.element_size()
    st = _lib.load().gdn_attn_decode_shared(
        p_q, _dptr(k_cache, "k_cache", dev, dt), _dptr(v_cache, "v_cache", dev, dt),
        _dptr(page_table, "page_table", dev, i32), _dptr(seq_lens, "seq_lens", dev, i32),
        _dptr(prefix_lens, "prefix_lens", dev, i32), _dptr(cu_groups, "cu_groups", dev, i32, (G + 1,)), scale,
        _dptr(gate, "gate", dev, dt, shape), p_o, p_e, B, K, H_q, H, D, ps, n_pages, mp, G, p_w, nws, code,
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _lib.check(st, "gdn_attn_decode_shared")
    return (out, lse) if return_lse else out


def gdn_draft_accept(target_probs, draft_probs, draft_tokens, uniforms, n_draft=None, slots=None, n_accept=None,
                     tokens=None, next_slot=None, stream=None):
    """Speculative sampling from given uniforms [B, K + 1]: which of the drafted
    tokens [B, K] hold under target_probs [B, K + 1, V] and draft_probs [B, K, V]
    (None: drafts that were not sampled), and the token after them.  n_draft [B]:
    drafts per sequence (None: K).  slots [B, K + 2]: the slots of the
    gdn_decode_verify call over the K + 1 tokens.  Returns (n_accept [B], tokens
    [B, K + 1]: held drafts, next token, then -1; next_slot [B]: slots[b, n + 1],
    None without slots), all int32."""
    dt, i32, dev = target_probs.dtype, torch.int32, target_probs.get_device()
    if _elsewhere(dev, stream):
        return _on_stream(dev, stream, (target_probs, draft_probs, draft_tokens, uniforms, n_draft, slots, n_accept,
                                        tokens, next_slot),
                          lambda: gdn_draft_accept(target_probs, draft_probs, draft_tokens, uniforms, n_draft, slots,
                                                   n_accept, tokens, next_slot))
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise ValueError("target_probs: expected [B, K + 1, V]")
    B, K1, V = target_probs.shape
    K, on = K1 - 1, target_probs.device
    if n_accept is None:
        n_accept = torch.empty((B,), dtype=i32, device=on)
        p_n = n_accept.data_ptr()
    else:
        p_n = _dptr(n_accept, "n_accept", dev, i32, (B,))
    if tokens is None:
        tokens = torch.empty((B, K1), dtype=i32, device=on)
        p_t = tokens.data_ptr()
    else:
        p_t = _dptr(tokens, "tokens", dev, i32, (B, K1))
    if next_slot is None and slots is not None:
        next_slot = torch.empty((B,), dtype=i32, device=on)
        p_s = next_slot.data_ptr()
    else:
        p_s = _dptr(next_slot, "next_slot", dev, i32, (B,))
    st = _lib.load().gdn_draft_accept(
        _dptr(target_probs, "target_probs", dev, dt), _dptr(draft_probs, "draft_probs", dev, dt, (B, K, V)),
        _dptr(draft_tokens, "draft_tokens", dev, i32, (B, K)),
        _dptr(uniforms, "uniforms", dev, torch.float32, (B, K1)), _dptr(n_draft, "n_draft", dev, i32, (B,)),
        _dptr(slots, "slots", dev, i32, (B, K + 2)), B, K, V, p_n, p_t, p_s, _dtype_code(target_probs),
        torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _lib.check(st, "gdn_draft_accept")
    return n_accept, tokens, next_slot


@dataclass(frozen=True)
class HeadShard:
    """One rank's part of the layer core under head sharding: key heads
    [kh0, kh1), their value heads [h0, h1), and the matching conv channels
    (its q, k and v slices of conv_dim, in that order)."""
    dims: GDNDims
    kh0: int
    kh1: int
    h0: int
    h1: int
    channels: torch.Tensor  # int64 [conv_dim of the shard], indices into the full conv_dim


def head_shard(dims, rank: int, world: int) -> HeadShard:
    """Head sharding of the layer core over `world` ranks: rank takes a contiguous
    block of H_k / world key heads with their H_v / H_k value heads each.  Heads,
    their conv channels and their states are independent through the whole core,
    so every rank calls the same entry points with `shard.dims` on its slices
    (q, k, v channels, z and out columns, a, b, A_log and dt_bias entries, state
    heads) and no exchange is needed inside the core; the pages' tensor-parallel
    runs split the layer this way, with the one all-reduce after out_proj.
    world must divide H_k."""
    if world < 1 or rank < 0 or rank >= world or dims.H_k % world != 0:
        raise ValueError(f"head_shard: world {world} must divide H_k {dims.H_k} (rank {rank})")
    r = dims.H_v // dims.H_k
    nk = dims.H_k // world
    kh0, kh1 = rank * nk, (rank + 1) * nk
    h0, h1 = kh0 * r, kh1 * r
    dk, dv = dims.d_k, dims.d_v
    ch = torch.cat([torch.arange(kh0 * dk, kh1 * dk), torch.arange(dims.H_k * dk + kh0 * dk, dims.H_k * dk + kh1 * dk),
                    torch.arange(2 * dims.H_k * dk + h0 * dv, 2 * dims.H_k * dk + h1 * dv)])
    return HeadShard(GDNDims(nk, h1 - h0, dk, dv, dims.conv_k), kh0, kh1, h0, h1, ch)

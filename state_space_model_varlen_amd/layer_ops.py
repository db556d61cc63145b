"""The operators of the layers around the SSD scan: the short causal
convolution, the channel-wise selective scan, attention over packed prompts,
the paged key / value cache (bf16, or 8 bits with a scale a row) and attention
of single tokens over it.

As in the package itself, argument marshalling only: tensors are checked
against the problem's sizes and passed on by pointer with the current stream.
Token rows may be slices of wider rows: their distance is taken from the
tensor, everything inside a row must be contiguous.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _DT, _TORCH, _check, _lib, _stream, ssd_dt_transform
from ._layer_abi import (attn_decode_problem, attn_problem, conv_problem, kv_cache_problem,
                         scan_problem)

ACT_NONE, ACT_SILU = 0, 1
_ACT = {None: ACT_NONE, "none": ACT_NONE, "silu": ACT_SILU}
E4M3 = 3
_CACHE_DT = {torch.bfloat16: _DT[torch.bfloat16], torch.float8_e4m3fn: E4M3}
_CACHE_TORCH = {v: k for k, v in _CACHE_DT.items()}


def _refuse(t, name, dtype, shape):
    """Says what is wrong with t, if anything is."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")


# A verify step's kernels take a few microseconds, no more than careless checks of their arguments
# would: pointers are passed as plain integers, and what is in order is passed with one look at
# each property.

def _arr(t, name, dtype, shape, optional=False):
    """Pointer of a contiguous array (an empty one's may be anything)."""
    if t is None and optional:
        return None
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape):
        _refuse(t, name, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or 16


def _rows(t, name, dtype, shape, k, optional=False):
    """Pointer and row distance of t: the last k dimensions of `shape` are a token's row and
    contiguous, the rows of consecutive tokens (the dimensions before) evenly spaced. Tokens given
    as [R,T] may also come as [R T]."""
    if t is None and optional:
        return None, 0
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape):
        flat = (-1,) if len(shape) - k < 2 else (shape[0] * shape[1],) + tuple(shape[2:])
        if not isinstance(t, torch.Tensor) or tuple(t.shape) != flat:
            _refuse(t, name, dtype, shape)
        _refuse(t, name, dtype, flat)
        shape = flat
    n = math.prod(shape[-k:])
    if t.is_contiguous():
        return t.data_ptr() or 16, n
    st, nl, want = t.stride(), len(shape) - k, 1
    for d in range(len(shape) - 1, nl - 1, -1):
        if shape[d] != 1 and st[d] != want:
            raise ValueError(f"{name}: the elements of a token's row must be contiguous")
        want *= shape[d]
    if nl == 1:
        stride = st[0] if shape[0] > 1 else n
    elif shape[1] == 1:
        stride = st[0] if shape[0] > 1 else n
    else:
        stride = st[1]
        if shape[0] > 1 and st[0] != shape[1] * stride:
            raise ValueError(f"{name}: token rows must be evenly spaced")
    if stride < n:
        raise ValueError(f"{name}: token rows overlap")
    return t.data_ptr() or 16, stride


def _on(stream):
    """The stream's handle; None: the current one of the current device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return _stream(stream)


def _workspace(w):
    if w is None:
        return None, 0
    n = w.numel() if isinstance(w, torch.Tensor) else 0
    return _arr(w, "workspace", torch.uint8, (n,)), n


def _with(p, **strides):
    """A copy of the problem with these row distances."""
    q = type(p).from_buffer_copy(p)
    for k, v in strides.items():
        setattr(q, k, v)
    return q


# ---------------------------------------------------------------------------
# short causal convolution

def make_conv_problem(total_tokens: int, num_seqs: int, channels: int, width: int, num_slots: int,
                      in_dtype: torch.dtype, state_dtype: torch.dtype,
                      activation="silu") -> conv_problem:
    p = conv_problem()
    p.total_tokens, p.num_seqs, p.channels = int(total_tokens), int(num_seqs), int(channels)
    p.width, p.num_slots = int(width), int(num_slots)
    p.in_dtype, p.state_dtype = _DT[in_dtype], _DT[state_dtype]
    p.activation = _ACT[activation]
    return p


def _conv_args(p, x, weight, bias, conv_cache, state_indices, y):
    """The problem with its row distances and the outputs' shares of the channels, and the
    pointers that the prompt form and the update have in common."""
    q, ti, T, C = type(p).from_buffer_copy(p), _TORCH[p.in_dtype], p.total_tokens, p.channels
    ys = (y,) if isinstance(y, torch.Tensor) else tuple(y)
    if not 1 <= len(ys) <= 3:
        raise ValueError("y must be one tensor, or two or three that share the channels")
    out, total = [None, None, None], 0
    for i, t in enumerate(ys):
        c = t.shape[-1] if isinstance(t, torch.Tensor) and t.dim() else 0
        out[i], q.y_stride[i] = _rows(t, "y", ti, (T, c), 1)
        q.y_channels[i] = c
        total += c
    if total != C:
        raise ValueError(f"y must have {C} channels together (got {total})")
    xp, q.x_stride = _rows(x, "x", ti, (T, C), 1)
    return (q, xp, _arr(weight, "weight", torch.float32, (C, p.width)),
            _arr(bias, "bias", torch.float32, (C,), True),
            _arr(conv_cache, "conv_cache", _TORCH[p.state_dtype], (p.num_slots, p.width - 1, C)),
            _arr(state_indices, "state_indices", torch.int32, (p.num_seqs,)), out)


def causal_conv1d_varlen(p: conv_problem, x, weight, bias, cu_seqlens, conv_cache, state_indices,
                         has_initial_state, y, stream=None):
    """y = act(conv(x)) over packed sequences; y: [T,C], or a tuple of up to three tensors that
    share the channels. The cache slots [num_slots,W-1,C] are read where has_initial_state is
    set, and left with each sequence's last W-1 tokens."""
    q, xp, w, b, cache, idx, ys = _conv_args(p, x, weight, bias, conv_cache, state_indices, y)
    rc = _lib.causal_conv1d_varlen(
        ctypes.byref(q), xp, w, b,
        _arr(cu_seqlens, "cu_seqlens", torch.int32, (p.num_seqs + 1,)), cache, idx,
        _arr(has_initial_state, "has_initial_state", torch.uint8, (p.num_seqs,), True),
        *ys, _on(stream))
    _check("causal_conv1d_varlen", rc)


def causal_conv1d_update(p: conv_problem, x, weight, bias, conv_cache, state_indices, y,
                         update_cache: bool = True, stream=None):
    """Decode / MTP verify: x [T,C], request r owning rows r T/R .. (r+1) T/R - 1 and continuing
    its slot. update_cache=False leaves the cache for causal_conv1d_commit."""
    q, xp, w, b, cache, idx, ys = _conv_args(p, x, weight, bias, conv_cache, state_indices, y)
    rc = _lib.causal_conv1d_update(ctypes.byref(q), xp, w, b, cache, idx, *ys,
                                   int(bool(update_cache)), _on(stream))
    _check("causal_conv1d_update", rc)


def causal_conv1d_commit(p: conv_problem, x, conv_cache, state_indices, num_accepted, stream=None):
    """After a verify step with update_cache=False: slot r takes 1 + num_accepted[r] tokens in."""
    xp, xs = _rows(x, "x", _TORCH[p.in_dtype], (p.total_tokens, p.channels), 1)
    rc = _lib.causal_conv1d_commit(
        ctypes.byref(_with(p, x_stride=xs)), xp,
        _arr(conv_cache, "conv_cache", _TORCH[p.state_dtype],
             (p.num_slots, p.width - 1, p.channels)),
        _arr(state_indices, "state_indices", torch.int32, (p.num_seqs,)),
        _arr(num_accepted, "num_accepted", torch.int32, (p.num_seqs,)), _on(stream))
    _check("causal_conv1d_commit", rc)


# ---------------------------------------------------------------------------
# channel-wise selective scan

def make_scan_problem(total_tokens: int, num_seqs: int, channels: int, d_state: int, ngroups: int,
                      num_slots: int, in_dtype: torch.dtype,
                      state_dtype: torch.dtype) -> scan_problem:
    p = scan_problem()
    p.total_tokens, p.num_seqs, p.channels = int(total_tokens), int(num_seqs), int(channels)
    p.d_state, p.ngroups, p.num_slots = int(d_state), int(ngroups), int(num_slots)
    p.in_dtype, p.state_dtype = _DT[in_dtype], _DT[state_dtype]
    return p


def selective_scan_workspace_bytes(p: scan_problem) -> int:
    return int(_lib.selective_scan_workspace_bytes(ctypes.byref(p)))


def selective_scan_varlen_kernel(p: scan_problem) -> str:
    """How the prompt form runs p: its lanes a channel and segments ("": p is refused)."""
    return _lib.selective_scan_varlen_kernel(ctypes.byref(p)).decode()


def alloc_scan_workspace(p: scan_problem, device="cuda"):
    """Workspace of selective_scan_varlen, or None where it needs none."""
    n = selective_scan_workspace_bytes(p)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _scan_common(p, x, dt, A, B, C, D, z, y):
    ti, T, ch, N = _TORCH[p.in_dtype], p.total_tokens, p.channels, p.d_state
    q, row, bc = type(p).from_buffer_copy(p), (T, ch), (T, p.ngroups, N)
    xp, q.x_stride = _rows(x, "x", ti, row, 1)
    dp, q.dt_stride = _rows(dt, "dt", ti, row, 1)
    bp, q.b_stride = _rows(B, "B", ti, bc, 2)
    cp, q.c_stride = _rows(C, "C", ti, bc, 2)
    zp, q.z_stride = _rows(z, "z", ti, row, 1, True)
    yp, q.y_stride = _rows(y, "y", ti, row, 1)
    return (q, yp, xp, dp, _arr(A, "A", torch.float32, (ch, N)), bp, cp,
            _arr(D, "D", torch.float32, (ch,), True), zp)


def _scan_transform(p, tf):
    if tf is None:
        return None
    if not isinstance(tf, ssd_dt_transform):
        raise TypeError("dt_transform must come from make_dt_transform")
    bias = getattr(tf, "_dt_bias_tensor", None)
    if bias is not None and tuple(bias.shape) != (p.channels,):
        raise ValueError(f"dt_bias must have shape {(p.channels,)} (got {tuple(bias.shape)})")
    return ctypes.addressof(tf)


def selective_scan_varlen(p: scan_problem, x, dt, A, B, C, D, z, dt_transform, cu_seqlens,
                          state_cache, state_indices, has_initial_state, y, workspace=None,
                          stream=None):
    """Prompts: x, dt, z, y [T,C]; B, C [T,G,N]; A [C,N]; state cache [num_slots,C,N].
    workspace: alloc_scan_workspace(p)."""
    q, yp, *a = _scan_common(p, x, dt, A, B, C, D, z, y)
    rc = _lib.selective_scan_varlen(
        ctypes.byref(q), *a, _scan_transform(p, dt_transform),
        _arr(cu_seqlens, "cu_seqlens", torch.int32, (p.num_seqs + 1,)),
        _arr(state_cache, "state_cache", _TORCH[p.state_dtype],
             (p.num_slots, p.channels, p.d_state)),
        _arr(state_indices, "state_indices", torch.int32, (p.num_seqs,)),
        _arr(has_initial_state, "has_initial_state", torch.uint8, (p.num_seqs,), True),
        yp, *_workspace(workspace), _on(stream))
    _check("selective_scan_varlen", rc)


def selective_scan_update(p: scan_problem, x, dt, A, B, C, D, z, dt_transform, state_cache,
                          state_indices, y, intermediate_states=None, stream=None):
    """Decode / MTP verify: rows r T/R .. of x [T,C] etc. belong to request r, which continues
    its slot. intermediate_states [T,C,N]: the state after every token (the cache is then left
    alone); None: the last state is written back."""
    q, yp, *a = _scan_common(p, x, dt, A, B, C, D, z, y)
    ts, cn = _TORCH[p.state_dtype], (p.channels, p.d_state)
    rc = _lib.selective_scan_update(
        ctypes.byref(q), *a, _scan_transform(p, dt_transform),
        _arr(state_cache, "state_cache", ts, (p.num_slots,) + cn),
        _arr(state_indices, "state_indices", torch.int32, (p.num_seqs,)), yp,
        _arr(intermediate_states, "intermediate_states", ts, (p.total_tokens,) + cn,
             True), _on(stream))
    _check("selective_scan_update", rc)


# ---------------------------------------------------------------------------
# attention over packed prompts

def make_attn_problem(total_q: int, total_k: int, num_seqs: int, nheads: int, nkv_heads: int,
                      headdim: int, dtype: torch.dtype, causal: bool = True,
                      scale: float = 0.0, bf16_weights: bool = False) -> attn_problem:
    """scale 0: 1 / sqrt(headdim). bf16_weights: softmax weights may be rounded to bf16."""
    p = attn_problem()
    p.total_q, p.total_k, p.num_seqs = int(total_q), int(total_k), int(num_seqs)
    p.nheads, p.nkv_heads, p.headdim = int(nheads), int(nkv_heads), int(headdim)
    p.dtype, p.causal, p.scale = _DT[dtype], int(bool(causal)), float(scale or 0.0)
    p.bf16_weights = int(bool(bf16_weights))
    return p


def attention_varlen_kernel(p: attn_problem) -> str:
    """The kernel that runs p ("": p is refused)."""
    return _lib.attention_varlen_kernel(ctypes.byref(p)).decode()


def attention_varlen(p: attn_problem, q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse=None,
                     stream=None):
    """q, out [total_q,H,D]; k, v [total_k,Hkv,D]; lse [total_q,H] float32 or None. Causal
    queries are the last ones of their sequence's keys."""
    t = _TORCH[p.dtype]
    qrow, krow = (p.total_q, p.nheads, p.headdim), (p.total_k, p.nkv_heads, p.headdim)
    qp, qs = _rows(q, "q", t, qrow, 2)
    kp, ks = _rows(k, "k", t, krow, 2)
    vp, vs = _rows(v, "v", t, krow, 2)
    op, os_ = _rows(out, "out", t, qrow, 2)
    rc = _lib.attention_varlen(
        ctypes.byref(_with(p, q_stride=qs, k_stride=ks, v_stride=vs, o_stride=os_)), qp, kp, vp,
        _arr(cu_seqlens_q, "cu_seqlens_q", torch.int32, (p.num_seqs + 1,)),
        _arr(cu_seqlens_k, "cu_seqlens_k", torch.int32, (p.num_seqs + 1,)), op,
        _arr(lse, "lse", torch.float32, (p.total_q, p.nheads), True), _on(stream))
    _check("attention_varlen", rc)


# ---------------------------------------------------------------------------
# paged key / value cache

def make_kv_cache_problem(num_pages: int, page_size: int, nkv_heads: int, headdim: int,
                          in_dtype: torch.dtype, cache_dtype: torch.dtype) -> kv_cache_problem:
    """cache_dtype: torch.bfloat16 or torch.float8_e4m3fn."""
    p = kv_cache_problem()
    p.num_pages, p.page_size = int(num_pages), int(page_size)
    p.nkv_heads, p.headdim = int(nkv_heads), int(headdim)
    p.in_dtype, p.cache_dtype = _DT[in_dtype], _CACHE_DT[cache_dtype]
    return p


def alloc_kv_cache(p: kv_cache_problem, device="cuda") -> dict:
    """k_cache, v_cache and their scales (None for a bf16 cache), zeroed."""
    shape, got = (p.num_pages, p.nkv_heads, p.page_size), {}
    for n in ("k", "v"):
        got[n + "_cache"] = torch.zeros(shape + (p.headdim,), dtype=torch.uint8 if p.cache_dtype ==
                                        E4M3 else torch.bfloat16, device=device).view(
                                            _CACHE_TORCH[p.cache_dtype])
        got[n + "_scale"] = (torch.ones(shape, dtype=torch.uint8, device=device)
                             if p.cache_dtype == E4M3 else None)
    return got


def _kv_ptrs(p, k_cache, v_cache, k_scale, v_scale):
    shape, t = (p.num_pages, p.nkv_heads, p.page_size), _CACHE_TORCH[p.cache_dtype]
    none = p.cache_dtype != E4M3
    if none and (k_scale is not None or v_scale is not None):
        raise ValueError("a bfloat16 cache has no scales")
    return (_arr(k_cache, "k_cache", t, shape + (p.headdim,)),
            _arr(v_cache, "v_cache", t, shape + (p.headdim,)),
            _arr(k_scale, "k_scale", torch.uint8, shape, none),
            _arr(v_scale, "v_scale", torch.uint8, shape, none))


def kv_cache_store(p: kv_cache_problem, k, v, slot_mapping, k_cache, v_cache, k_scale=None,
                   v_scale=None, stream=None):
    """Writes rows k, v [T,Hkv,D] to positions slot_mapping [T] int64 (page * page_size + place;
    negative: skipped), in the cache's type."""
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch tensor")
    n, t = (k.shape[0] if k.dim() else 0), _TORCH[p.in_dtype]
    row = (n, p.nkv_heads, p.headdim)
    kp, ks = _rows(k, "k", t, row, 2)
    vp, vs = _rows(v, "v", t, row, 2)
    rc = _lib.kv_cache_store(
        ctypes.byref(_with(p, k_stride=ks, v_stride=vs)), n, kp, vp,
        _arr(slot_mapping, "slot_mapping", torch.int64, (n,)),
        *_kv_ptrs(p, k_cache, v_cache, k_scale, v_scale), _on(stream))
    _check("kv_cache_store", rc)


def kv_cache_load(p: kv_cache_problem, cu_seqlens, block_table, k_cache, v_cache, k_scale,
                  v_scale, k, v, stream=None):
    """Reads sequences of cu_seqlens [S+1] back into packed rows k, v [T,Hkv,D] through
    block_table [S,max_pages] int32."""
    if not isinstance(k, torch.Tensor) or not isinstance(block_table, torch.Tensor):
        raise TypeError("k and block_table must be torch tensors")
    if block_table.dim() != 2:
        raise ValueError("block_table must have shape (num_seqs, max_pages)")
    n, t = (k.shape[0] if k.dim() else 0), _TORCH[p.in_dtype]
    row, (S, mp) = (n, p.nkv_heads, p.headdim), block_table.shape
    kp, ks = _rows(k, "k", t, row, 2)
    vp, vs = _rows(v, "v", t, row, 2)
    rc = _lib.kv_cache_load(
        ctypes.byref(_with(p, k_stride=ks, v_stride=vs)), n, S, mp,
        _arr(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,)),
        _arr(block_table, "block_table", torch.int32, (S, mp)),
        *_kv_ptrs(p, k_cache, v_cache, k_scale, v_scale), kp, vp, _on(stream))
    _check("kv_cache_load", rc)


# ---------------------------------------------------------------------------
# attention of single tokens over the cache

def make_attn_decode_problem(kv: kv_cache_problem, num_reqs: int, tokens_per_req: int, nheads: int,
                             max_pages: int, scale: float = 0.0) -> attn_decode_problem:
    p = attn_decode_problem()
    p.kv = kv
    p.num_reqs, p.tokens_per_req, p.nheads = int(num_reqs), int(tokens_per_req), int(nheads)
    p.max_pages, p.scale = int(max_pages), float(scale or 0.0)
    return p


def attn_decode_workspace_bytes(p: attn_decode_problem) -> int:
    return int(_lib.attn_decode_workspace_bytes(ctypes.byref(p)))


def alloc_attn_decode_workspace(p: attn_decode_problem, device="cuda"):
    """Workspace of attention_decode, or None where it needs none."""
    n = attn_decode_workspace_bytes(p)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def attention_decode(p: attn_decode_problem, q, k_cache, v_cache, k_scale, v_scale, block_table,
                     context_lens, out, lse=None, workspace=None, stream=None):
    """q, out [R,T,H,D]: the last T of each request's context_lens [R] cached tokens (their own
    keys included); block_table [R,max_pages]; lse [R,T,H] float32 or None; workspace:
    alloc_attn_decode_workspace(p)."""
    R, T, t = p.num_reqs, p.tokens_per_req, _TORCH[p.kv.in_dtype]
    row = (R, T, p.nheads, p.kv.headdim)
    qp, qs = _rows(q, "q", t, row, 2)
    op, os_ = _rows(out, "out", t, row, 2)
    rc = _lib.attention_decode(
        ctypes.byref(_with(p, q_stride=qs, o_stride=os_)), qp,
        *_kv_ptrs(p.kv, k_cache, v_cache, k_scale, v_scale),
        _arr(block_table, "block_table", torch.int32, (R, p.max_pages)),
        _arr(context_lens, "context_lens", torch.int32, (R,)), op,
        _arr(lse, "lse", torch.float32, (R, T, p.nheads), True),
        *_workspace(workspace), _on(stream))
    _check("attention_decode", rc)

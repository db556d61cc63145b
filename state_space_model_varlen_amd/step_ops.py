"""The operators between and behind the layers of a serving step: the
root-mean-square norm (with the residual's addition or a gate, into 16, 32 or 8
bits), products with 4-bit weights, token probabilities and the verification of
drafted tokens, whose counts the state commits take.

As in the package itself, argument marshalling only. Token rows may be slices
of wider rows. All tensors of a call lie on one GPU; the call runs there, on its
current stream unless one is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import _DT, _TORCH, _check, _lib
from ._step_abi import linear_problem, norm_problem, probs_problem, verify_problem
from .layer_ops import E4M3, _arr, _on, _rows, _with

_ROW_DT = {**_DT, torch.float8_e4m3fn: E4M3}
_ROW_TORCH = {**_TORCH, E4M3: torch.float8_e4m3fn}


_T, _current, _stream_of = torch.Tensor, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _gpu(t):
    """The GPU that the call runs on: its first tensor's (-2, which no tensor has: none)."""
    dev = t.get_device() if isinstance(t, _T) else -1
    return dev if dev >= 0 else -2


def _same_gpu(t, name, dev):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, like the call's first tensor (got {t.device})")


# (What is in order is passed with one look at each property, as in layer_ops: a call of a few
# microseconds takes as long to check as to run. What is not goes there to be told why.)

def _row(t, name, dtype, shape, dev, optional=False):
    """Pointer and row distance of t, whose rows are its last dimension."""
    if type(t) is _T and t.dtype is dtype and t.shape == shape and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr() or 16, shape[-1]
    if t is None and optional:
        return None, 0
    got = _rows(t, name, dtype, shape, 1)
    _same_gpu(t, name, dev)
    return got


def _array(t, name, dtype, shape, dev, optional=False):
    """Pointer of a contiguous array."""
    if type(t) is _T and t.dtype is dtype and t.shape == shape and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr() or 16
    if t is None and optional:
        return None
    got = _arr(t, name, dtype, shape)
    _same_gpu(t, name, dev)
    return got


def _space(w, dev):
    """Pointer and size of a workspace."""
    if w is None:
        return None, 0
    n = w.numel() if isinstance(w, _T) else 0
    return _array(w, "workspace", torch.uint8, (n,), dev), n


def _call(name, fn, stream, dev, *args):
    """Runs the entry point on the GPU that its tensors lie on."""
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"{name}: the stream is not of cuda:{dev}")
    if dev == _current():
        rc = fn(*args, _stream_of(dev) if stream is None else _on(stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream_of(dev) if stream is None else _on(stream))
    if rc:
        _check(name, rc)


def _alloc(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


# ---------------------------------------------------------------------------
# root-mean-square norm

def make_norm_problem(rows: int, hidden: int, in_dtype: torch.dtype, out_dtype: torch.dtype,
                      groups: int = 1, residual_dtype: torch.dtype = None,
                      eps: float = 1e-5) -> norm_problem:
    """out_dtype: float32, bfloat16, or float8_e4m3fn (8-bit rows for linear_w4).
    residual_dtype None: that of in_dtype."""
    p = norm_problem()
    p.rows, p.hidden, p.ngroups, p.eps = int(rows), int(hidden), int(groups), float(eps)
    p.in_dtype, p.out_dtype = _DT[in_dtype], _ROW_DT[out_dtype]
    p.residual_dtype = _DT[in_dtype if residual_dtype is None else residual_dtype]
    return p


def rms_norm(p: norm_problem, x, weight, out, residual=None, residual_out=None, gate=None,
             out_scale=None, stream=None):
    """out = v / sqrt(mean(v^2) + eps) * weight, v = x, x + residual or x * silu(gate): [rows,
    hidden] each. residual_out keeps the sum (it may be residual itself). weight [hidden] float32
    or None. out_scale [rows,hidden/32] uint8 with 8-bit rows."""
    q, row, dev = type(p).from_buffer_copy(p), (p.rows, p.hidden), _gpu(x)
    ti, tr, e4m3 = _TORCH[p.in_dtype], _TORCH[p.residual_dtype], p.out_dtype == E4M3
    if not e4m3 and out_scale is not None:
        raise ValueError("out_scale belongs to 8-bit rows")
    if residual_out is not None and residual is None:
        raise ValueError("residual_out needs residual")
    if gate is not None and residual is not None:
        raise ValueError("gate and residual exclude each other")
    xp, q.x_stride = _row(x, "x", ti, row, dev)
    gp, q.gate_stride = _row(gate, "gate", ti, row, dev, True)
    rp, q.residual_stride = _row(residual, "residual", tr, row, dev, True)
    sp, q.residual_out_stride = _row(residual_out, "residual_out", tr, row, dev, True)
    op, q.out_stride = _row(out, "out", _ROW_TORCH[p.out_dtype], row, dev)
    _call("rms_norm", _lib.rms_norm, stream, dev, ctypes.byref(q), xp, gp, rp,
          _array(weight, "weight", torch.float32, (p.hidden,), dev, True), op,
          _array(out_scale, "out_scale", torch.uint8, (p.rows, p.hidden // 32), dev, not e4m3), sp)


# ---------------------------------------------------------------------------
# products with 4-bit weights

def make_linear_problem(tokens: int, in_features: int, out_features: int, x_dtype: torch.dtype,
                        out_dtype: torch.dtype, cut_products: bool = False) -> linear_problem:
    """x_dtype: bfloat16, or float8_e4m3fn with a scale byte for 32 elements. cut_products: those of
    8-bit rows into bfloat16 may be cut at 2^-13 of the largest of their 32."""
    p = linear_problem()
    p.tokens, p.in_features, p.out_features = int(tokens), int(in_features), int(out_features)
    p.x_dtype, p.out_dtype = _ROW_DT[x_dtype], _DT[out_dtype]
    p.cut_products = int(bool(cut_products))
    return p


def linear_w4_workspace_bytes(p: linear_problem) -> int:
    return int(_lib.linear_w4_workspace_bytes(ctypes.byref(p)))


def linear_w4_kernel(p: linear_problem) -> str:
    """The kernel that runs p ("": p is refused)."""
    return _lib.linear_w4_kernel(ctypes.byref(p)).decode()


def alloc_linear_workspace(p: linear_problem, device="cuda"):
    """Workspace of linear_w4, or None where it needs none."""
    return _alloc(linear_w4_workspace_bytes(p), device)


def alloc_linear_weights(p: linear_problem, device="cuda") -> dict:
    """weight and weight_scale as linear_w4_encode writes and linear_w4 reads them."""
    n, k = p.out_features, p.in_features
    return dict(weight=torch.zeros(n, k // 2, dtype=torch.uint8, device=device),
                weight_scale=torch.ones(n, k // 32, dtype=torch.uint8, device=device))


def _weights(p, weight, weight_scale, dev):
    n, k = p.out_features, p.in_features
    return (_array(weight, "weight", torch.uint8, (n, k // 2), dev),
            _array(weight_scale, "weight_scale", torch.uint8, (n, k // 32), dev))


def linear_w4(p: linear_problem, x, weight, weight_scale, out, x_scale=None, bias=None,
              workspace=None, stream=None):
    """out [T,N] = x [T,K] times the 4-bit weights [N,K] (weight [N,K/2], weight_scale [N,K/32]
    uint8), plus bias [N] float32. x_scale [T,K/32] uint8 with 8-bit rows. workspace:
    alloc_linear_workspace(p)."""
    T, K, N, e4m3 = p.tokens, p.in_features, p.out_features, p.x_dtype == E4M3
    if not e4m3 and x_scale is not None:
        raise ValueError("x_scale belongs to 8-bit rows")
    dev = _gpu(x)
    xp, xs = _row(x, "x", _ROW_TORCH[p.x_dtype], (T, K), dev)
    op, os_ = _row(out, "out", _TORCH[p.out_dtype], (T, N), dev)
    _call("linear_w4", _lib.linear_w4, stream, dev,
          ctypes.byref(_with(p, x_stride=xs, out_stride=os_)), xp,
          _array(x_scale, "x_scale", torch.uint8, (T, K // 32), dev, not e4m3),
          *_weights(p, weight, weight_scale, dev),
          _array(bias, "bias", torch.float32, (N,), dev, True), op, *_space(workspace, dev))


def linear_w4_encode(p: linear_problem, w, weight, weight_scale, stream=None):
    """w [N,K] float32 or bfloat16 as 4-bit codes and scales."""
    if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("w must be a float32 or bfloat16 tensor")
    dev = _gpu(w)
    _call("linear_w4_encode", _lib.linear_w4_encode, stream, dev, ctypes.byref(p), _DT[w.dtype],
          _array(w, "w", w.dtype, (p.out_features, p.in_features), dev),
          *_weights(p, weight, weight_scale, dev))


# ---------------------------------------------------------------------------
# probabilities of tokens

def make_probs_problem(num_reqs: int, tokens_per_req: int, vocab: int,
                       in_dtype: torch.dtype) -> probs_problem:
    p = probs_problem()
    p.num_reqs, p.tokens_per_req, p.vocab = int(num_reqs), int(tokens_per_req), int(vocab)
    p.in_dtype = _DT[in_dtype]
    return p


def token_probs_workspace_bytes(p: probs_problem) -> int:
    return int(_lib.token_probs_workspace_bytes(ctypes.byref(p)))


def alloc_probs_workspace(p: probs_problem, device="cuda"):
    """Workspace of token_probs, or None where it needs none."""
    return _alloc(token_probs_workspace_bytes(p), device)


def token_probs(p: probs_problem, logits, temperature, probs, workspace=None, stream=None):
    """probs [R,T,V] float32 = softmax(logits [R,T,V] / temperature [R]); a temperature of 0: 1 on
    the first of the largest. temperature None: 1. workspace: alloc_probs_workspace(p)."""
    row, dev = (p.num_reqs, p.tokens_per_req, p.vocab), _gpu(logits)
    lp, ls = _row(logits, "logits", _TORCH[p.in_dtype], row, dev)
    pp, ps = _row(probs, "probs", torch.float32, row, dev)
    _call("token_probs", _lib.token_probs, stream, dev,
          ctypes.byref(_with(p, logits_stride=ls, probs_stride=ps)), lp,
          _array(temperature, "temperature", torch.float32, (p.num_reqs,), dev, True), pp,
          *_space(workspace, dev))


# ---------------------------------------------------------------------------
# verification of drafted tokens

def make_verify_problem(num_reqs: int, tokens_per_req: int, vocab: int) -> verify_problem:
    """tokens_per_req: 1 + the most drafts of a request."""
    p = verify_problem()
    p.num_reqs, p.tokens_per_req, p.vocab = int(num_reqs), int(tokens_per_req), int(vocab)
    return p


def verify_drafts_workspace_bytes(p: verify_problem) -> int:
    return int(_lib.verify_drafts_workspace_bytes(ctypes.byref(p)))


def alloc_verify_workspace(p: verify_problem, device="cuda"):
    """Workspace of verify_drafts, or None where it needs none."""
    return _alloc(verify_drafts_workspace_bytes(p), device)


def verify_drafts(p: verify_problem, target_probs, draft_probs, draft_tokens, num_drafts, uniform,
                  num_accepted, tokens, workspace=None, stream=None):
    """num_accepted [R] and tokens [R,T] int32 (the accepted drafts, the next token, then -1) from
    target_probs [R,T,V], draft_probs [R,T-1,V] (None: certain drafts), draft_tokens [R,T-1] int32
    (None with T = 1), num_drafts [R] int32 (None: T-1 each) and uniform [R,T] in [0, 1).
    workspace: alloc_verify_workspace(p)."""
    R, T, V, i32, f32 = p.num_reqs, p.tokens_per_req, p.vocab, torch.int32, torch.float32
    dev = _gpu(target_probs)
    tp, ts = _row(target_probs, "target_probs", f32, (R, T, V), dev)
    dp, ds, tok = None, 0, None
    if T > 1:
        dp, ds = _row(draft_probs, "draft_probs", f32, (R, T - 1, V), dev, True)
        tok = _array(draft_tokens, "draft_tokens", i32, (R, T - 1), dev)
    _call("verify_drafts", _lib.verify_drafts, stream, dev,
          ctypes.byref(_with(p, target_stride=ts, draft_stride=ds)), tp, dp, tok,
          _array(num_drafts, "num_drafts", i32, (R,), dev, True),
          _array(uniform, "uniform", f32, (R, T), dev),
          _array(num_accepted, "num_accepted", i32, (R,), dev),
          _array(tokens, "tokens", i32, (R, T), dev), *_space(workspace, dev))

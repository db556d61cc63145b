"""ctypes structs and signatures of the operators between and behind the layers
(``include/ssd_mi355x.h``, "Operators between and behind the layers of a serving step")."""
from __future__ import annotations

import ctypes

_i32, _i64, _f, _vp, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                            ctypes.c_size_t)


class norm_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "rows", "hidden", "ngroups", "in_dtype", "residual_dtype", "out_dtype")] + [
            ("eps", _f), ("reserved", _i32)] + [(n, _i64) for n in (
                "x_stride", "gate_stride", "residual_stride", "residual_out_stride",
                "out_stride")]


class linear_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "tokens", "in_features", "out_features", "x_dtype", "out_dtype", "cut_products")] + [
            ("x_stride", _i64), ("out_stride", _i64)]


class probs_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("num_reqs", "tokens_per_req", "vocab", "in_dtype")] + [
        ("logits_stride", _i64), ("probs_stride", _i64)]


class verify_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("num_reqs", "tokens_per_req", "vocab", "reserved")] + [
        ("target_stride", _i64), ("draft_stride", _i64)]


_np, _lp, _pp, _vpp = (ctypes.POINTER(t) for t in (
    norm_problem, linear_problem, probs_problem, verify_problem))

STEP_SIGS = {
    "rms_norm": ([_np] + [_vp] * 8, ctypes.c_int),
    "linear_w4_workspace_bytes": ([_lp], _sz),
    "linear_w4_kernel": ([_lp], ctypes.c_char_p),
    "linear_w4": ([_lp] + [_vp] * 7 + [_sz, _vp], ctypes.c_int),
    "linear_w4_encode": ([_lp, _i32] + [_vp] * 4, ctypes.c_int),
    "token_probs_workspace_bytes": ([_pp], _sz),
    "token_probs": ([_pp] + [_vp] * 4 + [_sz, _vp], ctypes.c_int),
    "verify_drafts_workspace_bytes": ([_vpp], _sz),
    "verify_drafts": ([_vpp] + [_vp] * 8 + [_sz, _vp], ctypes.c_int),
}

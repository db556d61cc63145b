"""ctypes structs and signatures of the operators around the scan
(``include/ssd_mi355x.h``, "Operators of the layers around the SSD scan")."""
from __future__ import annotations

import ctypes

_i32, _i64, _f, _vp, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p,
                            ctypes.c_size_t)


class conv_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "total_tokens", "num_seqs", "channels", "width", "num_slots", "in_dtype", "state_dtype",
        "activation")] + [("x_stride", _i64), ("y_channels", _i32 * 3), ("reserved", _i32),
                          ("y_stride", _i64 * 3)]


class scan_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "total_tokens", "num_seqs", "channels", "d_state", "ngroups", "num_slots", "in_dtype",
        "state_dtype")] + [(n, _i64) for n in (
            "x_stride", "dt_stride", "z_stride", "b_stride", "c_stride", "y_stride")]


class attn_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "total_q", "total_k", "num_seqs", "nheads", "nkv_heads", "headdim", "dtype",
        "causal")] + [("scale", _f), ("bf16_weights", _i32)] + [(n, _i64) for n in (
            "q_stride", "k_stride", "v_stride", "o_stride")]


class kv_cache_problem(ctypes.Structure):
    _fields_ = [(n, _i32) for n in (
        "num_pages", "page_size", "nkv_heads", "headdim", "in_dtype",
        "cache_dtype")] + [("k_stride", _i64), ("v_stride", _i64)]


class attn_decode_problem(ctypes.Structure):
    _fields_ = [("kv", kv_cache_problem)] + [(n, _i32) for n in (
        "num_reqs", "tokens_per_req", "nheads", "max_pages")] + [
            ("scale", _f), ("reserved", _i32), ("q_stride", _i64), ("o_stride", _i64)]


_cp, _sp, _ap, _kp, _dp = (ctypes.POINTER(t) for t in (
    conv_problem, scan_problem, attn_problem, kv_cache_problem, attn_decode_problem))

LAYER_SIGS = {
    "causal_conv1d_varlen": ([_cp] + [_vp] * 11, ctypes.c_int),
    "causal_conv1d_update": ([_cp] + [_vp] * 8 + [_i32, _vp], ctypes.c_int),
    "causal_conv1d_commit": ([_cp] + [_vp] * 5, ctypes.c_int),
    "selective_scan_workspace_bytes": ([_sp], _sz),
    "selective_scan_varlen_kernel": ([_sp], ctypes.c_char_p),
    "selective_scan_varlen": ([_sp] + [_vp] * 14 + [_sz, _vp], ctypes.c_int),
    "selective_scan_update": ([_sp] + [_vp] * 13, ctypes.c_int),
    "attention_varlen_kernel": ([_ap], ctypes.c_char_p),
    "attention_varlen": ([_ap] + [_vp] * 8, ctypes.c_int),
    "kv_cache_store": ([_kp, _i32] + [_vp] * 8, ctypes.c_int),
    "kv_cache_load": ([_kp, _i32, _i32, _i32] + [_vp] * 9, ctypes.c_int),
    "attn_decode_workspace_bytes": ([_dp], _sz),
    "attention_decode": ([_dp] + [_vp] * 10 + [_sz, _vp], ctypes.c_int),
}

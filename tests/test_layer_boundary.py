"""Refusals of the operators around the scan: every bad argument is turned down on the host,
before anything reaches the GPU (no GPU needed)."""
import ctypes

import pytest
import torch

ssd = pytest.importorskip("state_space_model_varlen_amd")
LIB = ssd._lib
OK = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)          # aligned to 8, not to 16
OFF = ctypes.c_void_p(257)
BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16
NULL, SHAPE, DTYPE, UNSUP, WORK, ALIGN = 1, 2, 3, 4, 5, 7


def conv(**kw):
    p = ssd.make_conv_problem(64, 2, 32, 4, 4, BF, BF)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call_conv(p, *over):
    a = [OK] * 8 + [None, None, None]        # x w bias cu cache idx has y0 y1 y2 stream
    for i, v in over:
        a[i] = v
    return LIB.causal_conv1d_varlen(ctypes.byref(p), *a)


@pytest.mark.parametrize("kw,status", [
    (dict(channels=0), SHAPE), (dict(total_tokens=-1), SHAPE), (dict(num_slots=0), SHAPE),
    (dict(num_seqs=0), SHAPE), (dict(width=1), UNSUP), (dict(width=5), UNSUP),
    (dict(activation=2), UNSUP), (dict(in_dtype=2), DTYPE), (dict(state_dtype=2), DTYPE),
    (dict(in_dtype=3), DTYPE), (dict(x_stride=31), SHAPE), (dict(x_stride=-64), SHAPE),
    (dict(y_channels=(ctypes.c_int32 * 3)(16, 8, 0)), SHAPE),
    (dict(y_channels=(ctypes.c_int32 * 3)(40, -8, 0)), SHAPE),
    (dict(y_stride=(ctypes.c_int64 * 3)(31, 0, 0)), SHAPE),
    (dict(y_channels=(ctypes.c_int32 * 3)(16, 16, 0)), NULL),       # y1 missing
    (dict(total_tokens=2 ** 31 - 1, channels=2 ** 20), UNSUP),
])
def test_conv_refusals(kw, status):
    assert call_conv(conv(**kw)) == status


def test_conv_pointers():
    p = conv()
    for i in (0, 1, 3, 4, 5, 7):
        assert call_conv(p, (i, None)) == NULL, i
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert call_conv(p, (i, OFF)) == ALIGN, i
    assert LIB.causal_conv1d_varlen(None, *([OK] * 11)) == NULL
    # the update: whole requests
    q = conv(total_tokens=65)
    assert LIB.causal_conv1d_update(ctypes.byref(q), *([OK] * 6), None, None, 1, None) == SHAPE
    assert LIB.causal_conv1d_commit(ctypes.byref(q), *([OK] * 4), None) == SHAPE
    assert LIB.causal_conv1d_commit(ctypes.byref(conv()), OK, OK, OK, None, None) == NULL


def scan(**kw):
    p = ssd.make_scan_problem(64, 2, 32, 16, 2, 4, BF, F32)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call_scan(p, *over, ws=1 << 40, tf=None):
    a = [OK] * 7 + [tf, OK, OK, OK, OK, OK, OK]   # x dt A B C D z tf cu cache idx has y workspace
    for i, v in over:
        a[i] = v
    return LIB.selective_scan_varlen(ctypes.byref(p), *a, ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("kw,status", [
    (dict(channels=0), SHAPE), (dict(channels=33), SHAPE), (dict(d_state=0), SHAPE),
    (dict(ngroups=0), SHAPE), (dict(num_slots=0), SHAPE), (dict(num_seqs=0), SHAPE),
    (dict(d_state=8), UNSUP), (dict(d_state=128), UNSUP), (dict(in_dtype=2), DTYPE),
    (dict(state_dtype=3), DTYPE), (dict(x_stride=31), SHAPE), (dict(dt_stride=1), SHAPE),
    (dict(z_stride=31), SHAPE), (dict(b_stride=31), SHAPE), (dict(c_stride=31), SHAPE),
    (dict(y_stride=31), SHAPE), (dict(num_seqs=2 ** 30, channels=2 ** 20), UNSUP),
])
def test_scan_refusals(kw, status):
    assert call_scan(scan(**kw)) == status
    assert ssd.selective_scan_workspace_bytes(scan(**kw)) == 0


def test_scan_pointers_and_workspace():
    p = scan()
    for i in (0, 1, 2, 3, 4, 8, 9, 10, 12):
        assert call_scan(p, (i, None)) == NULL, i
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 12):
        assert call_scan(p, (i, OFF)) == ALIGN, i
    assert call_scan(p, (2, ODD)) == ALIGN and call_scan(p, (9, ODD)) == ALIGN
    bad = ssd.make_dt_transform(None, 1.0, 0.5)
    assert call_scan(p, tf=ctypes.addressof(bad)) == SHAPE
    nan = ssd.make_dt_transform(None, float("nan"), 1.0)
    assert call_scan(p, tf=ctypes.addressof(nan)) == SHAPE
    # a problem that needs a workspace, with too small a one
    for n in (1, 2):
        big = scan(total_tokens=8192 * n, num_seqs=1)
        need = ssd.selective_scan_workspace_bytes(big)
        if need:
            assert call_scan(big, ws=need - 1) == WORK
            assert call_scan(big, (13, None), ws=need) == NULL
            assert call_scan(big, (13, ODD), ws=need) == ALIGN
    q = scan(total_tokens=65)
    assert LIB.selective_scan_update(ctypes.byref(q), *([OK] * 7), None, *([OK] * 4), None) == SHAPE
    assert LIB.selective_scan_update(ctypes.byref(p), *([OK] * 7), None, OK, OK, OK, ODD,
                                     None) == ALIGN


def attn(**kw):
    p = ssd.make_attn_problem(64, 64, 2, 8, 2, 64, BF)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call_attn(p, *over):
    a = [OK] * 6 + [None, None]              # q k v cuq cuk out lse stream
    for i, v in over:
        a[i] = v
    return LIB.attention_varlen(ctypes.byref(p), *a)


@pytest.mark.parametrize("kw,status", [
    (dict(total_q=-1), SHAPE), (dict(nheads=0), SHAPE), (dict(nheads=7), SHAPE),
    (dict(nkv_heads=0), SHAPE), (dict(num_seqs=0), SHAPE), (dict(headdim=0), SHAPE),
    (dict(headdim=96), UNSUP), (dict(dtype=2), DTYPE), (dict(dtype=9), DTYPE),
    (dict(q_stride=8), SHAPE), (dict(k_stride=8), SHAPE), (dict(v_stride=8), SHAPE),
    (dict(o_stride=8), SHAPE), (dict(q_stride=516), ALIGN), (dict(k_stride=130), ALIGN),
    (dict(k_stride=1 << 22), UNSUP), (dict(scale=-1.0), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(num_seqs=2 ** 30), UNSUP),
])
def test_attention_refusals(kw, status):
    assert call_attn(attn(**kw)) == status


def test_attention_pointers():
    for i in range(6):
        assert call_attn(attn(), (i, None)) == NULL, i
        assert call_attn(attn(), (i, OFF)) == ALIGN, i
    assert call_attn(attn(), (6, OFF)) == ALIGN
    assert call_attn(attn(), (0, ODD)) == ALIGN and call_attn(attn(), (5, ODD)) == ALIGN


def kv(dtype=torch.float8_e4m3fn, **kw):
    p = ssd.make_kv_cache_problem(8, 64, 2, 64, BF, dtype)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=48), UNSUP),
    (dict(page_size=8), UNSUP), (dict(page_size=512), UNSUP), (dict(headdim=80), UNSUP),
    (dict(nkv_heads=0), SHAPE), (dict(cache_dtype=0), DTYPE), (dict(cache_dtype=2), DTYPE),
    (dict(in_dtype=2), DTYPE), (dict(k_stride=64), SHAPE), (dict(v_stride=130), ALIGN),
])
def test_kv_refusals(kw, status):
    p = kv(**kw)
    assert LIB.kv_cache_store(ctypes.byref(p), 4, *([OK] * 7), None) == status
    assert LIB.kv_cache_load(ctypes.byref(p), 4, 1, 1, *([OK] * 8), None) == status


def test_kv_pointers():
    p = kv()
    for i in range(7):
        a = [OK] * 7
        a[i] = None
        assert LIB.kv_cache_store(ctypes.byref(p), 4, *a, None) == NULL, i
    for i in range(8):
        a = [OK] * 8
        a[i] = None
        assert LIB.kv_cache_load(ctypes.byref(p), 4, 1, 1, *a, None) == NULL, i
    # a bf16 cache has no scales
    q = kv(BF)
    assert LIB.kv_cache_store(ctypes.byref(q), -1, *([OK] * 5), None, None, None) == SHAPE
    for i in (0, 1, 3, 4):
        a = [OK] * 7
        a[i] = ODD
        assert LIB.kv_cache_store(ctypes.byref(p), 4, *a, None) == ALIGN, i
    assert LIB.kv_cache_load(ctypes.byref(p), -1, 1, 1, *([OK] * 8), None) == SHAPE
    assert LIB.kv_cache_load(ctypes.byref(p), 4, 0, 1, *([OK] * 8), None) == SHAPE
    assert LIB.kv_cache_store(ctypes.byref(p), 2 ** 31 - 1, *([OK] * 7), None) == UNSUP


def decode(**kw):
    p = ssd.make_attn_decode_problem(kv(), 2, 3, 8, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(num_reqs=-1), SHAPE), (dict(tokens_per_req=-1), SHAPE), (dict(nheads=7), SHAPE),
    (dict(nheads=0), SHAPE), (dict(max_pages=-1), SHAPE), (dict(num_reqs=70000), UNSUP),
    (dict(max_pages=2 ** 30), UNSUP), (dict(scale=-0.5), SHAPE), (dict(q_stride=8), SHAPE),
    (dict(o_stride=8), SHAPE), (dict(q_stride=516), ALIGN), (dict(kv=kv(in_dtype=0)), UNSUP),
    (dict(kv=kv(page_size=24)), UNSUP), (dict(kv=kv(num_pages=0)), SHAPE),
])
def test_decode_refusals(kw, status):
    p = decode(**kw)
    rc = LIB.attention_decode(ctypes.byref(p), *([OK] * 8), None, OK, ctypes.c_size_t(1 << 40), None)
    assert rc == status
    if status not in (ALIGN,):
        assert ssd.attn_decode_workspace_bytes(p) == 0


def test_decode_pointers_and_workspace():
    p = decode()
    for i in range(8):
        a = [OK] * 8
        a[i] = None
        assert LIB.attention_decode(ctypes.byref(p), *a, None, OK, ctypes.c_size_t(1 << 40),
                                    None) == NULL, i
    need = ssd.attn_decode_workspace_bytes(p)       # 4096-token contexts of 2 requests: split
    assert need > 0
    call = lambda ws, n: LIB.attention_decode(ctypes.byref(p), *([OK] * 8), None, ws,   # noqa: E731
                                              ctypes.c_size_t(n), None)
    assert call(OK, need - 1) == WORK and call(None, need) == NULL and call(ODD, need) == ALIGN
    # contexts of one page: nothing to split, no workspace
    assert ssd.attn_decode_workspace_bytes(decode(max_pages=1)) == 0


def test_binding_checks_tensors():
    """Wrong device, type, shape or layout raise in the binding, before the library is called."""
    p = ssd.make_conv_problem(4, 1, 8, 4, 1, BF, BF)
    x = torch.zeros(4, 8, dtype=BF)
    with pytest.raises(ValueError, match="on the GPU"):
        ssd.causal_conv1d_varlen(p, x, None, None, None, None, None, None, x)
    with pytest.raises(KeyError):
        ssd.make_kv_cache_problem(1, 64, 1, 64, BF, torch.float16)
    with pytest.raises(ValueError, match="no scales"):
        q = ssd.make_kv_cache_problem(1, 64, 1, 64, BF, BF)
        ssd.layer_ops._kv_ptrs(q, x, x, x, x)


def test_attention_weights_choice():
    assert call_attn(attn(bf16_weights=2)) == UNSUP and call_attn(attn(bf16_weights=-1)) == UNSUP
    assert ssd.make_attn_problem(1, 1, 1, 1, 1, 64, BF).bf16_weights == 0
    assert ssd.make_attn_problem(1, 1, 1, 1, 1, 64, BF, bf16_weights=True).bf16_weights == 1
    assert ctypes.sizeof(ssd.attn_problem) == 72       # (the field took a reserved one's place)


def test_scan_takes_step_size_transforms_only():
    """Another struct's bytes would be read as a device pointer and bounds."""
    p = scan()
    for wrong in (conv(), p, 0.5, (0.0, 1.0)):
        with pytest.raises(TypeError, match="dt_transform"):
            ssd.layer_ops._scan_transform(p, wrong)
    good = ssd.make_dt_transform(None, 0.0, 1.0)
    assert ssd.layer_ops._scan_transform(p, good) == ctypes.addressof(good)
    assert ssd.layer_ops._scan_transform(p, None) is None

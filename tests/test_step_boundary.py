"""Refusals of the operators between and behind the layers: every bad argument is turned down on the
host, before anything reaches the GPU (no GPU needed)."""
import ctypes

import pytest
import torch

ssd = pytest.importorskip("state_space_model_varlen_amd")
LIB = ssd._lib
OK = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)          # aligned to 8, not to 16
OFF = ctypes.c_void_p(257)
BF, F32, E4, U8, I32 = (torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8,
                        torch.int32)
NULL, SHAPE, DTYPE, UNSUP, WORK, ALIGN = 1, 2, 3, 4, 5, 7


def with_(p, kw):
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def norm(**kw):
    return with_(ssd.make_norm_problem(8, 64, BF, kw.pop("out", BF)), kw)


def call_norm(p, *over, residual=OK, gate=None, scale=None, keep=OK):
    a = [OK, gate, residual, OK, OK, scale, keep, None]   # x gate residual weight out scale sum stream
    for i, v in over:
        a[i] = v
    return LIB.rms_norm(ctypes.byref(p), *a)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE),
    (dict(in_dtype=2), DTYPE), (dict(in_dtype=3), DTYPE), (dict(residual_dtype=3), DTYPE),
    (dict(out_dtype=2), DTYPE), (dict(out_dtype=4), DTYPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(x_stride=63), SHAPE),
    (dict(residual_stride=63), SHAPE), (dict(residual_out_stride=-64), SHAPE), (dict(out_stride=1), SHAPE),
    (dict(gate_stride=63), SHAPE), (dict(out_dtype=3, ngroups=4), UNSUP),
    (dict(out_dtype=3, hidden=48), UNSUP), (dict(rows=2 ** 31 - 1, ngroups=2), UNSUP),
    # more threads than a launch takes
    (dict(rows=2 ** 28, hidden=1), UNSUP), (dict(rows=2 ** 26, hidden=512), UNSUP),
    (dict(rows=2 ** 22, hidden=32768), UNSUP),
    (dict(rows=1, hidden=2 ** 31 - 64), UNSUP), (dict(rows=1, hidden=2 ** 30 + 32), UNSUP),   # counts past 31 bits
    (dict(out_dtype=3), NULL),                            # no scales
])
def test_norm_refusals(kw, status):
    assert call_norm(norm(**kw)) == status


def test_norm_pointers():
    p = norm()
    for i in (0, 4):
        assert call_norm(p, (i, None)) == NULL, i
    for i in (0, 2, 3, 4, 6):
        assert call_norm(p, (i, OFF)) == ALIGN, i
    assert call_norm(p, residual=None, gate=OFF, keep=None) == ALIGN
    assert call_norm(p, residual=None) == NULL            # a sum to keep and nothing to add
    assert call_norm(p, gate=OK) == UNSUP                 # a gate and a residual
    assert LIB.rms_norm(None, *[OK] * 7, None) == NULL


def linear(**kw):
    return with_(ssd.make_linear_problem(8, 64, 48, kw.pop("x", BF), BF), kw)


def call_linear(p, *over, ws=1 << 40):
    a = [OK] * 7                                          # x x_scale weight scale bias out workspace
    for i, v in over:
        a[i] = v
    return LIB.linear_w4(ctypes.byref(p), *a, ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), SHAPE), (dict(in_features=0), SHAPE), (dict(out_features=0), SHAPE),
    (dict(x_dtype=0), DTYPE), (dict(x_dtype=2), DTYPE), (dict(out_dtype=2), DTYPE), (dict(out_dtype=3), DTYPE),
    (dict(in_features=48), UNSUP), (dict(in_features=33), UNSUP), (dict(x_stride=63), SHAPE),
    (dict(out_stride=47), SHAPE), (dict(x_stride=2 ** 21 + 32), UNSUP), (dict(in_features=2 ** 21 + 32), UNSUP),
    (dict(tokens=2 ** 31 - 1, out_features=2 ** 20), UNSUP), (dict(out_features=2 ** 28), UNSUP),
])
def test_linear_refusals(kw, status):
    p = linear(**kw)
    assert call_linear(p) == status
    assert ssd.linear_w4_workspace_bytes(p) == 0 and ssd.linear_w4_kernel(p) == ""


def test_linear_pointers():
    p = linear()
    for i in (0, 2, 3, 5):
        assert call_linear(p, (i, None)) == NULL, i
    assert call_linear(linear(x=E4), (1, None)) == NULL
    for i in (0, 2):
        assert call_linear(p, (i, ODD)) == ALIGN, i
    for i in (4, 5):
        assert call_linear(p, (i, OFF)) == ALIGN, i
    assert call_linear(linear(x_stride=68)) == ALIGN      # rows off 16 bytes
    assert LIB.linear_w4(None, *[OK] * 7, 0, None) == NULL
    enc = lambda p, dt, *a: LIB.linear_w4_encode(ctypes.byref(p), dt, *a, None)   # noqa: E731
    assert enc(p, 0, None, OK, OK) == NULL and enc(p, 0, OK, None, OK) == NULL and enc(p, 0, OK, OK, None) == NULL
    assert enc(p, 2, OK, OK, OK) == DTYPE and enc(p, 0, ODD, OK, OK) == ALIGN and enc(p, 0, OK, ODD, OK) == ALIGN
    assert enc(linear(in_features=16), 0, OK, OK, OK) == UNSUP
    assert enc(linear(out_features=0), 0, OK, OK, OK) == SHAPE
    assert enc(linear(in_features=2 ** 20, out_features=2 ** 17), 0, OK, OK, OK) == UNSUP
    assert LIB.linear_w4_encode(None, 0, OK, OK, OK, None) == NULL


def test_tiles_fit_a_launch():
    """Small tiles of more threads than a launch takes give way to larger ones."""
    threads = {"16x16": 256, "16x32": 128, "32x32": 256, "64x64": 256}
    for t, n in ((17, 2 ** 27), (16, 2 ** 28 - 2 ** 10), (2 ** 17, 2 ** 17), (2 ** 21, 2 ** 17), (100, 2 ** 27)):
        for k in (32, 4096):
            name = ssd.linear_w4_kernel(linear(tokens=t, in_features=k, out_features=n))
            rows, cols = map(int, name.split("x"))
            assert -(-t // rows) * -(-n // cols) * threads.get(name, 512) < 2 ** 32, (t, n, k, name)


def test_linear_workspace_is_checked():
    for t in (1, 16, 64, 100, 300):
        for k in (64, 1024, 8192):
            p = linear(tokens=t, in_features=k)
            need = ssd.linear_w4_workspace_bytes(p)
            if need:
                assert call_linear(p, ws=need - 1) == WORK
                assert call_linear(p, (6, None), ws=need) == NULL
                assert call_linear(p, (6, ODD), ws=need) == ALIGN


def probs(**kw):
    return with_(ssd.make_probs_problem(2, 3, 100, BF), kw)


def call_probs(p, *over, ws=1 << 40):
    a = [OK] * 4                                          # logits temperature probs workspace
    for i, v in over:
        a[i] = v
    return LIB.token_probs(ctypes.byref(p), *a, ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_reqs=-1), SHAPE), (dict(tokens_per_req=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(in_dtype=2), DTYPE),
    (dict(in_dtype=3), DTYPE), (dict(logits_stride=99), SHAPE), (dict(probs_stride=99), SHAPE),
    (dict(vocab=2 ** 27 + 1), UNSUP), (dict(num_reqs=2 ** 30), UNSUP), (dict(num_reqs=2 ** 17, vocab=2 ** 26), UNSUP),
    (dict(num_reqs=2 ** 21, vocab=1), UNSUP), (dict(num_reqs=2 ** 16, vocab=2 ** 19), UNSUP),
])
def test_probs_refusals(kw, status):
    assert call_probs(probs(**kw)) == status
    assert ssd.token_probs_workspace_bytes(probs(**kw)) == 0


def test_probs_pointers():
    for i in (0, 2):
        assert call_probs(probs(), (i, None)) == NULL
    for i in (0, 1, 2):
        assert call_probs(probs(), (i, OFF)) == ALIGN
    assert LIB.token_probs(None, *[OK] * 4, 0, None) == NULL
    for p in (probs(), probs(vocab=200000), probs(num_reqs=1, tokens_per_req=1, vocab=1 << 20)):
        need = ssd.token_probs_workspace_bytes(p)
        if need:
            assert call_probs(p, ws=need - 1) == WORK
            assert call_probs(p, (3, None), ws=need) == NULL
            assert call_probs(p, (3, ODD), ws=need) == ALIGN


def verify(**kw):
    return with_(ssd.make_verify_problem(2, 3, 100), kw)


def call_verify(p, *over, ws=1 << 40):
    a = [OK] * 8          # target draft draft_tokens num_drafts uniform num_accepted tokens workspace
    for i, v in over:
        a[i] = v
    return LIB.verify_drafts(ctypes.byref(p), *a, ctypes.c_size_t(ws), None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_reqs=-1), SHAPE), (dict(tokens_per_req=0), SHAPE), (dict(vocab=0), SHAPE),
    (dict(target_stride=99), SHAPE), (dict(draft_stride=99), SHAPE), (dict(tokens_per_req=66), UNSUP),
    (dict(vocab=2 ** 27 + 1), UNSUP), (dict(num_reqs=65536), UNSUP),
])
def test_verify_refusals(kw, status):
    assert call_verify(verify(**kw)) == status
    assert ssd.verify_drafts_workspace_bytes(verify(**kw)) == 0


def test_verify_pointers():
    p = verify()
    for i in (0, 2, 4, 5, 6):
        assert call_verify(p, (i, None)) == NULL, i
    for i in range(7):
        assert call_verify(p, (i, OFF)) == ALIGN, i
    assert ssd.verify_drafts_workspace_bytes(p) == 0
    p = verify(vocab=20000)
    need = ssd.verify_drafts_workspace_bytes(p)
    assert need > 0
    assert call_verify(p, ws=need - 1) == WORK
    assert call_verify(p, (7, None), ws=need) == NULL and call_verify(p, (7, ODD), ws=need) == ALIGN
    assert LIB.verify_drafts(None, *[OK] * 8, 0, None) == NULL


def test_binding_refuses_wrong_tensors():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)                        # noqa: E731
    p = ssd.make_norm_problem(2, 64, BF, BF)
    with pytest.raises(ValueError, match="GPU"):
        ssd.rms_norm(p, z(2, 64), None, z(2, 64))
    with pytest.raises(ValueError, match="exclude"):
        ssd.rms_norm(p, z(2, 64), None, z(2, 64), residual=z(2, 64), gate=z(2, 64))
    with pytest.raises(ValueError, match="needs residual"):
        ssd.rms_norm(p, z(2, 64), None, z(2, 64), residual_out=z(2, 64))
    with pytest.raises(ValueError, match="8-bit"):
        ssd.rms_norm(p, z(2, 64), None, z(2, 64), out_scale=z(2, 2, dtype=U8))
    lp = ssd.make_linear_problem(2, 64, 8, BF, BF)
    with pytest.raises(ValueError, match="8-bit"):
        ssd.linear_w4(lp, z(2, 64), z(8, 32, dtype=U8), z(8, 2, dtype=U8), z(2, 8), x_scale=z(2, 2, dtype=U8))
    with pytest.raises(TypeError):
        ssd.linear_w4_encode(lp, z(8, 64, dtype=torch.float16), z(8, 32, dtype=U8), z(8, 2, dtype=U8))
    with pytest.raises(KeyError):
        ssd.make_norm_problem(2, 64, E4, BF)
    with pytest.raises(KeyError):
        ssd.make_linear_problem(2, 64, 8, BF, E4)
    with pytest.raises(ValueError, match="GPU"):
        ssd.token_probs(ssd.make_probs_problem(1, 1, 8, F32), z(1, 1, 8, dtype=F32), None, z(1, 1, 8, dtype=F32))
    with pytest.raises(ValueError, match="GPU"):
        ssd.verify_drafts(ssd.make_verify_problem(1, 2, 8), z(1, 2, 8, dtype=F32), None, z(1, 1, dtype=I32), None,
                          z(1, 2, dtype=F32), z(1, dtype=I32), z(1, 2, dtype=I32))

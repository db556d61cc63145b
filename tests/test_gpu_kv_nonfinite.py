"""Cached values that are not finite and that a token does see reach its result, and no others:
token attention on the GPU against oracle/layers.py."""
import numpy as np
import pytest
import torch

from oracle import layers as ol
from test_gpu_kv_cache import decode, make

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def put_value(c, ct, table, page, r, j, dim, bad):
    """Value `bad` into dimension `dim` of request r's cached row j, every head."""
    pg, o = int(table[r, j // page]), j % page
    if ct == E4:
        c["v_cache"].view(torch.uint8)[pg, :, o, dim] = 0x7f
    else:
        c["v_cache"][pg, :, o, dim] = bad


@pytest.mark.parametrize("ct,bad", [(BF, float("inf")), (BF, float("-inf")), (BF, float("nan")),
                                    (E4, float("nan"))])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("L,D,H,Hkv", [(70, 64, 4, 2), (96, 64, 2, 1), (64, 128, 4, 1),
                                       (1100, 64, 2, 1), (1025, 128, 12, 1)])
def test_decode_values_of_the_last_tiles(ct, bad, T, L, D, H, Hkv):
    """One value that is not finite, at each of the last 64 keys and the first one (a request
    each): the tokens that see the key get it, the others and the other dimensions are as
    without it. L = 1100 and 1025 are split over blocks."""
    where = [0] + list(range(L - 64, L))
    R, page, dim = len(where), 16, 5
    lens = [L] * R
    p, c, table, q, rk, rv = make(L + T, ct, lens, T, H, Hkv, D, page)
    d = ssd.make_attn_decode_problem(p, R, T, H, table.shape[1])
    assert (ssd.attn_decode_workspace_bytes(d) > 0) == (L > 128)
    want, _, mag, top = ol.decode_attention(q, rk, rv, lens)
    for r, j in enumerate(where):
        put_value(c, ct, table, page, r, j, dim, bad)
    got = decode(p, c, table, q, lens)[0].cpu().double().numpy()
    tol = ol.attention_tolerance(want, mag, top, D, L, BF)
    sees = np.array([[j <= L - T + t for t in range(T)] for j in where])
    hit = got[sees][:, :, dim]
    assert np.isnan(hit).all() if np.isnan(bad) else (hit == bad).all(), \
        [where[r] for r in range(R) if np.isfinite(got[r][sees[r]][:, :, dim]).any()]
    clean = np.ones(got.shape, dtype=bool)
    clean[sees, :, dim] = False
    assert np.all(np.abs(got - want)[clean] <= tol[clean])


@pytest.mark.parametrize("ct", [BF, E4])
def test_decode_values_seen_by_some_tokens(ct):
    """Contexts of 33 .. 40 keys, the last 8 values of each not finite, 8 tokens a request: token t
    sees the first t + 1 of them."""
    lens = list(range(33, 41))
    p, c, table, q, rk, rv = make(3, ct, lens, 8, 2, 1, 64, 16)
    want, _, mag, top = ol.decode_attention(q, rk, rv, lens)
    for r, L in enumerate(lens):
        for i in range(8):
            put_value(c, ct, table, 16, r, L - 8 + i, i, float("nan"))
    got = decode(p, c, table, q, lens)[0].cpu().double().numpy()
    tol = ol.attention_tolerance(want, mag, top, 64, 40, BF)
    for t in range(8):
        assert np.isnan(got[:, t, :, :t + 1]).all()
        assert np.all((np.abs(got - want) <= tol)[:, t, :, t + 1:])

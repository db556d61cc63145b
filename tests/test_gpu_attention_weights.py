"""Attention's softmax weights on the GPU are as good as float32: against oracle/layers.py, within a
tolerance that has no room for weights rounded to bf16.

A weight goes into the bf16 products as its rounded value and what that rounding left, rounded in
turn: off by at most 2^-8 2^-8 of itself. Beside it, as in attention_tolerance: the score's sum
(which moves a weight and the weights' sum), two products a key in the result's sum, and the
rounding of the result, 2^-8 of its own value. Results near zero, the sum of values that cancel,
are where weights of 8 bits show."""
import numpy as np
import pytest
import torch

from oracle import layers as ol
from test_gpu_attention import call, compare as compare_rounded, make
from test_gpu_kv_cache import decode, make as make_cache

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
DEV = "cuda"


def compare(out, ref, D, nk):
    want, _, mag, top = ref
    got = out.cpu().double().numpy()
    rel = 2 * ((2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -20) + (2 * nk + 8) * 2.0 ** -24 + 2.0 ** -16
    bad = ~(np.abs(got - want) <= rel[..., None] * mag + 2.0 ** -8 * np.abs(want) + 1e-30)
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(np.abs(got - want))))


@pytest.mark.parametrize("ct", [BF, E4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,T,lens", [(4, 4, 1, [2, 5, 40]), (8, 1, 3, [3, 33, 64]),
                                          (24, 2, 2, [4, 17, 129]), (4, 2, 1, [1100, 3, 257])])
def test_tokens(ct, D, H, Hkv, T, lens):
    p, c, table, q, rk, rv = make_cache(H + T + D, ct, lens, T, H, Hkv, D, 16)
    compare(decode(p, c, table, q, lens)[0], ol.decode_attention(q, rk, rv, lens), D, max(lens))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,T,L,zero", [(2, 1, 75, False), (2, 1, 75, True), (12, 2, 700, False)])
def test_tokens_with_infinite_values(D, H, T, L, zero):
    """Infinities among the values come out as they are, whatever a weight's remainder is (of equal
    scores, q = 0, it is nothing); both signs of one give NaN; a NaN stays one."""
    lens = [L, L]
    p, c, table, q, rk, rv = make_cache(L + D, BF, lens, T, H, 1, D, 16)
    q = torch.zeros_like(q) if zero else q
    want, _, mag, top = ol.decode_attention(q, rk, rv, lens)
    inf = float("inf")
    for j, dim, bad in ((0, 1, inf), (37, 2, -inf), (3, 3, inf), (40, 3, inf), (4, 4, inf), (33, 4, -inf),
                        (5, 6, float("nan"))):
        c["v_cache"][int(table[0, j // 16]), :, j % 16, dim] = bad
    got = decode(p, c, table, q, lens)[0].cpu().double().numpy()
    for dim, bad in ((1, inf), (2, -inf), (3, inf)):
        assert (got[0, :, :, dim] == bad).all(), dim
    assert np.isnan(got[0][:, :, [4, 6]]).all()
    tol = ol.attention_tolerance(want, mag, top, D, L, BF)
    keep = np.ones(got.shape, dtype=bool)
    keep[0][:, :, [1, 2, 3, 4, 6]] = False
    assert np.all(np.abs(got - want)[keep] <= tol[keep])


# whole blocks of 1, 2 and 4 heads of a group and of groups of 5; few heads, whose keys are shared
HEADS = [(160, 160), (160, 80), (160, 40), (160, 32), (4, 2), (5, 1)]
LENS = [([3, 1, 66], [3, 5, 70], True), ([33, 2], [200, 7], True), ([20, 4], [9, 33], False)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", HEADS)
@pytest.mark.parametrize("lens,klens,causal", LENS)
def test_prompts(D, H, Hkv, lens, klens, causal):
    m = make(sum(lens) + D, lens, klens, H, Hkv, D, BF)
    out, _ = call(m, m["q"].to(DEV), m["k"].to(DEV), m["v"].to(DEV), causal)
    compare(out, ol.attention(m["q"], m["k"], m["v"], m["cuq"], m["cuk"], causal), D, max(klens))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", HEADS)
@pytest.mark.parametrize("zero", [False, True])
def test_prompts_with_infinite_values(D, H, Hkv, zero):
    """As test_tokens_with_infinite_values: in tiles that every query of a block sees, and in those
    that hide keys from some."""
    lens, klens = [40, 150], [240, 150]
    m = make(7 + D, lens, klens, H, Hkv, D, BF)
    q = torch.zeros_like(m["q"]) if zero else m["q"]
    want, _, mag, top = ol.attention(q, m["k"], m["v"], m["cuq"], m["cuk"])
    v, inf = m["v"].clone(), float("inf")
    put = ((0, 1, inf), (67, 2, -inf), (3, 3, inf), (220, 3, inf), (4, 4, inf), (133, 4, -inf),
           (5, 6, float("nan")), (130, 8, inf), (239, 9, inf), (230, 10, inf), (1, 10, -inf))
    for j, dim, bad in put:
        v[j, :, dim] = bad
    v[240 + 100, :, 7] = inf                     # sequence 1: seen by its queries from 100 on
    out, _ = call(m, q.to(DEV), m["k"].to(DEV), v.to(DEV))
    got = out.cpu().double().numpy()
    for dim in {d for _, d, _ in put}:
        for i in range(40):
            seen = sum(b for j, d, b in put if d == dim and j <= i + 200)
            assert np.array_equal(got[i, :, dim], np.full(H, seen), equal_nan=True) or seen == 0, (i, dim)
    assert (got[40 + 100:, :, 7] == inf).all()
    keep = np.ones(got.shape, dtype=bool)
    for j, dim, _ in put:
        keep[max(0, j - 200):40, :, dim] = False
    keep[40 + 100:, :, 7] = False
    tol = ol.attention_tolerance(want, mag, top, D, 240, BF)
    assert np.all(np.abs(got - want)[keep] <= tol[keep])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_prompts_with_rounded_weights(D, H, Hkv):
    """bf16_weights: within the tolerance that has room for them, and hidden values stay hidden."""
    lens, klens = [40, 1, 130], [104, 200, 131]
    m = make(9 + D, lens, klens, H, Hkv, D, BF)
    p = ssd.make_attn_problem(171, 435, 3, H, Hkv, D, BF, bf16_weights=True)
    v = m["v"].clone()
    v[103, :, 5] = float("nan")                  # the last key of sequence 0
    out, lse = torch.full(m["q"].shape, 7.0, dtype=BF, device=DEV), torch.zeros(171, H, device=DEV)
    ssd.attention_varlen(p, m["q"].to(DEV), m["k"].to(DEV), v.to(DEV), m["cuq"].to(DEV), m["cuk"].to(DEV),
                         out, lse)
    assert torch.isnan(out[39, :, 5]).all()
    ref = ol.attention(m["q"], m["k"], m["v"], m["cuq"], m["cuk"])
    out[39, :, 5] = torch.as_tensor(ref[0][39, :, 5]).to(BF)
    compare_rounded(out, lse, ref, D, 200, BF)

"""Every kernel of prompt attention on its own ground, on the GPU: long keys (tiles in both buffers,
again and again), running maxima that rise, many sequences, strided rows, streams and graphs. Each
test says which kernel it means and checks that the host's rule takes it.

The reference is the definition in float64, a sequence and head at a time (tested against
oracle/layers.py, which goes row by row); the tolerance is attention_tolerance's, with two products
a key and weights off by 2^-16 of themselves in bf16."""
import numpy as np
import pytest
import torch

from oracle import layers as ol
from test_gpu_attention import make, packed

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def reference(q, k, v, cuq, cuk, causal=True, scale=None):
    """out, lse, mag, top as oracle.layers.attention has them, in float64 on q's device."""
    q, k, v = (t.double() for t in (q, k, v))
    H, D = q.shape[1:]
    group, scale = H // k.shape[1], D ** -0.5 if scale is None else scale
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse, top = torch.full_like(q[..., 0], -torch.inf), torch.zeros_like(q[..., 0])
    for s in range(len(cuq) - 1):
        a, e, ka, ke = (int(x) for x in (cuq[s], cuq[s + 1], cuk[s], cuk[s + 1]))
        if e == a or ke == ka:
            continue
        rows = torch.arange(e - a, device=q.device)
        seen = rows + (ke - ka) - (e - a) if causal else rows * 0 + ke - ka - 1
        hide = torch.arange(ke - ka, device=q.device) > seen[:, None]
        some = seen >= 0
        for h in range(H):
            qq, kk, vv = q[a:e, h], k[ka:ke, h // group], v[ka:ke, h // group]
            sc = (scale * (qq @ kk.T)).masked_fill(hide, -torch.inf)
            lse[a:e, h] = torch.logsumexp(sc, 1)
            p = torch.where(some[:, None], torch.softmax(sc, 1), 0.0)
            out[a:e, h], mag[a:e, h] = p @ vv, p @ vv.abs()
            top[a:e, h] = (scale * (qq.abs() @ kk.abs().T)).masked_fill(hide, 0.0).amax(1)
    return out, lse, mag, top


def close(out, lse, ref, D, nk, dt, where=None):
    want, wl, mag, top = ref
    bf = dt == BF
    rel = 2 * ((2 * D + 8) * 2.0 ** -24 * top + 2.0 ** -20) + ((2 if bf else 1) * nk + 8) * 2.0 ** -24
    tol = (rel + (2.0 ** -16 if bf else 0.0))[..., None] * mag + ol.STEP[dt] * want.abs() + 1e-30
    good = (out.double() - want).abs() <= tol
    if where is not None:
        good = good | ~where
    assert bool(good.all()), (int((~good).sum()), good.numel())
    if lse is not None:
        inf = torch.isneginf(wl)
        assert torch.equal(torch.isneginf(lse), inf)
        tl = (2 * D + 8) * 2.0 ** -24 * top + (nk + 16) * 2.0 ** -24 + 2.0 ** -22 * wl.abs()
        assert bool((((lse.double() - wl).abs() <= tl) | inf).all())


def go(kernel, m, q, k, v, causal=True, scale=None, lse=True):
    """attention_varlen into the first rows of longer arrays, whose rest has to stay."""
    T, H, D = q.shape
    p = ssd.make_attn_problem(T, k.shape[0], len(m["lens"]), H, k.shape[1], D, q.dtype, causal, scale or 0.0)
    assert ssd.attention_varlen_kernel(p) == kernel
    out = torch.full((T + 130, H, D), 7.0, dtype=q.dtype, device=DEV)
    ls = torch.full((T + 130, H), 7.0, device=DEV)
    ssd.attention_varlen(p, q, k, v, m["cuq"].to(DEV), m["cuk"].to(DEV), out[:T], ls[:T] if lse else None)
    assert bool((out[T:] == 7.0).all()) and bool((ls[T:] == 7.0).all())
    return out[:T], ls[:T] if lse else None


def run(kernel, seed, lens, klens, H, Hkv, D, dt, causal=True, scale=None, spread=1.0):
    m = make(seed, lens, klens, H, Hkv, D, dt, spread)
    q, k, v = (m[n].to(DEV) for n in "qkv")
    out, lse = go(kernel, m, q, k, v, causal, scale)
    close(out, lse, reference(q, k, v, m["cuq"], m["cuk"], causal, scale), D, max(klens), dt)


def test_the_reference():
    for causal in (True, False):
        m = make(1, [5, 0, 9, 3], [7, 2, 4, 0], 4, 2, 64, F32)
        want = ol.attention(m["q"], m["k"], m["v"], m["cuq"], m["cuk"], causal, 0.3)
        got = reference(m["q"].to(DEV), m["k"].to(DEV), m["v"].to(DEV), m["cuq"], m["cuk"], causal, 0.3)
        for a, b in zip(got, want):
            assert np.allclose(a.cpu().numpy(), b, rtol=1e-12, atol=1e-12)


# heads and the heads of a group that a block takes: 1, 1 of 5, 2, 4
BLOCKS = [(40, 40, 1), (40, 8, 1), (48, 24, 2), (48, 12, 4)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", BLOCKS)
def test_long_prompts(H, Hkv, hpb, D):
    run("attn_kernel<%d, %d>" % (D, hpb), D + H, [1500], [1500], H, Hkv, D, BF)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", BLOCKS)
def test_continued_prompts(H, Hkv, hpb, D):
    run("attn_kernel<%d, %d>" % (D, hpb), 2 + D + H, [130, 700, 1, 0, 333], [1130, 1400, 999, 3, 100], H, Hkv,
        D, BF)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", BLOCKS)
def test_all_keys(H, Hkv, hpb, D):
    run("attn_kernel<%d, %d>" % (D, hpb), 3 + D + H, [900, 261], [1001, 190], H, Hkv, D, BF, causal=False,
        scale=0.2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", BLOCKS)
def test_large_scores(H, Hkv, hpb, D):
    # the running maximum rises by hundreds, in tile after tile
    run("attn_kernel<%d, %d>" % (D, hpb), 4 + D + H, [1400], [1400], H, Hkv, D, BF, spread=20.0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", [(40, 40, 1), (10, 2, 4), (16, 8, 2), (16, 4, 4)])
def test_many_sequences(H, Hkv, hpb, D):
    lens = [(3 * i) % 7 + (150 if i % 50 == 0 else 0) for i in range(130)]
    run("attn_kernel<%d, %d>" % (D, hpb), 5, lens, [n + i % 70 for i, n in enumerate(lens)], H, Hkv, D, BF)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", BLOCKS)
def test_rows_of_a_fused_projection(H, Hkv, hpb, D):
    g = torch.Generator().manual_seed(8)
    lens = [700, 440]
    row = torch.randn(sum(lens), (H + 2 * Hkv) * D + 8, generator=g).to(BF).to(DEV)
    q = row[:, :H * D].unflatten(1, (H, D))
    k, v = (row[:, (H + i * Hkv) * D:(H + (i + 1) * Hkv) * D].unflatten(1, (Hkv, D)) for i in (0, 1))
    m = dict(lens=lens, klens=lens, cuq=packed(lens), cuk=packed(lens))
    out, lse = go("attn_kernel<%d, %d>" % (D, hpb), m, q, k, v)
    close(out, lse, reference(q, k, v, m["cuq"], m["cuk"]), D, 700, BF)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv,hpb", BLOCKS)
def test_hidden_rows_of_long_prompts(H, Hkv, hpb, D):
    """Keys and values that are not finite from key 1000 on, and a value at key 10."""
    m = make(6, [1300], [1300], H, Hkv, D, BF)
    q, k, v = (m[n].to(DEV) for n in "qkv")
    ref = reference(q, k, v, m["cuq"], m["cuk"])
    k[1000:, :, 3], v[1000:] = float("nan"), float("inf")
    v[10, :, 7] = float("-inf")
    out, _ = go("attn_kernel<%d, %d>" % (D, hpb), m, q, k, v, lse=False)
    where = torch.ones(out.shape, dtype=torch.bool, device=DEV)
    where[1000:], where[10:, :, 7] = False, False
    close(out, None, ref, D, 1300, BF, where)
    assert bool((out[10:1000, :, 7] == float("-inf")).all()) and not bool(torch.isfinite(out[1000:]).any())


@pytest.mark.parametrize("kernel,H,Hkv,dt", [("attn_split_kernel<128>", 40, 40, BF), ("attn_kernel<128, 1>", 56, 56, BF),
                                             ("attn_kernel<128, 2>", 48, 24, BF),
                                             ("attn_kernel<128, 4>", 48, 12, BF),
                                             ("attn_f32_kernel<128, 2>", 40, 10, F32),
                                             ("attn_f32_kernel<128, 1>", 4, 2, F32)])
def test_another_stream_and_a_graph(kernel, H, Hkv, dt):
    m = make(11, [700, 140], [700, 600], H, Hkv, 128, dt)
    q, k, v, cuq, cuk = (m[n].to(DEV) for n in ("q", "k", "v", "cuq", "cuk"))
    p = ssd.make_attn_problem(840, 1300, 2, H, Hkv, 128, dt)
    assert ssd.attention_varlen_kernel(p) == kernel
    out = torch.empty_like(q)
    call = lambda: ssd.attention_varlen(p, q, k, v, cuq, cuk, out)           # noqa: E731
    call()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        call()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# the form whose waves share the keys: past two rounds of blocks too
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,klens,H,Hkv", [([3000], [3000], 12, 12), ([32], [8000], 2, 2),
                                              ([700, 0, 90, 5], [2700, 0, 1500, 3], 8, 2)])
def test_shared_keys(D, lens, klens, H, Hkv):
    run("attn_split_kernel<%d>" % D, 12 + D, lens, klens, H, Hkv, D, BF)


# float32 with two tiles of queries a block
MOST = [(160, 160), (160, 32)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", MOST)
def test_float(D, H, Hkv):
    name = "attn_f32_kernel<%d, 2>" % D
    run(name, 20 + D, [40, 1, 130], [104, 200, 131], H, Hkv, D, F32)
    run(name, 21 + D, [9, 33, 0, 20, 2], [40, 33, 5, 10, 0], H, Hkv, D, F32)
    run(name, 22 + D, [70, 3, 0, 5], [33, 129, 7, 0], H, Hkv, D, F32, causal=False)
    run(name, 23 + D, [150, 9, 3], [20, 9, 0], H, Hkv, D, F32)       # the first queries see nothing


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [1.0, 20.0])
def test_float_on_long_keys(D, spread):
    run("attn_f32_kernel<%d, 2>" % D, 30 + D, [333], [1503], 48, 12, D, F32, spread=spread)
    run("attn_f32_kernel<%d, 2>" % D, 31 + D, [(7 * i) % 20 for i in range(70)],
        [(7 * i) % 20 + i for i in range(70)], 16, 4, D, F32, spread=spread)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H,Hkv", MOST)
def test_float_hidden_rows(D, bad, H, Hkv):
    m = make(6, [100, 70], [130, 70], H, Hkv, D, F32)
    q, k, v = (m[n].to(DEV) for n in "qkv")
    ref = reference(q, k, v, m["cuq"], m["cuk"])
    k[110:130], v[110:130, :, 5], v[130 + 40:, :, 3] = bad, bad, bad
    out, _ = go("attn_f32_kernel<%d, 2>" % D, m, q, k, v)
    where = torch.ones(out.shape, dtype=torch.bool, device=DEV)
    where[80:100], where[100 + 40:, :, 3] = False, False
    close(out, None, ref, D, 130, F32, where)
    assert not bool(torch.isfinite(out[100 + 40:, :, 3]).any())

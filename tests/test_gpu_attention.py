"""Attention over packed prompts on the GPU against oracle/layers.py (attention_tolerance says
what a result may be off by)."""
import numpy as np
import pytest
import torch

from oracle import layers as ol

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def packed(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def make(seed, lens, klens, H, Hkv, D, dt, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return dict(q=(torch.randn(sum(lens), H, D, generator=g) * spread).to(dt),
                k=torch.randn(sum(klens), Hkv, D, generator=g).to(dt),
                v=torch.randn(sum(klens), Hkv, D, generator=g).to(dt), cuq=packed(lens),
                cuk=packed(klens), lens=lens, klens=klens)


def call(m, q, k, v, causal=True, scale=0.0, lse=True):
    p = ssd.make_attn_problem(q.shape[0], k.shape[0], len(m["lens"]), q.shape[1], k.shape[1],
                              q.shape[2], q.dtype, causal, scale)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    ls = torch.full(q.shape[:2], 7.0, device=DEV) if lse else None
    ssd.attention_varlen(p, q, k, v, m["cuq"].to(DEV), m["cuk"].to(DEV), out, ls)
    return out, ls


def compare(out, lse, ref, D, nk, dt):
    want, wl, mag, top = ref
    got = out.cpu().double().numpy()
    tol = ol.attention_tolerance(want, mag, top, D, nk, dt)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want))))
    if lse is not None:
        f = np.isfinite(wl)
        gl = lse.cpu().double().numpy()
        assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
        gl, wl = np.where(f, gl, 0), np.where(f, wl, 0)
        tl = (2 * D + 8) * 2.0 ** -24 * top + (nk + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(
            np.where(f, wl, 0))
        assert np.all(np.abs(gl - wl)[f] <= tl[f])


def run(seed, lens, klens, H, Hkv, D, dt, causal=True, scale=None, spread=1.0):
    m = make(seed, lens, klens, H, Hkv, D, dt, spread)
    out, lse = call(m, m["q"].to(DEV), m["k"].to(DEV), m["v"].to(DEV), causal, scale or 0.0)
    ref = ol.attention(m["q"], m["k"], m["v"], m["cuq"], m["cuk"], causal, scale)
    compare(out, lse, ref, D, max(klens + [0]), dt)


LENS = [([1], [1]), ([63, 0, 65, 1], [63, 0, 65, 1]), ([127, 129], [127, 129]),
        ([40, 1, 130], [104, 200, 131])]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,klens", LENS)
def test_causal(dt, D, lens, klens):
    run(len(lens) + D, lens, klens, 4, 2, D, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (8, 8), (12, 3)])
def test_heads(dt, H, Hkv):
    run(H, [70, 33], [70, 90], H, Hkv, 64, dt)


# many heads: whole blocks of 1, 2 or 4 heads of a group, and groups that do not fill them
MANY = [(64, 64), (64, 32), (64, 16), (40, 8), (48, 16)]


@pytest.mark.parametrize("H,Hkv", MANY)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,klens", [([63, 0, 65, 1], [63, 9, 100, 129]), ([129], [300]),
                                        ([9, 33, 20, 2], [40, 33, 10, 0])])
def test_many_heads(H, Hkv, D, lens, klens):
    run(H + Hkv, lens, klens, H, Hkv, D, BF)


@pytest.mark.parametrize("H,Hkv,dt", [(64, 64, BF), (64, 16, BF), (64, 32, F32)])
def test_many_heads_full(H, Hkv, dt):
    run(12, [70, 3, 0, 5], [33, 129, 7, 0], H, Hkv, 64, dt, causal=False)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_full_and_scaled(dt, D):
    run(2, [70, 3, 0, 5], [33, 129, 7, 0], 2, 1, D, dt, causal=False)
    run(3, [70], [70], 2, 1, D, dt, scale=0.5)


@pytest.mark.parametrize("dt", [BF, F32])
def test_large_scores(dt):
    # the running maximum rises by hundreds; most weights vanish
    run(4, [200], [200], 2, 1, 64, dt, spread=20.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_queries_that_see_nothing(dt):
    # more queries than keys: the first ones have none
    run(5, [150, 9, 3], [20, 9, 0], 4, 2, 64, dt)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H,Hkv", [(2, 1), (48, 48), (64, 16)])
def test_hidden_rows_do_not_matter(dt, D, bad, H, Hkv):
    """Non-finite keys and values behind a query, in the same sequence or the next, change
    nothing; a value seen by a query reaches it."""
    lens, klens = [100, 70], [130, 70]
    m = make(6, lens, klens, H, Hkv, D, dt)
    ref = ol.attention(m["q"], m["k"], m["v"], m["cuq"], m["cuk"])
    k, v = m["k"].clone(), m["v"].clone()
    k[110:130] = bad           # seen by the last 20 queries of sequence 0 at most
    v[110:130, :, 5] = bad
    v[130 + 40:, :, 3] = bad   # sequence 1, places 40 ..
    out, _ = call(m, m["q"].to(DEV), k.to(DEV), v.to(DEV))
    got, want = out.cpu().double().numpy(), ref[0]
    tol = ol.attention_tolerance(want, ref[2], ref[3], D, 130, dt)
    clean = np.ones(got.shape, dtype=bool)
    clean[80:100] = False                      # they see a bad key: whatever comes of it
    clean[100 + 40:, :, 3] = False
    assert np.all(np.abs(got - want)[clean] <= tol[clean])
    assert not np.isfinite(got[100 + 40:, :, 3]).any()


# enough heads for a whole block of queries each (with fewer, waves share the keys): blocks
# of 1, 2 and 4 heads of a group, and of groups of 5
MOST = [(160, 160), (160, 80), (160, 40), (160, 32)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("H,Hkv", MOST)
def test_hidden_rows_do_not_matter_to_most_heads(D, bad, H, Hkv):
    test_hidden_rows_do_not_matter(BF, D, bad, H, Hkv)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", MOST)
def test_most_heads(D, H, Hkv):
    run(20 + D, [40, 1, 130], [104, 200, 131], H, Hkv, D, BF)
    run(21 + D, [9, 33, 0, 20, 2], [40, 33, 5, 10, 0], H, Hkv, D, BF)
    run(22 + D, [70, 3, 0, 5], [33, 129, 7, 0], H, Hkv, D, BF, causal=False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,klens", [([1100], [1100]), ([40, 33, 2, 1], [900, 33, 1500, 1]), ([33], [1300])])
def test_few_heads_on_long_keys(D, lens, klens):
    """Several rounds of key tiles for the waves that share them, past a queries' tile end too."""
    run(30 + D, lens, klens, 4, 2, D, BF)


@pytest.mark.parametrize("dt", [BF, F32])
def test_rows_of_a_fused_projection(dt):
    g = torch.Generator().manual_seed(8)
    T, H, Hkv, D = 90, 4, 2, 64
    row = torch.randn(T, (H + 2 * Hkv) * D + 8, generator=g).to(dt)
    cut = lambda t: (t[:, :H * D].unflatten(1, (H, D)),                      # noqa: E731
                     t[:, H * D:(H + Hkv) * D].unflatten(1, (Hkv, D)),
                     t[:, (H + Hkv) * D:(H + 2 * Hkv) * D].unflatten(1, (Hkv, D)))
    m = dict(lens=[50, 40], klens=[50, 40], cuq=packed([50, 40]), cuk=packed([50, 40]))
    out, lse = call(m, *cut(row.to(DEV)))
    compare(out, lse, ol.attention(*cut(row), m["cuq"], m["cuk"]), D, 50, dt)


def test_many_sequences():
    lens = [(3 * i) % 7 for i in range(130)]
    run(9, lens, [n + i % 5 for i, n in enumerate(lens)], 2, 1, 64, BF)


def test_long_prompt_sampled_rows():
    """8 K queries: sampled rows against the definition, and all against the plain form on the GPU."""
    m = make(10, [8200], [8200], 4, 1, 128, BF)
    out, lse = call(m, m["q"].to(DEV), m["k"].to(DEV), m["v"].to(DEV))
    for i in (0, 1, 63, 64, 127, 128, 4095, 4096, 8191, 8199):
        ref = ol.attention(m["q"][i:i + 1], m["k"][:i + 1], m["v"][:i + 1], [0, 1], [0, i + 1])
        compare(out[i:i + 1], lse[i:i + 1], ref, 128, i + 1, BF)


def test_another_stream_and_a_graph():
    m = make(11, [300, 40], [300, 100], 4, 2, 128, BF)
    q, k, v, cuq, cuk = (m[n].to(DEV) for n in ("q", "k", "v", "cuq", "cuk"))
    p = ssd.make_attn_problem(340, 400, 2, 4, 2, 128, BF)
    out = torch.empty_like(q)
    go = lambda: ssd.attention_varlen(p, q, k, v, cuq, cuk, out)             # noqa: E731
    go()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        go()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

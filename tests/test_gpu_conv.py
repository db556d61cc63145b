"""The short causal convolution on the GPU against oracle/layers.py.

Tolerance per element: the sum of W products and the bias in float32, at most (2 W + 2) roundings
of 2^-24 of its magnitudes, the activation a few more (its exponential and reciprocal are good to
2^-22, and it is no steeper than 1.1), and the rounding of the result.
"""
import numpy as np
import pytest
import torch

from oracle import layers as ol

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def make(seed, lens, C, W, ti, ts, slots=None, row=None, at=0):
    g = torch.Generator().manual_seed(seed)
    T, S = sum(lens), len(lens)
    wide = torch.randn(T, row or C, generator=g).to(ti)
    idx = torch.randperm(S + 2, generator=g)[:S].to(torch.int32) if slots is None else \
        torch.tensor(slots, dtype=torch.int32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    has = (torch.arange(S) % 2).to(torch.uint8)
    return dict(wide=wide, x=wide[:, at:at + C], w=torch.randn(C, W, generator=g) * W ** -0.5,
                b=torch.randn(C, generator=g) * 0.1, cu=cu, idx=idx, has=has,
                cache=torch.randn(S + 2, W - 1, C, generator=g).to(ts), T=T, S=S, C=C, W=W, ti=ti,
                ts=ts, at=at)


def check(got, want, mag, W, ti):
    got = got.cpu().double().numpy()
    tol = ol.STEP[ti] * np.abs(want) + ((2 * W + 2) * 2.0 ** -24 * 1.1 + 2.0 ** -21) * mag + 1e-30
    bad = np.abs(got - want) > tol
    assert not bad.any(), (bad.sum(), np.abs(got - want).max())


def check_cache(got, want, ts):
    want = torch.as_tensor(want).to(ts)        # rows are copied: one rounding at most
    assert torch.equal(got.cpu(), want)


def run(m, split=None, act="silu", has=True, bias=True):
    d = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in m.items()}
    x = d["wide"][:, m["at"]:m["at"] + m["C"]]
    p = ssd.make_conv_problem(m["T"], m["S"], m["C"], m["W"], m["S"] + 2, m["ti"], m["ts"], act)
    ys = [torch.full((m["T"], c), 7.0, dtype=m["ti"], device=DEV) for c in (split or [m["C"]])]
    cache = d["cache"].clone()
    ssd.causal_conv1d_varlen(p, x, d["w"], d["b"] if bias else None, d["cu"], cache, d["idx"],
                             d["has"] if has else None, ys[0] if split is None else tuple(ys))
    want, left, mag = ol.conv(m["x"], m["w"], m["b"] if bias else None, m["cu"], m["cache"],
                              m["idx"], m["has"] if has else None, act == "silu")
    check(torch.cat(ys, 1), want, mag, m["W"], m["ti"])
    check_cache(cache, left, m["ts"])


@pytest.mark.parametrize("ti,ts", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [2, 0, 3, 17], [15, 33, 1, 0, 64, 16]])
def test_prompts(ti, ts, W, lens):
    run(make(len(lens) + W, lens, 520, W, ti, ts))


@pytest.mark.parametrize("C", [1, 7, 65, 513])
def test_odd_channels(C):
    run(make(C, [5, 40, 3], C, 4, BF, BF))


@pytest.mark.parametrize("act,has,bias", [("none", True, True), ("silu", False, True),
                                          ("silu", True, False)])
def test_options(act, has, bias):
    run(make(3, [9, 20], 24, 4, BF, BF), act=act, has=has, bias=bias)


@pytest.mark.parametrize("split", [[64, 16, 16], [88, 8], [60, 18, 18], [95, 1]])
def test_split_outputs(split):
    run(make(4, [30, 1, 21], 96, 4, BF, BF), split=split)


@pytest.mark.parametrize("row,at", [(200, 96), (199, 96), (200, 97), (104, 8)])
def test_rows_of_a_wider_projection(row, at):
    run(make(5, [30, 1, 21], 96, 4, BF, BF, row=row, at=at))


def test_more_sequences_than_lanes():
    run(make(6, [(7 * i) % 5 for i in range(200)], 40, 4, BF, BF))


def test_bad_slots_are_skipped():
    m = make(7, [6, 20, 5], 32, 4, BF, BF, slots=[-1, 2, 5])
    run(m)     # slots -1 and 5 (of 5): no initial rows, nothing written


def test_nothing_to_do():
    p = ssd.make_conv_problem(0, 0, 32, 4, 2, BF, BF)
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device=DEV)     # noqa: E731
    cache = torch.ones(2, 3, 32, dtype=BF, device=DEV)
    ssd.causal_conv1d_varlen(p, e(0, 32), e(32, 4, dtype=F32), None,
                             torch.zeros(1, dtype=torch.int32, device=DEV), cache,
                             e(0, dtype=torch.int32), None, e(0, 32))
    torch.cuda.synchronize()
    assert bool((cache == 1).all())


@pytest.mark.parametrize("ti,ts", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("R,T,C", [(1, 1, 520), (5, 3, 520), (3, 7, 33), (70, 4, 64)])
def test_update_and_commit(ti, ts, R, T, C):
    m = make(R + T, [T] * R, C, 4, ti, ts)
    m["idx"][0] = -1 if R > 2 else m["idx"][0]
    d = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in m.items()}
    p = ssd.make_conv_problem(R * T, R, C, 4, R + 2, ti, ts)
    one = torch.ones(R, dtype=torch.uint8)
    want, left, mag = ol.conv(m["x"], m["w"], m["b"], m["cu"], m["cache"], m["idx"], one)
    y, cache = torch.empty_like(d["x"]), d["cache"].clone()
    ssd.causal_conv1d_update(p, d["x"], d["w"], d["b"], cache, d["idx"], y)
    check(y, want, mag, 4, ti)
    check_cache(cache, left, ts)
    # a verify step leaves the cache; the commit takes 1 + accepted tokens in
    y2, kept = torch.empty_like(y), d["cache"].clone()
    ssd.causal_conv1d_update(p, d["x"], d["w"], d["b"], kept, d["idx"], y2, update_cache=False)
    assert torch.equal(y, y2) and torch.equal(kept, d["cache"])
    acc = torch.tensor([(i % (T + 2)) - 1 for i in range(R)], dtype=torch.int32)   # -1 .. T
    ssd.causal_conv1d_commit(p, d["x"], kept, d["idx"], acc.to(DEV))
    ref = m["cache"].clone()
    for r in range(R):
        a, s = int(acc[r]), int(m["idx"][r])
        if 0 <= a < T and s >= 0:
            rows = torch.cat([ref[s].to(ti).float() if ts == BF else ref[s].float(),
                              m["x"][r * T:r * T + a + 1].float()])
            ref[s] = rows[-3:].to(ts)
    assert torch.equal(kept.cpu(), ref)


def test_another_stream_and_a_graph():
    m = make(9, [40, 3, 90], 256, 4, BF, BF)
    d = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in m.items()}
    p = ssd.make_conv_problem(m["T"], 3, 256, 4, 5, BF, BF)
    y, cache = torch.empty_like(d["x"]), d["cache"].clone()
    call = lambda: ssd.causal_conv1d_varlen(p, d["x"], d["w"], d["b"], d["cu"], cache,   # noqa: E731
                                            d["idx"], d["has"], y)
    call()
    want, left = y.clone(), cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.zero_()
        cache.copy_(d["cache"])
        call()
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(cache, left)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        y.zero_()
        cache.copy_(d["cache"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(cache, left)

"""Every form of the channel-wise scan's prompt kernel on its own ground, on the GPU: 4 and 16 lanes a
channel, whole sequences and segments of 128, 256 and 512 tokens. Each test says which form it means
and checks that the host's rule takes it. What lies behind the inputs' last rows is NaN, and what lies
behind y's has to stay.

The reference is the recurrence in float64, a token of every sequence at a time (tested against
oracle/layers.py). It carries along how far the state may be off: a step scales that by the decay and
adds (16 + 32) 2^-24 of the state's magnitudes, 16 for the step's own roundings (the step size is good
to 2^-21, and its product with A enters an exponential that is no larger than 1), 32 for the joins of
segments, whose decay comes from the sum of the steps of a segment; y adds the roundings of its N + 8
sums, the gate's (2^-20 of the result) and its own."""
import numpy as np
import pytest
import torch

from oracle import layers as ol

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16
DEV = "cuda"
PAST = 70          # rows behind the last one


def make(seed, lens, C, N, G, ti, ts):
    g = torch.Generator(DEV).manual_seed(seed)
    T, S = sum(lens), len(lens)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)                # noqa: E731

    def rows(*s):
        t = torch.full((T + PAST,) + s, float("nan"), dtype=ti, device=DEV)
        t[:T] = rnd(T, *s).to(ti)
        return t[:T]
    m = dict(T=T, S=S, C=C, N=N, G=G, ti=ti, ts=ts, lens=lens, x=rows(C), dt=rows(C), z=rows(C),
             B=rows(G, N), C_=rows(G, N))
    m["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(rnd(C, N) * 0.1)
    m["D"] = rnd(C)
    step = torch.exp(torch.rand(C, generator=g, device=DEV) * 4.6 - 6.9)
    m["bias"] = torch.log(torch.expm1(step))
    m["idx"] = torch.randperm(S + 2, generator=g, device=DEV)[:S].to(torch.int32)
    m["has"] = (torch.arange(S, device=DEV) % 2 == 0).to(torch.uint8)
    m["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    m["cache"] = (rnd(S + 2, C, N) * 0.2).to(ts)
    return m


def reference(m):
    """y and the cache as left, each with its tolerance."""
    f = {k: m[k].double() for k in ("x", "dt", "z", "A", "B", "C_", "D", "bias", "cache")}
    C, N, per, eps = m["C"], m["N"], m["C"] // m["G"], 2.0 ** -24
    dt = torch.logaddexp(f["dt"] + f["bias"], torch.zeros((), device=DEV, dtype=torch.float64))
    gate = f["z"] / (1 + torch.exp(-f["z"]))
    lens = torch.tensor(m["lens"], device=DEV)
    order = torch.argsort(lens, descending=True)
    by_len, start, slot = lens[order].tolist(), m["cu"].long()[:-1][order], m["idx"].long()[order]
    h = f["cache"][slot] * m["has"][order].bool()[:, None, None]
    mag, err = h.abs(), torch.zeros_like(h)
    y, ytol = torch.empty_like(f["x"]), torch.empty_like(f["x"])
    live = len(by_len)
    for t in range(by_len[0] if by_len else 0):
        while by_len[live - 1] <= t:
            live -= 1
        r = start[:live] + t
        wide = lambda v: v[r].repeat_interleave(per, 1)                      # noqa: E731
        da = torch.exp(dt[r][..., None] * f["A"])
        u = (dt[r] * f["x"][r])[..., None] * wide(f["B"])
        h[:live] = da * h[:live] + u
        mag[:live] = da * mag[:live] + u.abs()
        err[:live] = da * err[:live] + 48 * eps * mag[:live]
        c = wide(f["C_"])
        y[r] = ((h[:live] * c).sum(-1) + f["D"] * f["x"][r]) * gate[r]
        part = (mag[:live] * c.abs()).sum(-1) + (f["D"] * f["x"][r]).abs()
        ytol[r] = gate[r].abs() * ((err[:live] * c.abs()).sum(-1) + ((N + 8) * eps + 2.0 ** -20) * part)
    step = ol.STEP[m["ti"]]
    cache, ctol = f["cache"].clone(), torch.zeros_like(f["cache"])
    cache[slot] = h
    ctol[slot] = err + 16 * eps * mag + ol.STEP[m["ts"]] * h.abs() + (2.0 ** -25 if m["ts"] == F16 else 1e-30)
    return y, ytol + step * y.abs() + 1e-30, cache, ctol


def run(form, seed, lens, C, N, G, ti, ts):
    m = make(seed, lens, C, N, G, ti, ts)
    p = ssd.make_scan_problem(m["T"], m["S"], C, N, G, m["S"] + 2, ti, ts)
    assert ssd.selective_scan_varlen_kernel(p) == form
    assert (ssd.selective_scan_workspace_bytes(p) > 0) == ("segments" in form)
    y = torch.full((m["T"] + PAST, C), 7.0, dtype=ti, device=DEV)
    cache = m["cache"].clone()
    ssd.selective_scan_varlen(p, m["x"], m["dt"], m["A"], m["B"], m["C_"], m["D"], m["z"],
                              ssd.make_dt_transform(m["bias"], 0.0, 1e30), m["cu"], cache, m["idx"], m["has"],
                              y[:m["T"]], ssd.alloc_scan_workspace(p, DEV))
    want, ytol, left, ctol = reference(m)
    assert bool((y[m["T"]:] == 7.0).all())
    for got, ref, tol in ((y[:m["T"]], want, ytol), (cache, left, ctol)):
        good = (got.double() - ref).abs() <= tol              # (a NaN is not)
        assert bool(good.all()), (int((~good).sum()), good.numel())


def test_the_reference():
    m = make(1, [9, 0, 4, 30], 6, 16, 2, F32, F32)
    c = {k: (v.cpu() if isinstance(v, torch.Tensor) else v) for k, v in m.items()}
    want, _, left, *_ = ol.scan(c["x"], c["dt"], c["A"], c["B"], c["C_"], c["D"], c["z"], c["cu"], c["cache"],
                                c["idx"], c["has"], c["bias"], 0.0, 1e30)
    y, _, cache, _ = reference(m)
    assert np.allclose(y.cpu().numpy(), want, rtol=1e-11, atol=1e-12)
    assert np.allclose(cache.cpu().numpy(), left, rtol=1e-11, atol=1e-12)


# short ones end inside a kernel's stage: 3 tokens leave 29 or 61 of it past the sequence's end
@pytest.mark.parametrize("lens", [[3], [1, 3, 29, 2], [33, 0, 31, 5]])
@pytest.mark.parametrize("N", [16, 64])
def test_ends_inside_a_stage(lens, N):
    run("16 lanes", 2, lens, 40, N, 1, BF, F32)
    run("4 lanes", 3, lens * 40, 2048, N, 2, F32, BF)


MANY = [(11 * i * i) % 500 for i in range(20)]


@pytest.mark.parametrize("N,G,ti,ts", [(16, 2, BF, F32), (32, 1, F32, F32), (64, 2, BF, BF), (16, 1, F32, F16)])
def test_4_lanes(N, G, ti, ts):
    run("4 lanes", 4 + N, MANY, 2060, N, G, ti, ts)


@pytest.mark.parametrize("N,G,ti,ts", [(16, 2, BF, F32), (32, 4, BF, BF), (64, 2, BF, F16), (64, 1, F32, F32),
                                       (32, 1, F32, F32)])
@pytest.mark.parametrize("lens", [[2900], [1501, 1, 128, 2300]])
def test_4_lanes_in_segments_of_128(N, G, ti, ts, lens):
    run("4 lanes, segments of 128", 5 + N, lens, 1036, N, G, ti, ts)


@pytest.mark.parametrize("N,C,G", [(16, 1024, 1), (32, 516, 2), (64, 260, 1)])
def test_4_lanes_in_segments_of_256(N, C, G):
    run("4 lanes, segments of 256", 6 + N, [4000, 300, 3700], C, N, G, BF, F32)


@pytest.mark.parametrize("N,C,G", [(16, 512, 1), (64, 132, 2)])
def test_4_lanes_in_segments_of_512(N, C, G):
    run("4 lanes, segments of 512", 7 + N, [9000, 700, 22300 - 2 * N], C, N, G, BF, F32)


@pytest.mark.parametrize("N,G,ti,ts", [(16, 2, BF, BF), (32, 1, F32, F32), (64, 2, BF, F16)])
def test_16_lanes_in_segments_of_128(N, G, ti, ts):
    run("16 lanes, segments of 128", 8 + N, [1100, 0, 127, 129, 300, 1, 640, 128], 16, N, G, ti, ts)


@pytest.mark.parametrize("N,C", [(16, 64), (64, 16)])
def test_16_lanes_in_segments_of_256(N, C):
    run("16 lanes, segments of 256", 9 + N, [6000, 1, 7000, 257, 256, 4000, 3000, 3486], C, N, 1, BF, F32)


@pytest.mark.parametrize("N", [16, 32, 64])
def test_segments_of_more_than_64_sequences(N):
    lens = [(37 * i) % 460 + (900 if i == 69 else 0) for i in range(70)]
    run("16 lanes, segments of 128", 10 + N, lens, 16, N, 1, BF, F32)
    lens = [(37 * i) % 680 for i in range(100)]
    run("4 lanes, segments of 128", 11 + N, lens, {16: 64, 32: 40, 64: 16}[N], N, 1, BF, F32)


def test_segments_on_another_stream_and_in_a_graph():
    m = make(18, [1900, 3, 900], 1024, 16, 1, BF, F32)
    p = ssd.make_scan_problem(m["T"], 3, 1024, 16, 1, 5, BF, F32)
    assert ssd.selective_scan_varlen_kernel(p) == "4 lanes, segments of 128"
    tf = ssd.make_dt_transform(m["bias"], 0.0, 1e30)
    y, cache, ws = torch.empty_like(m["x"]), m["cache"].clone(), ssd.alloc_scan_workspace(p, DEV)
    call = lambda: ssd.selective_scan_varlen(                                # noqa: E731
        p, m["x"], m["dt"], m["A"], m["B"], m["C_"], m["D"], m["z"], tf, m["cu"], cache, m["idx"],
        m["has"], y, ws)
    call()
    want, left = y.clone(), cache.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y.zero_()
        cache.copy_(m["cache"])
        call()
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(cache, left)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        y.zero_()
        cache.copy_(m["cache"])
        ws.fill_(0xff)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(cache, left)

"""The channel-wise selective scan on the GPU against oracle/layers.py.

Tolerance per element: every step rounds the state's terms a few times in float32 and its decay
(whose exponent dt A is itself rounded, and whose step size comes out of softplus good to 2^-21);
none of it grows where the state decays, so a state t tokens on is off by at most
(16 t + 64) 2^-24 of its magnitudes, y by as much of its own; plus the rounding of what is stored.
"""
import numpy as np
import pytest
import torch

from oracle import layers as ol

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16
DEV = "cuda"


def make(seed, lens, C, N, G, ti, ts, slots=None, strided=False):
    g = torch.Generator().manual_seed(seed)
    T, S = sum(lens), len(lens)
    pad = 3 if strided else 0
    m = dict(T=T, S=S, C=C, N=N, G=G, ti=ti, ts=ts)
    for k in ("x", "dt", "z"):
        m[k] = torch.randn(T, C + pad, generator=g).to(ti)[:, pad:]
    bc = torch.randn(T, 2 * G * N + pad, generator=g).to(ti)[:, pad:]
    m["B"], m["C_"] = bc[:, :G * N].unflatten(1, (G, N)), bc[:, G * N:].unflatten(1, (G, N))
    m["A"] = -torch.arange(1, N + 1).float() * torch.exp(torch.randn(C, N, generator=g) * 0.1)
    m["D"] = torch.randn(C, generator=g)
    step = torch.exp(torch.rand(C, generator=g) * 4.6 - 6.9)
    m["bias"] = torch.log(torch.expm1(step))
    m["idx"] = torch.randperm(S + 2, generator=g)[:S].to(torch.int32) if slots is None else \
        torch.tensor(slots, dtype=torch.int32)
    m["has"] = (torch.arange(S) % 2).to(torch.uint8)
    m["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    m["cache"] = (torch.randn(S + 2, C, N, generator=g) * 0.2).to(ts)
    return m


def close(got, want, mag, n, dtype, what):
    got = got.detach().cpu().double().numpy()
    tol = (16 * n + 64) * 2.0 ** -24 * mag + ol.STEP[dtype] * np.abs(want)
    tol = tol + (2.0 ** -25 if dtype == F16 else 1e-30)      # (half precision's subnormal step)
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want).max()))


def dev(m):
    def move(t):       # keeps the row distance of a slice
        if not isinstance(t, torch.Tensor):
            return t
        if t.is_contiguous() or t.numel() == 0:
            return t.to(DEV)
        base = torch.empty(t.shape[0], t.stride(0), dtype=t.dtype, device=DEV)
        n = t[0].numel()
        v = base[:, base.shape[1] - n:].unflatten(1, t.shape[1:]) if t.dim() == 3 else \
            base[:, base.shape[1] - n:]
        v.copy_(t)
        return v
    return {k: move(v) for k, v in m.items()}


def run(m, lens, gate=True, skip=True, transform=True, has=True, clamp=(0.0, 1e30)):
    d = dev(m)
    p = ssd.make_scan_problem(m["T"], m["S"], m["C"], m["N"], m["G"], m["S"] + 2, m["ti"], m["ts"])
    tf = ssd.make_dt_transform(d["bias"], *clamp) if transform else None
    dt = d["dt"] if transform else (d["dt"].abs() * 0.1)
    y = torch.full((m["T"], m["C"]), 7.0, dtype=m["ti"], device=DEV)
    cache = d["cache"].clone()
    ssd.selective_scan_varlen(p, d["x"], dt, d["A"], d["B"], d["C_"], d["D"] if skip else None,
                              d["z"] if gate else None, tf, d["cu"], cache, d["idx"],
                              d["has"] if has else None, y, ssd.alloc_scan_workspace(p, DEV))
    want, _, left, ymag, _, cmag = ol.scan(
        m["x"], dt.cpu(), m["A"], m["B"], m["C_"], m["D"] if skip else None,
        m["z"] if gate else None, m["cu"], m["cache"], m["idx"], m["has"] if has else None,
        m["bias"] if transform else None, clamp[0] if transform else None, clamp[1])
    n = max(lens) if lens else 0
    close(y, want, ymag, n, m["ti"], "y")
    close(cache, left, cmag, n, m["ts"], "cache")
    untouched = sorted(set(range(m["S"] + 2)) - set(m["idx"].tolist()))
    assert torch.equal(cache[untouched].cpu(), m["cache"][untouched])


@pytest.mark.parametrize("ti,ts", [(F32, F32), (BF, F32), (BF, BF), (BF, F16), (F32, BF), (F32, F16)])
@pytest.mark.parametrize("N", [16, 32, 64])
@pytest.mark.parametrize("lens", [[1], [31, 0, 33, 64], [65, 3, 200]])
def test_prompts(ti, ts, N, lens):
    run(make(len(lens) + N, lens, 80, N, 1, ti, ts), lens)


@pytest.mark.parametrize("C,G", [(1, 1), (15, 3), (65, 1), (130, 2), (256, 4)])
def test_channels_and_groups(C, G):
    run(make(C, [40, 5], C, 16, G, BF, F32), [40, 5])


@pytest.mark.parametrize("kw", [dict(gate=False), dict(skip=False), dict(transform=False),
                                dict(has=False), dict(clamp=(0.02, 0.05))])
def test_options(kw):
    run(make(11, [50, 9], 48, 16, 1, BF, F32), [50, 9], **kw)


@pytest.mark.parametrize("N", [16, 32])
def test_rows_of_wider_projections(N):
    run(make(12, [50, 9], 48, N, 2, BF, F32, strided=True), [50, 9])


# one prompt over few channels, long enough to be cut into pieces that run side by side, and
# batches that mix such prompts with short ones
@pytest.mark.parametrize("lens,C", [([1030], 40), ([2500], 130), ([700, 1, 0, 513], 64)])
@pytest.mark.parametrize("ti,ts", [(F32, F32), (BF, F32)])
def test_long_prompts(lens, C, ti, ts):
    run(make(13, lens, C, 16, 1, ti, ts), lens)


@pytest.mark.parametrize("N,G", [(16, 1), (32, 2), (64, 1)])
@pytest.mark.parametrize("ti,ts", [(F32, F32), (BF, BF)])
def test_many_channels_and_sequences(N, G, ti, ts):
    # enough to fill the chip without segments, and with few lanes a channel
    lens = [3 + (7 * i) % 11 for i in range(40)] + [37]
    run(make(19, lens, 900, N, G, ti, ts), lens)


def test_many_sequences():
    lens = [(5 * i) % 9 for i in range(150)]
    run(make(14, lens, 20, 16, 1, BF, F32), lens)


def test_bad_slots_are_skipped():
    run(make(15, [40, 20, 33], 32, 16, 1, BF, F32, slots=[-1, 2, 5]), [40, 20, 33])


def test_softplus_ends():
    m = make(16, [8], 16, 16, 1, F32, F32)
    m["dt"] = torch.tensor([-200.0, -90.0, -30.0, -10.0, 0.0, 10.0, 30.0, 100.0])[:, None].expand(
        8, 16).contiguous()
    m["bias"] = torch.zeros(16)
    m["A"] = m["A"] * 1e-3
    run(m, [8])


@pytest.mark.parametrize("ti,ts", [(BF, BF), (F32, F32), (BF, F16)])
@pytest.mark.parametrize("R,T,C,N", [(1, 1, 80, 16), (3, 3, 65, 16), (5, 4, 64, 32), (2, 6, 48, 64),
                                     (70, 2, 16, 16)])
def test_update(ti, ts, R, T, C, N):
    m = make(R + T, [T] * R, C, N, 1, ti, ts)
    if R > 2:
        m["idx"][0] = -1
    d = dev(m)
    p = ssd.make_scan_problem(R * T, R, C, N, 1, R + 2, ti, ts)
    tf = ssd.make_dt_transform(d["bias"], 0.0, 1e30)
    one = torch.ones(R, dtype=torch.uint8)
    want, st, left, ymag, smag, cmag = ol.scan(m["x"], m["dt"], m["A"], m["B"], m["C_"], m["D"],
                                               m["z"], m["cu"], m["cache"], m["idx"], one,
                                               m["bias"], 0.0, 1e30)
    args = (p, d["x"], d["dt"], d["A"], d["B"], d["C_"], d["D"], d["z"], tf)
    y, cache = torch.empty_like(d["x"]), d["cache"].clone()
    ssd.selective_scan_update(*args, cache, d["idx"], y)
    close(y, want, ymag, T, ti, "y")
    close(cache, left, cmag, T, ts, "cache")
    y2, kept = torch.empty_like(y), d["cache"].clone()
    inter = torch.empty(R * T, C, N, dtype=ts, device=DEV)
    ssd.selective_scan_update(*args, kept, d["idx"], y2, inter)
    assert torch.equal(y, y2) and torch.equal(kept, d["cache"])
    close(inter, st, smag, T, ts, "states")
    if C % 16 == 0 and N == 16:      # rolled back with the framework's commit
        acc = torch.tensor([i % T for i in range(R)], dtype=torch.int32)
        up = ssd.make_ssu_problem(R, T, C // 16, 16, 16, 1, R + 2, BF, ts)
        ssd.ssd_state_commit(up, kept.view(R + 2, C // 16, 16, 16), d["idx"],
                             inter.view(R, T, C // 16, 16, 16), acc.to(DEV))
        for r in range(R):
            if int(m["idx"][r]) >= 0:
                assert torch.equal(kept[int(m["idx"][r])], inter[r * T + int(acc[r])])


def test_another_stream_and_a_graph():
    m = make(18, [300, 3, 90], 64, 16, 1, BF, F32)
    d = dev(m)
    p = ssd.make_scan_problem(m["T"], 3, 64, 16, 1, 5, BF, F32)
    tf = ssd.make_dt_transform(d["bias"], 0.0, 1e30)
    y, cache, ws = torch.empty_like(d["x"]), d["cache"].clone(), ssd.alloc_scan_workspace(p, DEV)
    call = lambda: ssd.selective_scan_varlen(                                # noqa: E731
        p, d["x"], d["dt"], d["A"], d["B"], d["C_"], d["D"], d["z"], tf, d["cu"], cache, d["idx"],
        d["has"], y, ws)
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

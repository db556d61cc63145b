"""The root-mean-square norm on the GPU against oracle/steps.py."""
import numpy as np
import pytest
import torch

from oracle import steps as os_
from oracle.layers import STEP

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DEV = "cuda"


def values(out, scale):
    v = out.cpu().double().numpy()
    b = scale.cpu().numpy().astype(np.float64)
    return (v.reshape(v.shape[0], -1, 32) * 2.0 ** (b - 127)[..., None]).reshape(v.shape), b


def check_out(out, scale, ref):
    want, _, tol = ref
    if out.dtype != E4:
        got = out.cpu().double().numpy()
        bad = ~(np.abs(got - want) <= tol + STEP[out.dtype] * np.abs(want))
        assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want))))
        return
    got, b = values(out, scale)
    # half a step of 3 bits behind the leading one, of the smallest exponent's below that
    unit = np.repeat(2.0 ** (b - 127), 32, -1)
    assert np.all(np.abs(got - want) <= tol * (1 + 2.0 ** -4) + np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * unit))
    # the least power of two that holds the largest, which is known to `tol`
    top = np.abs(want).reshape(b.shape + (32,)).max(-1)
    off = tol.reshape(b.shape + (32,)).max(-1)
    s = 2.0 ** (b - 127)
    assert np.all(top - off <= 448 * s) and np.all((top + off > 224 * s) | (b == 1))


def run(x, out_dtype, weight=None, residual=None, gate=None, groups=1, eps=1e-5, keep=True, inplace=False):
    rows, h = x.shape
    dev = lambda t: None if t is None else t.to(DEV)                            # noqa: E731
    p = ssd.make_norm_problem(rows, h, x.dtype, out_dtype, groups,
                              residual.dtype if residual is not None else None, eps)
    out = torch.full((rows, h), 7.0, device=DEV).to(out_dtype)
    scale = torch.full((rows, h // 32), 9, dtype=torch.uint8, device=DEV) if out_dtype == E4 else None
    r = dev(residual)
    kept = None if residual is None or not keep else (r if inplace else torch.full_like(r, 7.0))
    ssd.rms_norm(p, dev(x), dev(weight), out, r, kept, dev(gate), scale)
    ref = os_.rms_norm(x, weight, residual, gate, groups, eps)
    check_out(out, scale, ref)
    if kept is not None:
        want = ref[1]
        assert np.all(np.abs(kept.cpu().double().numpy() - want) <= (STEP[r.dtype] + 2.0 ** -24) * np.abs(want) + 1e-38)
    elif residual is not None:
        assert torch.equal(r.cpu(), residual)
    return out, scale, kept


def data(seed, rows, h, ti=BF):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, t=ti: torch.randn(*s, generator=g).to(t)                     # noqa: E731
    return n, n(rows, h)


@pytest.mark.parametrize("ti", [BF, F32])
@pytest.mark.parametrize("to", [BF, F32, E4])
@pytest.mark.parametrize("mode", ["plain", "add_bf16", "add_f32", "gate"])
@pytest.mark.parametrize("rows,h,groups", [(1, 32, 1), (3, 256, 1), (5, 2560, 1), (2, 1024, 4), (7, 96, 3)])
def test_norm(ti, to, mode, rows, h, groups):
    n, x = data(h + rows, rows, h, ti)
    kw = {}
    if mode.startswith("add"):
        kw["residual"] = n(rows, h, t=BF if mode == "add_bf16" else F32) * 3
    elif mode == "gate":
        kw["gate"] = n(rows, h) * 4
    run(x, to, n(h, t=F32), groups=groups, **kw)


@pytest.mark.parametrize("h", [1, 2, 7, 31, 33, 63, 65, 100, 1001, 8190])
@pytest.mark.parametrize("ti,to", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_odd_sizes(h, ti, to):
    n, x = data(h, 3, h, ti)
    run(x, to, n(h, t=F32), residual=n(3, h, t=F32))
    run(x, to, None, gate=n(3, h))


@pytest.mark.parametrize("to", [BF, E4])
@pytest.mark.parametrize("h", [8192, 8224, 16384, 16416, 32768, 33024])
def test_long_rows(h, to):
    """One, two and four vectors a thread, and past them."""
    n, x = data(h, 2, h)
    run(x, to, n(h, t=F32), residual=n(2, h, t=F32))
    run(x, to, n(h, t=F32), residual=n(2, h, t=F32), groups=2 if h % 64 == 0 else 1, keep=False)


@pytest.mark.parametrize("to", [BF, E4])
def test_many_rows_and_groups(to):
    n, x = data(5, 1000, 512)
    run(x, to, n(512, t=F32), groups=8)
    run(x, to, n(512, t=F32), residual=n(1000, 512))


@pytest.mark.parametrize("to", [BF, F32, E4])
@pytest.mark.parametrize("h", [64, 2560, 33024])
def test_in_place_sum(h, to):
    n, x = data(h, 4, h)
    run(x, to, n(h, t=F32), residual=n(4, h, t=F32), inplace=True)
    run(x, to, n(h, t=F32), residual=n(4, h), inplace=True)


@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("to", [BF, E4, F32])
def test_strides_and_alignment(shift, to):
    """Slices of wider rows, on and off 16 bytes; what lies between them is left as it was."""
    n, _ = data(shift, 1, 1)
    rows, h = 5, 192
    wide = n(rows, 3 * h).to(DEV)
    x, gate = wide[:, shift:shift + h], wide[:, shift + h:shift + 2 * h]
    ob = torch.full((rows, 2 * h), 7.0, device=DEV).to(to)
    out = ob[:, shift:shift + h]
    scale = torch.zeros(rows, h // 32, dtype=torch.uint8, device=DEV) if to == E4 else None
    w = n(h + 1, t=F32).to(DEV)
    w = w[1:] if shift == 1 else w[:h]
    ssd.rms_norm(ssd.make_norm_problem(rows, h, BF, to), x, w, out, gate=gate, out_scale=scale)
    check_out(out, scale, os_.rms_norm(x.cpu(), w.cpu(), gate=gate.cpu()))
    rest = ob.float().cpu()
    rest[:, shift:shift + h] = 7.0
    assert bool((rest == 7.0).all())
    # residual and sum as slices
    res = n(rows, 2 * h, t=F32).to(DEV)
    r, keep = res[:, shift:shift + h], torch.full((rows, 2 * h), 7.0, device=DEV)
    k = keep[:, shift:shift + h]
    ssd.rms_norm(ssd.make_norm_problem(rows, h, BF, to, residual_dtype=F32), x, w, out, r, k, out_scale=scale)
    ref = os_.rms_norm(x.cpu(), w.cpu(), residual=r.cpu())
    check_out(out, scale, ref)
    assert np.all(np.abs(k.cpu().double().numpy() - ref[1]) <= 2.0 ** -23 * np.abs(ref[1]))
    keep[:, shift:shift + h] = 7.0
    assert bool((keep == 7.0).all())


def test_zeros_and_magnitudes():
    x = torch.zeros(4, 64)
    x[1] = 1e-20
    x[2] = 1e15
    x[3, 5] = 1.0
    for to in (BF, F32, E4):
        run(x, to)
    out, scale, _ = run(torch.zeros(2, 64), E4)
    assert bool((scale == 1).all()) and bool((out.view(torch.uint8) == 0).all())
    run(torch.full((1, 64), 2.0), E4, torch.cat([torch.full((32,), 448.0), torch.full((32,), 460.0)]), eps=0.0)


def test_non_finite():
    """A NaN or an infinity makes its own group NaN where it stands, and no other row or group."""
    n, x = data(3, 4, 128)
    x[1, 3], x[2, 100] = float("nan"), float("inf")
    for to in (BF, F32, E4):
        out = torch.empty(4, 128, device=DEV).to(to)
        scale = torch.empty(4, 4, dtype=torch.uint8, device=DEV) if to == E4 else None
        ssd.rms_norm(ssd.make_norm_problem(4, 128, BF, to, 2), x.to(DEV), None, out, out_scale=scale)
        got = out.float().cpu()
        assert bool(torch.isnan(got[1, :64]).all()) and bool(torch.isfinite(got[1, 64:]).all())
        assert bool(torch.isnan(got[2, 100])) and bool((got[2, 64:100] == 0).all())
        assert bool(torch.isfinite(got[2, :64]).all()) and bool(torch.isfinite(got[[0, 3]]).all())
    # in 8 bits a NaN of the weights does not enter its block's scale
    w = torch.ones(64)
    w[3], w[40] = float("nan"), float("inf")
    out, scale = torch.empty(1, 64, device=DEV).to(E4), torch.empty(1, 2, dtype=torch.uint8, device=DEV)
    ssd.rms_norm(ssd.make_norm_problem(1, 64, F32, E4, eps=0.0), torch.ones(1, 64, device=DEV), w.to(DEV), out,
                 out_scale=scale)
    got, b = values(out, scale)
    assert np.array_equal(np.flatnonzero(np.isnan(got[0])), [3, 40]) and np.array_equal(b, [[119, 119]])
    assert np.nanmin(got) == np.nanmax(got) == 1


def test_rows_past_4gb():
    rows, h = 33000, 32768
    x = torch.zeros(rows, h, dtype=F32, device=DEV)         # 4.3 GB
    out = torch.empty(rows, h, dtype=BF, device=DEV)
    n, a = data(1, 2, h, F32)
    x[-1], x[20000] = a[0].to(DEV), a[1].to(DEV)
    ssd.rms_norm(ssd.make_norm_problem(rows, h, F32, BF), x, None, out)
    ref = os_.rms_norm(a)
    check_out(out[[rows - 1, 20000]], None, ref)
    assert bool((out[:100] == 0).all()) and bool((out[-100:-1] == 0).all())


def test_no_rows_another_stream_and_a_graph():
    p = ssd.make_norm_problem(0, 64, BF, BF)
    ssd.rms_norm(p, torch.empty(0, 64, dtype=BF, device=DEV), None, torch.empty(0, 64, dtype=BF, device=DEV))
    n, x = data(9, 64, 2560)
    xd, r, w = x.to(DEV), n(64, 2560, t=F32).to(DEV), n(2560, t=F32).to(DEV)
    out, sc, keep = (torch.empty(64, 2560, device=DEV).to(E4), torch.empty(64, 80, dtype=torch.uint8, device=DEV),
                     torch.empty_like(r))
    p = ssd.make_norm_problem(64, 2560, BF, E4, residual_dtype=F32)
    go = lambda: ssd.rms_norm(p, xd, w, out, r, keep, out_scale=sc)             # noqa: E731
    go()
    want = [t.clone() for t in (out.view(torch.uint8), sc, keep)]

    def same():
        assert all(torch.equal(a, b) for a, b in zip((out.view(torch.uint8), sc, keep), want))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.view(torch.uint8).zero_()
        go()
    side.synchronize()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        out.view(torch.uint8).zero_()
        keep.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same()

"""The channel-wise scan on the GPU against oracle/layers.py where its inputs are not finite."""
import numpy as np
import pytest
import torch

from oracle import layers as ol
from test_gpu_scan import dev, make

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
F32 = torch.float32
DEV = "cuda"


def same(got, want, mag, n, dtype, what):
    """Within the scan tests' tolerance where the definition gives numbers (and a number there),
    NaN where it gives NaN."""
    got, nan = got.detach().cpu().double().numpy(), np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), (what, int(np.isnan(got).sum()), int(nan.sum()))
    tol = (16 * n + 64) * 2.0 ** -24 * mag + ol.STEP[dtype] * np.abs(want) + 1e-30
    assert np.all((np.abs(got - want) <= tol)[~nan]), what


# few channels; many of them (4 lanes a channel); one sequence cut into pieces
@pytest.mark.parametrize("lens,C,N", [([40, 1, 33], 48, 16), ([3 + i % 9 for i in range(40)], 900, 32),
                                      ([1030], 40, 16)])
@pytest.mark.parametrize("clamp", [(0.0, 1e30), (0.02, 0.05)])
def test_scan_of_a_nan_step(lens, C, N, clamp):
    """A step size that is NaN leaves its channel's state NaN, whatever the bounds."""
    m = make(21, lens, C, N, 1, F32, F32)
    m["dt"][m["T"] // 2, 3] = float("nan")
    m["dt"][0, C - 1] = float("nan")
    d = dev(m)
    p = ssd.make_scan_problem(m["T"], m["S"], C, N, 1, m["S"] + 2, F32, F32)
    tf = ssd.make_dt_transform(d["bias"], *clamp)
    y, cache = torch.full((m["T"], C), 7.0, device=DEV), d["cache"].clone()
    ssd.selective_scan_varlen(p, d["x"], d["dt"], d["A"], d["B"], d["C_"], d["D"], d["z"], tf, d["cu"],
                              cache, d["idx"], d["has"], y, ssd.alloc_scan_workspace(p, DEV))
    want, _, left, ymag, _, cmag = ol.scan(m["x"], m["dt"], m["A"], m["B"], m["C_"], m["D"], m["z"],
                                           m["cu"], m["cache"], m["idx"], m["has"], m["bias"], *clamp)
    assert np.isnan(want).any() and np.isnan(left).any()
    same(y, want, ymag, max(lens), F32, "y")
    same(cache, left, cmag, max(lens), F32, "cache")


@pytest.mark.parametrize("R,T", [(3, 1), (2, 3), (2, 6)])
def test_scan_update_of_a_nan_step(R, T):
    m = make(22, [T] * R, 48, 16, 1, F32, F32)
    m["dt"][T - 1, 3] = float("nan")
    d = dev(m)
    p = ssd.make_scan_problem(R * T, R, 48, 16, 1, R + 2, F32, F32)
    tf = ssd.make_dt_transform(d["bias"], 0.01, 0.05)
    y, inter = torch.empty_like(d["x"]), torch.empty(R * T, 48, 16, device=DEV)
    ssd.selective_scan_update(p, d["x"], d["dt"], d["A"], d["B"], d["C_"], d["D"], d["z"], tf,
                              d["cache"].clone(), d["idx"], y, inter)
    want, st, _, ymag, smag, _ = ol.scan(m["x"], m["dt"], m["A"], m["B"], m["C_"], m["D"], m["z"], m["cu"],
                                         m["cache"], m["idx"], torch.ones(R, dtype=torch.uint8), m["bias"],
                                         0.01, 0.05)
    assert np.isnan(want).any()
    same(y, want, ymag, T, F32, "y")
    same(inter, st, smag, T, F32, "states")


@pytest.mark.parametrize("lens,C,N", [([40, 1, 33, 64], 48, 16), ([3 + i % 9 for i in range(40)], 900, 32),
                                      ([1030], 40, 16), ([256], 40, 16)])
def test_scan_of_states_that_decay_at_once(lens, C, N):
    """A = -infinity: the state holds its last token alone, also where a sequence ends inside the
    kernel's stage of tokens."""
    m = make(23, lens, C, N, 1, F32, F32)
    m["A"][5], m["A"][:, 2] = -float("inf"), -float("inf")
    d = dev(m)
    p = ssd.make_scan_problem(m["T"], m["S"], C, N, 1, m["S"] + 2, F32, F32)
    tf = ssd.make_dt_transform(d["bias"], 0.0, 1e30)
    y, cache = torch.full((m["T"], C), 7.0, device=DEV), d["cache"].clone()
    ssd.selective_scan_varlen(p, d["x"], d["dt"], d["A"], d["B"], d["C_"], d["D"], d["z"], tf, d["cu"],
                              cache, d["idx"], d["has"], y, ssd.alloc_scan_workspace(p, DEV))
    want, _, left, ymag, _, cmag = ol.scan(m["x"], m["dt"], m["A"], m["B"], m["C_"], m["D"], m["z"],
                                           m["cu"], m["cache"], m["idx"], m["has"], m["bias"], 0.0, 1e30)
    same(y, want, ymag, max(lens), F32, "y")
    same(cache, left, cmag, max(lens), F32, "cache")

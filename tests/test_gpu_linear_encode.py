"""Codes and scales of weights at the upper end of float32, and the product with them."""
import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.mark.parametrize("dt", [BF, F32])
def test_largest_weights_stay_finite(dt):
    tops = [1.25 * 2.0 ** 127, 1.5 * 2.0 ** 127, 1.5 * 2.0 ** 127 * (1 + 2.0 ** -7), 3e38, torch.finfo(dt).max]
    g = torch.Generator().manual_seed(1)
    w = (torch.rand(2 * len(tops), 32, generator=g) - 0.5) * 2.0 ** 127
    for i, t in enumerate(tops):
        w[2 * i, 3], w[2 * i + 1, 30] = t, -t
    w = w.to(dt)
    n = w.shape[0]
    p = ssd.make_linear_problem(1, 32, n, BF, F32)
    held = ssd.alloc_linear_weights(p, DEV)
    ssd.linear_w4_encode(p, w.to(DEV), **held)
    got = os_.weights(held["weight"], held["weight_scale"])
    for i in range(n):
        want, byte = os_.encode_weights(w[i].double().numpy())
        assert int(held["weight_scale"][i, 0]) == byte <= 252, i
        assert np.array_equal(got[i], want), i
    x = torch.zeros(2, 32, dtype=BF)
    x[0, 3], x[1, 30] = 0.5, 0.25
    p = ssd.make_linear_problem(2, 32, n, BF, F32)
    out = torch.empty(2, n, device=DEV)
    ssd.linear_w4(p, x.to(DEV), held["weight"], held["weight_scale"], out)
    assert np.array_equal(out.cpu().double().numpy(), x.double().numpy() @ got.T)

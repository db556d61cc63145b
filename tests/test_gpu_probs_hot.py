"""Token probabilities at temperatures where logits count whose difference is past the largest float."""
import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
INF = float("inf")


@pytest.mark.parametrize("ti", [BF, F32])
@pytest.mark.parametrize("V", [5, 3000, 9000, 40000])
def test_differences_past_the_largest_float(V, ti):
    temp = [1e30, 1e36, 1e37, 1e38, 3e38, INF, 0.0]
    g = torch.Generator().manual_seed(V)
    x = (torch.rand(len(temp), 2, V, generator=g) * 2 - 1) * 3.3e38
    x[:, :, 0], x[:, :, V - 1], x[:, :, V // 2] = 3.3e38, -3.3e38, 1.0
    x[:, 1, 1::3] = -INF
    x = x.to(ti)
    p = ssd.make_probs_problem(len(temp), 2, V, ti)
    out = torch.full(x.shape, 7.0, device=DEV)
    ssd.token_probs(p, x.to(DEV), torch.tensor(temp, device=DEV), out, ssd.alloc_probs_workspace(p, DEV))
    want, tol = os_.probs(x, np.float32(temp).astype(np.float64))
    bad = ~(np.abs(out.cpu().double().numpy() - want) <= tol)
    assert not bad.any(), np.argwhere(bad)[:4]

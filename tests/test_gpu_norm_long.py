"""The norm of groups far longer than a block, whose sum is a long chain."""
import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.mark.parametrize("n", [2 ** 20, 2 ** 24, 2 ** 26 + 32])
@pytest.mark.parametrize("v", [0.7, 1.1, 1.3])
def test_equal_elements(n, v):
    """Equal elements come out as one. Their squares' sum is off by what oracle/steps.py counts, and a
    result of one by no rounding of its own that this does not count: 8 roundings of 2^-24 behind the sum."""
    x = torch.full((1, n), v, device=DEV)
    out = torch.empty_like(x)
    ssd.rms_norm(ssd.make_norm_problem(1, n, F32, F32, eps=0.0), x, None, out)
    assert float((out - 1).abs().max()) <= ((32 + 1 + 6 + 16) / 2 + 8) * 2.0 ** -24


@pytest.mark.parametrize("mode", ["plain", "add", "gate"])
def test_long_rows_against_the_reference(mode):
    rows, h = 2, 3 * 2 ** 20 + 5
    g = torch.Generator().manual_seed(7)
    x = (torch.rand(rows, h, generator=g) + 0.5).to(BF)
    other = None if mode == "plain" else torch.rand(rows, h, generator=g).to(BF)
    kw = {} if mode == "plain" else {"residual" if mode == "add" else "gate": other}
    out = torch.empty(rows, h, device=DEV)
    p = ssd.make_norm_problem(rows, h, BF, F32, residual_dtype=BF)
    ssd.rms_norm(p, x.to(DEV), None, out, **{k: t.to(DEV) for k, t in kw.items()})
    want, _, tol = os_.rms_norm(x, None, **kw)
    got = out.cpu().double().numpy()
    assert np.all(np.abs(got - want) <= tol + 2.0 ** -24 * np.abs(want))

"""The verification at the length where one launch gives way to two."""
import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
I32 = torch.int32
DEV = "cuda"


@pytest.mark.parametrize("R", [1, 6])
@pytest.mark.parametrize("V", [11000, 12287, 12288, 12289, 16000])
def test_both_forms(V, R):
    T = 3
    p = ssd.make_verify_problem(R, T, V)
    assert (ssd.verify_drafts_workspace_bytes(p) == 0) == (V <= 12288)
    g = torch.Generator().manual_seed(V)
    x = torch.randn(R, T, V, generator=g) * 2
    target = torch.softmax(x, -1)
    draft = torch.softmax(x[:, :T - 1] + torch.randn(R, T - 1, V, generator=g), -1).contiguous()
    d = torch.multinomial(draft.flatten(0, 1), 1, generator=g).view(R, T - 1).to(I32)
    u = torch.rand(R, T, generator=g)
    for q in (draft, None):
        acc, tok = (torch.full(s, -9, dtype=I32, device=DEV) for s in ((R,), (R, T)))
        ssd.verify_drafts(p, target.to(DEV), None if q is None else q.to(DEV), d.to(DEV), None, u.to(DEV), acc, tok,
                          ssd.alloc_verify_workspace(p, DEV))
        wa, wt = os_.verify(target, q, d, None, u)
        assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)

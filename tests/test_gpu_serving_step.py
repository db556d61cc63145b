"""The norm, the 4-bit products, the token probabilities and the verification together, as
examples/hybrid_stack.py answers with them behind its layers."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
pytest.importorskip("state_space_model_varlen_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location(
        "hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("lens,tokens", [((70, 1, 133), 3), ((300, 17), 1), ((2, 64, 65, 200), 4)])
def test_parts_and_verify_steps_give_the_whole(lens, tokens):
    """Both ways round the same values, but not in the same order of sums. Where they differ by d
    relative (2^-9 for each of about six bfloat16 roundings a layer, added as independent errors:
    d = 2^-9 sqrt(6) = 5e-3), rounding to 8 bits with steps of about 2^-3.5 of a value takes a share
    d / 2^-3.5 of them to the other side, by a step each: sqrt(d 2^-3.5) = 2e-2 of the row's size.
    Three such roundings, and as much again for the gated norm's and the cache's: 2e-2 sqrt(6) = 5e-2; a
    wrong state, row or scale is of the result's own size."""
    for e in load().check(256, lens, 3, tokens, four_bit=True):
        assert e < 5e-2


@pytest.mark.parametrize("drafts", [0, 1, 3])
@pytest.mark.parametrize("four_bit", [False, True])
def test_answers(drafts, four_bit):
    """Every step's decision is the reference's on the probabilities that it saw, greedy requests get
    the largest logit's token, and the slots hold what was accepted."""
    m = load()
    R, V = 3, 500
    st = m.Stack(256, R, 400, seed=1, four_bit=four_bit, vocab=V)
    g = torch.Generator("cuda").manual_seed(2)
    lens = [40, 1, 77]
    prompt = torch.randint(0, V, (sum(lens),), generator=g, device="cuda")
    st.prompt(st.emb[prompt], [2, 0, 1], lens)
    slots = [2, 0, 1]
    temp = torch.tensor([1.0, 0.0, 0.7], device="cuda")
    last = torch.randint(0, V, (R,), generator=g, device="cuda").to(torch.int32)
    held = list(lens)
    for _ in range(4):
        got, (target, draft, tokens, uniform, acc, out) = st.speculate(last, slots, drafts, temp, g)
        wa, wt = os_.verify(target.cpu(), None if draft is None else draft.cpu(),
                            None if tokens is None else tokens.cpu(), None, uniform.cpu())
        assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(out.cpu().numpy(), wt)
        assert float((target.sum(-1) - 1).abs().max()) < 1e-4
        for r in range(R):
            assert len(got[r]) == int(wa[r]) + 1 and all(0 <= t < V for t in got[r])
            held[r] += len(got[r])
            assert int(st.lens[slots[r]]) == held[r]
        # temperature 0: one at the largest, so accepted or corrected to it
        best = target[1].argmax(-1).tolist()
        assert got[1] == best[:len(got[1])]
        last = torch.tensor([t[-1] for t in got], dtype=torch.int32, device="cuda")

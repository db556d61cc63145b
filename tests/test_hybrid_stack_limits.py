"""examples/hybrid_stack.py turns down more tokens than a sequence has pages for on the host, before
an index past its table reaches the GPU (no GPU needed)."""
import importlib.util
import os

import pytest
import torch

pytest.importorskip("state_space_model_varlen_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def stack(tokens):
    spec = importlib.util.spec_from_file_location(
        "hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    st = m.Stack.__new__(m.Stack)                # its table of pages alone
    st.dev, st.pages_per_seq = torch.device("cpu"), -(-tokens // st.PAGE)
    st.pages = torch.arange(2 * st.pages_per_seq, dtype=torch.int32).view(2, -1)
    st.lens = torch.zeros(2, dtype=torch.int64)
    return st


def test_positions_up_to_the_last_page():
    st = stack(130)                              # 3 pages of 64
    st.lens[1] = 190
    got = st._positions([0, 1], [192, 2])
    assert got.tolist() == list(range(192)) + [192 + 190, 192 + 191]


@pytest.mark.parametrize("held,counts", [((0, 0), [193, 1]), ((0, 190), [1, 3]), ((192, 0), [1, 1])])
def test_too_many_tokens_are_refused(held, counts):
    st = stack(130)
    st.lens[:] = torch.tensor(held)
    with pytest.raises(ValueError, match="192"):
        st.prompt(None, [0, 1], counts)
    if held != (0, 0):
        with pytest.raises(ValueError, match="192"):
            st.verify(None, [0, 1], 3)
    assert st.lens.tolist() == list(held)

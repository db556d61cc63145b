"""The operators together, as examples/hybrid_stack.py serves a hybrid stack with them."""
import importlib.util
import os

import pytest

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
    """Both ways round the same values to bf16 at the same places (activations, the cache's 8-bit
    rows), but not in the same order of sums, so single values land on the other side of a rounding:
    half a step of 2^-8 for each of the two dozen roundings a token passes, added as independent
    errors, is 2^-8 sqrt(24) = 2e-2; a wrong state or cache row is of the result's own size."""
    for e in load().check(256, lens, 3, tokens):
        assert e < 2e-2

"""Choices of the 4-bit products that are checked on the host (no GPU needed)."""
import ctypes

import pytest
import torch

ssd = pytest.importorskip("state_space_model_varlen_amd")
LIB = ssd._lib
OK = ctypes.c_void_p(256)
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
UNSUP = 4


def test_products_are_cut_by_choice_alone():
    assert ssd.make_linear_problem(1, 32, 1, E4, BF).cut_products == 0
    assert ssd.make_linear_problem(1, 32, 1, E4, BF, cut_products=True).cut_products == 1
    for bad in (2, -1):
        p = ssd.make_linear_problem(8, 64, 48, E4, BF)
        p.cut_products = bad
        assert LIB.linear_w4(ctypes.byref(p), *[OK] * 7, 0, None) == UNSUP
        assert ssd.linear_w4_kernel(p) == ""


@pytest.mark.parametrize("xt", [BF, E4])
def test_no_workspace_is_needed_or_looked_at(xt):
    """Every problem's is empty, and what is passed for one decides nothing: a call goes on to what is wrong."""
    for t in (1, 16, 64, 300, 4096):
        for k in (64, 1024, 8192):
            p = ssd.make_linear_problem(t, k, 2560, xt, BF)
            assert ssd.linear_w4_workspace_bytes(p) == 0 and ssd.linear_w4_kernel(p) != ""
            assert ssd.alloc_linear_workspace(p, "cpu") is None
            for ws in (None, OK, ctypes.c_void_p(257)):
                args = [OK, OK, OK, OK, None, None, ws]               # no result
                assert LIB.linear_w4(ctypes.byref(p), *args, ctypes.c_size_t(0), None) == 1

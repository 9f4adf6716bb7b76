"""Refusals and sizes at the edges of the training and expert calls (no GPU):
nothing below launches."""
import ctypes

import pytest
import torch

from combine_fp32_router_amd import binding as B

OK, NULL, SHAPE, ALIGN, WORKSPACE, HIP, ALIAS = range(7)
F = ctypes.c_void_p(0x10000)  # aligned, never dereferenced
G = ctypes.c_void_p(0x20000)
H = ctypes.c_void_p(0x30000)


@pytest.fixture(scope="module")
def lib():
    return B.load()


def test_the_flag_of_masked_gates_is_no_size(lib):
    flag = B.MOE_ROUTE_MASKED_GATES
    f = lambda k, T=10: lib.moe_route_grad(F, F, F, F, None, F, F, F, T, 5, 8, k, None, None)  # noqa: E731
    assert f(2) == NULL and f(2 | flag) == NULL  # no output: past the sizes
    for k in (9, 0, -1, 2 | flag << 1):
        assert f(k) == SHAPE and f(k | flag) == SHAPE
    assert f(2 | flag, T=0) == OK
    assert lib.moe_balance_loss(None, None, None, 10, 5, 8, 2 | flag, None, None, None, None, None,
                                ctypes.byref(ctypes.c_size_t(0)), None) == SHAPE

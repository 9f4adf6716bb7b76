"""Refusals of the experts and of a group that runs them, on the host."""
import pytest
import torch

from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd.epgroup import EPGroup
from combine_fp32_router_amd.experts import ExpertMLP


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def mlp(act=B.MOE_ACT_SILU, E=4, H=32, I=16, max_rows=64, **kw):
    wide = 2 if act == B.MOE_ACT_SWIGLU else 1
    return ExpertMLP(bf16(E, wide * I, H), bf16(E, H, I), act, max_rows=max_rows, **kw)


def test_buffers_follow_the_activation():
    m = mlp(B.MOE_ACT_SWIGLU, train=True)
    assert m.hidden.shape == (64, 16) and m.preact.shape == (64, 32) == m.d_preact.shape
    assert mlp().preact is None
    g = mlp(train=True, b_up=torch.zeros(4, 16)).alloc_grads(torch.bfloat16)
    assert g.w_up.dtype == torch.bfloat16 and g.b_up.dtype == torch.float32 and g.b_down is None


@pytest.mark.parametrize("up,down,act,kw", [
    ((4, 16, 32), (4, 32, 32), B.MOE_ACT_SILU, {}),
    ((4, 16, 32), (4, 32, 16), B.MOE_ACT_SWIGLU, {}),
    ((3, 16, 32), (4, 32, 16), B.MOE_ACT_SILU, {}),
    ((4, 16), (4, 32, 16), B.MOE_ACT_SILU, {}),
    ((4, 16, 32), (4, 32, 16), B.MOE_ACT_SILU, {"b_up": torch.zeros(4, 32)}),
    ((4, 16, 32), (4, 32, 16), B.MOE_ACT_SILU, {"b_down": torch.zeros(4, 32, dtype=torch.float64)})])
def test_shapes_that_do_not_fit(up, down, act, kw):
    with pytest.raises(ValueError):
        ExpertMLP(bf16(*up), bf16(*down), act, max_rows=8, **kw)


def test_rows_that_do_not_fit():
    m, off = mlp(train=True), torch.zeros(5, dtype=torch.int32)
    for n, h in ((65, 32), (8, 16)):
        with pytest.raises(ValueError):
            m.forward(bf16(n, h), off, bf16(n, h))
        with pytest.raises(ValueError):
            m.backward(bf16(n, h), bf16(n, h), off, None, None)
    with pytest.raises(ValueError, match="train"):
        mlp().backward(bf16(8, 32), bf16(8, 32), off, None, None)


def test_host_tensors_are_refused():
    m, off = mlp(), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        m.forward(bf16(8, 32), off, bf16(8, 32))


def test_groups_that_the_experts_do_not_fit():
    for kw in ({"E": 8}, {"H": 64}, {"max_rows": 31}):
        with pytest.raises(ValueError):
            EPGroup(16, 32, 4, 2, 2, device="cpu", experts=mlp(**kw))


def test_backward_needs_a_run_to_go_back_through():
    x, z = bf16(16, 32), torch.zeros(16, 4)
    for grp in (EPGroup(16, 32, 4, 2, 2, device="cpu"),
                EPGroup(16, 32, 4, 2, 2, device="cpu", experts=mlp()),
                EPGroup(16, 32, 4, 2, 2, device="cpu", experts=mlp(train=True))):
        with pytest.raises(ValueError, match="backward"):
            grp.backward(x, None, z)
    grp._last = (z, 0, None, None)
    with pytest.raises(ValueError, match="Balance"):
        grp.backward(x, None, z, d_loss=torch.ones(1))
    with pytest.raises(ValueError, match="d_x"):
        grp.backward(x, bf16(8, 32), z)

"""Refusals and buffers of the experts in E4M3 codes, and the formulas of their
gradients against differences, on the host."""
import pytest
import torch

import fp8_ref as F
from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd.epgroup import EPGroup
from combine_fp32_router_amd.experts import ExpertMLP8


def bf16(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def mlp(act=B.MOE_ACT_SILU, E=4, H=144, I=272, max_rows=64, **kw):
    wide = 2 if act == B.MOE_ACT_SWIGLU else 1
    return ExpertMLP8(bf16(E, wide * I, H), bf16(E, H, I), act, max_rows=max_rows, **kw)


def test_buffers_follow_the_activation():
    m = mlp(B.MOE_ACT_SWIGLU, train=True)
    assert m.up8[0].shape == (4, 544, 144) and m.up8[1].shape == (4, 2, 3, 2)
    assert m.up8_t[0].shape == (4, 144, 544) and m.up8_t[1].shape == (4, 2, 2, 3)
    assert m.d_preact8[1].shape == (64, 2, 3) and m.hidden.shape == (64, 272)
    m = mlp()
    assert m.hidden is None and m.d_preact8 is None and m.up8_t == (None, None)
    assert m.hidden8[0].dtype == torch.float8_e4m3fn and m.hidden8[1].shape == (64, 3)


def test_rows_that_do_not_fit():
    m, off = mlp(train=True), torch.zeros(5, dtype=torch.int32)
    for n, h in ((65, 144), (8, 16)):
        with pytest.raises(ValueError):
            m.forward(bf16(n, h), off, bf16(n, h))
        with pytest.raises(ValueError):
            m.backward(bf16(n, h), bf16(n, h), off, None, None)
    with pytest.raises(ValueError, match="out"):
        m.forward(bf16(8, 144), off, bf16(7, 144))
    with pytest.raises(ValueError, match="before"):
        m.backward(bf16(8, 144), bf16(8, 144), off, None, None)
    with pytest.raises(ValueError, match="train"):
        mlp().backward(bf16(8, 144), bf16(8, 144), off, None, None)


def test_codes_need_their_scales():
    m, off = mlp(), torch.zeros(5, dtype=torch.int32)
    codes = torch.zeros(8, 144, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        m.forward(codes, off, bf16(8, 144))
    for scales in (torch.zeros(8, 3), torch.zeros(7), torch.zeros(8, dtype=torch.float64)):
        with pytest.raises(ValueError, match="x_scales"):
            m.forward(codes, off, bf16(8, 144), scales=scales)
    with pytest.raises(ValueError, match="codes"):
        m.forward(bf16(8, 144), off, bf16(8, 144), scales=torch.zeros(8))


def test_host_tensors_are_refused():
    m, off = mlp(), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        m.forward(bf16(8, 144), off, bf16(8, 144))
    with pytest.raises(ValueError, match="device tensor"):
        m.quantize()


def test_groups_that_the_experts_do_not_fit():
    for kw in ({"E": 8}, {"H": 64}, {"max_rows": 31}):
        with pytest.raises(ValueError):
            EPGroup(16, 144, 4, 2, 2, device="cpu", experts=mlp(**kw))


@pytest.mark.parametrize("act", [0, 2, 3, 4])
def test_gradient_formula_against_differences(act):
    """The 64-bit form of dx against central differences of act(z) . g: an error of
    h^2 / 6 times the third derivative, under 2 |g . W| for these, and of 2^-52 / h
    times the values'."""
    gen = torch.Generator().manual_seed(act)
    rows, K, N, wide, h = 6, 16, 32, 2 if act == 4 else 1, 2.0 ** -14
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    dy, wt, z = rand(rows, N), rand(1, K, N), rand(rows, wide * K)
    g = dy @ wt[0].T
    got, _, _ = F.product_dx(dy, torch.zeros(rows, N // 8).double(), [0, rows], wt, torch.zeros(1, K, N // 8).double(), act,
                             z if act else None)
    if not act:
        assert torch.equal(got, g)
        return
    # act(z) by the forward form: a product with the identity
    eye = torch.eye(wide * K, dtype=torch.float64)[None]
    none = torch.zeros(1, wide * K, wide * K // 8).double()

    def f(v):
        return F.product(v, torch.zeros(rows, wide * K // 8).double(), [0, rows], eye, none, None, act, None)[0]

    for c in range(wide * K):
        step = torch.zeros_like(z)
        step[:, c] = h
        want = ((f(z + step) - f(z - step)) / (2 * h) * g).sum(1)
        size = g[:, c % K].abs() * (1 + z.abs().amax(1))
        assert ((got[:, c] - want).abs() <= size * (2 * h * h + 2.0 ** -50 / h) + 1e-14).all()

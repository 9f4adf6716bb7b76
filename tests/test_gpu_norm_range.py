"""The norm and its gradient of rows whose sizes lie far from 1, whose squares or
whose products with the gradient may leave fp32, against their 64-bit forms."""
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B
from test_gpu_norm import check_norm, normal

pytestmark = pytest.mark.gpu

# A row of each kernel: a wave's, a workgroup's that holds it, one that reads it again.
WIDTHS = [16, 528, 1040, 2064, 7168, 16384, 32768, 65536]


def check_grad(s, d_y, ds, w, eps):
    T, H = s.shape
    d_x, d_w = torch.zeros_like(s), torch.zeros(H, device="cuda")
    B.moe_add_norm_grad(d_y, ds, s, w, eps, d_x, d_w)
    want, tol, want_w, tol_w = F.norm_grad(d_y, ds, s, w, eps)
    R.inside(d_x, want, F.bf16(want, tol), "d_x")
    R.inside(d_w, want_w, tol_w, "d_weight")
    for name in ("d_y", "sum"):  # in place
        a = dict(d_y=d_y.clone(), sum=s.clone())
        B.moe_add_norm_grad(a["d_y"], ds, a["sum"], w, eps, a[name])
        assert torch.equal(a[name], d_x), name


# sizes of the rows (2e-20: the root is there, its square is not) and of d_y, so that d_x stays inside bf16
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("scale,grad,eps", [(2e-20, 1.0, 0.0), (1e-19, 1e3, 1e-38), (1e15, 1e5, 1e-6)])
@pytest.mark.parametrize("stream", [True, False])
def test_norm_grad_of_small_and_large_rows(H, scale, grad, eps, stream):
    g = torch.Generator(device="cuda").manual_seed(H + stream)
    s, d_y, w = normal(g, 6, H, scale=scale), normal(g, 6, H, scale=grad), normal(g, H, dtype=torch.float32)
    ds = normal(g, 6, H, scale=grad / scale) if stream else None
    check_grad(s, d_y, ds, w, eps)


# 1e-23: squares below fp32's least value; 3e17: squares inside, the sum of a long row's not;
# 1e30: squares outside; 2e37: the largest rows whose sums with the residual stay finite
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("scale,eps", [(1e-36, 0.0), (1e-23, 0.0), (1e-20, 2.0 ** -136), (3e17, 1e-6), (1e30, 0.0), (2e37, 1e38)])
def test_norm_of_any_size(H, scale, eps):
    check_norm(5, H, True, True, False, eps=eps, scale=scale)
    check_norm(3, H, False, False, True, eps=eps, scale=scale)


@pytest.mark.parametrize("T,H", [(6000, 528), (6000, 2064), (1500, 32768)])
def test_norm_of_rows_of_every_size(T, H):
    """Rows of ordinary and other sizes take turns in a workgroup."""
    g = torch.Generator(device="cuda").manual_seed(3)
    size = torch.tensor([1.0, 1e30, 1e-30, 1e17, 2.0, 1e-18, 0.5], device="cuda")[torch.arange(T, device="cuda") % 7]
    x = (torch.randn(T, H, generator=g, device="cuda") * size[:, None]).bfloat16()
    check_norm(T, H, False, True, False, eps=0.0, x=x)
    check_grad(x, normal(g, T, H), normal(g, T, H), normal(g, H, dtype=torch.float32), 0.0)


# sizes of the rows and of d_y, so that d_x stays inside bf16; in the last three d_y s leaves fp32, or its sum does
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("scale,grad,eps", [(1e-36, 1e-20, 0.0), (1e-20, 1.0, 0.0), (1e-20, 1e-3, 2.0 ** -136), (1e-15, 1e-10, 0.0),
                                            (1e15, 1e5, 1e-6), (3e17, 1e2, 1e-6), (1e30, 1e10, 0.0), (1e37, 1e20, 1e38),
                                            (1e16, 1e23, 1e-6), (1e16, 1e21, 1e-6), (2.0, 3e36, 1e-6)])
@pytest.mark.parametrize("stream", [True, False])
def test_norm_grad_of_any_size(H, scale, grad, eps, stream):
    g = torch.Generator(device="cuda").manual_seed(H + stream)
    s, d_y, w = normal(g, 6, H, scale=scale), normal(g, 6, H, scale=grad), normal(g, H, dtype=torch.float32)
    ds = normal(g, 6, H, scale=grad / scale) if stream else None
    check_grad(s, d_y, ds, w, eps)


@pytest.mark.parametrize("H", [144, 2064, 32768])
def test_a_row_that_is_not_finite_reaches_no_other(H):
    g = torch.Generator(device="cuda").manual_seed(1)
    s, d_y = normal(g, 9, H), normal(g, 9, H)
    d_x = torch.zeros_like(s)
    B.moe_add_norm_grad(d_y, None, s, None, 0.0, d_x)
    s2, d_y2 = s.clone(), d_y.clone()
    s2[2, 5], s2[5, H - 1], d_y2[7, 0] = float("nan"), float("inf"), float("inf")
    got = torch.zeros_like(s)
    B.moe_add_norm_grad(d_y2, None, s2, None, 0.0, got)
    fine = [0, 1, 3, 4, 6, 8]
    assert torch.equal(got[fine], d_x[fine])
    assert not torch.isfinite(got[2]).any() and torch.isnan(got[5, H - 1]) and not torch.isfinite(got[7]).any()

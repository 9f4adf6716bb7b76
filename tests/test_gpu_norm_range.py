"""The norm's gradient of rows whose sizes lie far from 1, against its 64-bit form."""
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B
from test_gpu_norm import normal

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

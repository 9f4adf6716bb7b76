"""The training and expert calls on values and states at their edges: NaN and
infinities, masked tokens whose output counts, sums that must come out exactly."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

NONE, RELU, SILU, GELU, SWIGLU = range(5)


def offsets_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# rows, K, N of the kernel for few rows, of whole tiles and of tiles in parts
KERNELS = [(12, 80, 48), (3000, 80, 2064), (2100, 4096, 384)]


@pytest.mark.parametrize("act", [RELU, SILU, GELU, SWIGLU])
@pytest.mark.parametrize("rows,K,N", KERNELS)
def test_nan_passes_every_activation(rows, K, N, act):
    """A row of NaN comes out as a row of NaN, in preact and out alike."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    wide = 2 if act == SWIGLU else 1
    x, w = normal(g, rows, K), normal(g, 2, wide * N, K, scale=K ** -0.5)
    x[3] = float("nan")
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    pre = torch.zeros(rows, wide * N, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul(x, offsets_of([rows // 2, rows - rows // 2]), w, None, act, None, out, pre)
    for t in (out, pre):
        bad = torch.isnan(t)
        assert bad[3].all() and not bad[:3].any() and not bad[4:].any()


@pytest.mark.parametrize("rows,K,N", [(12, 48, 80), (3000, 528, 144), (100, 144, 8192)])
def test_gradient_passes_a_nan_of_relu(rows, K, N):
    """Where the pre-activation is NaN the gradient goes on as torch's does."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy, w, z = normal(g, rows, N), normal(g, 1, N, K, scale=K ** -0.5), normal(g, rows, K)
    z[1, 5], z[rows - 1, K - 1], z[2, 2] = float("nan"), float("nan"), 0.0
    dx = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul_dx(dy, offsets_of([rows]), w, RELU, z, dx)
    want, tol, _ = R.product_dx(dy, [0, rows], w, NONE, None)
    zz = z.double().requires_grad_()
    want, = torch.autograd.grad(torch.relu(zz), zz, want)
    assert want[1, 5] != 0 and want[2, 2] == 0
    R.inside(dx, want, tol, "dx")

"""Arrays of more than 2^32 bytes and 2^31 values: the rows behind, against the
64-bit forms of those alone."""
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B
from test_gpu_fp8_products import GELU, NONE, SWIGLU, coded_rows, coded_weights, normal, offsets_of

pytestmark = pytest.mark.gpu

T, H = 33000, 65536  # 2^31 < T * H
LAST = 40  # rows that are looked at


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def big(rows, n, dtype=torch.bfloat16):
    return torch.zeros(rows, n, dtype=dtype, device="cuda")


def test_norm_and_its_gradient():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, s, y, c = big(T, H), big(T, H), big(T, H), big(T, H, torch.uint8)
    x[-LAST:] = normal(g, LAST, H)
    w, v = normal(g, H, dtype=torch.float32), torch.zeros(T, F.blocks(H), device="cuda")
    B.moe_add_norm(x, None, w, 1e-5, s, y, c, v)
    assert torch.equal(s[-LAST:], x[-LAST:])
    _, want, tol = F.norm(x[-LAST:], None, w, 1e-5)
    R.inside(y[-LAST:], want, F.bf16(want, tol), "y")
    F.check_codes(c[-LAST:], v[-LAST:], want, tol, "y")
    assert not y[:LAST].any() and not c[:LAST].any()
    del c, v
    y.zero_()  # d_y now; the rows of zeros give nothing to the weights
    y[-LAST:] = normal(g, LAST, H)
    dw = torch.zeros(H, device="cuda")
    B.moe_add_norm_grad(y, None, s, w, 1e-5, x, dw)
    want, tol, want_w, tol_w = F.norm_grad(y[-LAST:], None, s[-LAST:], w, 1e-5)
    R.inside(x[-LAST:], want, F.bf16(want, tol), "d_x")
    # (a workgroup's sums are added to those of the others, zeros: at most as many steps again)
    R.inside(dw, want_w, 2 * tol_w, "d_weight")
    assert not x[:LAST].any()


def test_codes_of_rows_and_weights():
    g = torch.Generator(device="cuda").manual_seed(2)
    x, c, v = big(T, H), big(T, H, torch.uint8), torch.zeros(T, F.blocks(H), device="cuda")
    x[-LAST:] = normal(g, LAST, H)
    B.moe_quant_rows(x, c, v)
    want = x[-LAST:].double()
    F.check_codes(c[-LAST:], v[-LAST:], want, 0 * want, "rows")
    w = x[:32992].view(1, 32992, H)  # a multiple of 16 rows
    x[32960:32992] = normal(g, 32, H)
    codes, scales = c[:32992].view(1, 32992, H), torch.zeros(1, 1, F.blocks(32992), F.blocks(H), device="cuda")
    codes_t, scales_t = torch.zeros(1, H, 32992, dtype=torch.uint8, device="cuda"), \
        torch.zeros(1, F.blocks(H), 1, F.blocks(32992), device="cuda")
    B.moe_quant_weights(w, codes, scales, codes_t, scales_t)
    last = 32992 // 128 * 128  # first of the last block's 96 rows
    tops = w[0, last:].double().abs().amax(0).view(-1, 128).amax(1)
    R.inside(scales[0, 0, -1], tops / 448, 4 * R.U32 * tops / 448, "scales")
    assert torch.equal(scales_t[0, :, 0, -1], scales[0, 0, -1]) and torch.equal(codes_t[0, :, last:], codes[0, last:].T)
    q = w[0, last:].double() / F.at_columns(scales[0, 0, -1], H)
    # as check_codes: q is off by the scale's rounding, u, and the quotient's own, under 3 u
    # with the step by the reciprocal; a code of it by half a step of what that gives
    dq = 4 * R.U32 * q.abs()
    R.inside(F.e4m3(codes[0, last:]), q, dq + torch.maximum(F.UE4M3 * (q.abs() + dq), torch.full_like(q, F.LEAST)), "codes")


# K, activation of the forward call, of the gradient's
@pytest.mark.parametrize("act,back", [(NONE, NONE), (SWIGLU, SWIGLU), (GELU, NONE)])
def test_products(act, back):
    g = torch.Generator(device="cuda").manual_seed(3)
    K, N, wide = 64, H, 2 if act == SWIGLU else 1
    x, xs, x64, xp = coded_rows(g, T, K, True)
    w, ws, w64, wp = coded_weights(g, 2, wide, N, K)
    out, codes, scales = big(T, N), big(T, N, torch.uint8), torch.zeros(T, F.blocks(N), device="cuda")
    off = offsets_of([700, T - 705])  # five rows of no run
    B.moe_expert_matmul_fp8(x, xs, off, w, ws, None, act, None, out, codes, scales)
    part = slice(T - 5 - LAST, T - 5)
    y, dy, *_ = F.product(x64[part], xp[part], [0, LAST], w64[1:], wp[1:], None, act, None)
    R.inside(out[part], y, F.bf16(y, dy), "out")
    F.check_codes(codes[part], scales[part], y, dy, "out")
    assert not out[-5:].any() and not codes[-5:].any() and not scales[-5:].any()
    # the gradient of rows of as many columns: out is z, then dx
    del codes, scales
    C, n = (H, 64) if back != SWIGLU else (H // 2, 64)
    dy8, dys, d64, dp = coded_rows(g, T, n, False)
    wt, wts, wt64, wtp = coded_weights(g, 2, 1, C, n)  # any weights, taken as transposed ones
    wts = wts.view(2, F.blocks(C), 1, F.blocks(n))
    z = out[part].clone()
    B.moe_expert_matmul_fp8_dx(dy8, dys, off, wt, wts, back, out if back else None, out)
    dx, tol, _ = F.product_dx(d64[part], dp[part], [0, LAST], wt64[1:], wtp[1:], back, z if back else None)
    R.inside(out[part], dx, F.bf16(dx, tol), "dx")
    assert not out[-5:].any()

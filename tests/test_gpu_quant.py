"""E4M3 codes and scales of rows and of weights against the rule in 64 bits."""
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

MARK = 77


def check(codes, scales, x, what):
    F.check_codes(codes, scales, x.double(), 0 * x.double(), what)


@pytest.mark.parametrize("rows,H,halves", [(1, 16, 1), (3, 128, 1), (5, 144, 1), (33, 528, 1), (1, 7168, 1), (70, 2048, 1),
                                           (300, 8208, 1), (9000, 48, 1), (2, 65536, 1), (2, 32, 2), (40, 288, 2),
                                           (33, 1056, 2), (17, 4096, 2), (3, 131072, 2)])
def test_rows(rows, H, halves):
    g = torch.Generator(device="cuda").manual_seed(rows + H)
    x = (torch.randn(rows, H, generator=g, device="cuda") * torch.randn(rows, 1, generator=g, device="cuda").exp()).bfloat16()
    x[0, :16] = 0
    nb = F.blocks(H // halves)
    codes = torch.full((rows + 1, H), MARK, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 1, halves, nb), -1.0, device="cuda")
    B.moe_quant_rows(x, codes[:rows], scales[:rows] if halves == 2 else scales[:rows, 0], halves=halves)
    check(codes[:rows].view(rows, halves, -1), scales[:rows], x.view(rows, halves, -1), "rows")
    assert (codes[rows] == MARK).all() and (scales[rows] == -1).all()


def test_rows_follow_the_payloads_rule():
    """Rows of one block: the codes that a pack of one slot makes."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(500, 128, generator=g, device="cuda").bfloat16()
    codes, scales = torch.zeros(500, 128, dtype=torch.uint8, device="cuda"), torch.zeros(500, 1, device="cuda")
    B.moe_quant_rows(x, codes, scales)
    send, send_scales = B.alloc_rows(500, 128, B.MOE_QUANT_FP8, "cuda")
    B.moe_dispatch_pack(x, 500, 128, 1, torch.arange(500, dtype=torch.int32, device="cuda"), B.MOE_QUANT_FP8, send, send_scales)
    assert torch.equal(send, codes) and torch.equal(send_scales, scales[:, 0])


@pytest.mark.parametrize("rows", [40, 100])
def test_rows_of_runs(rows):
    """Offsets of a rank's own experts, ending inside the buffer or past it."""
    x = torch.randn(rows, 272, device="cuda").bfloat16()
    off = torch.tensor([500, 510, 510, 557], dtype=torch.int32, device="cuda")
    codes = torch.full((rows, 272), MARK, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 3), -1.0, device="cuda")
    B.moe_quant_rows(x, codes, scales, offsets=off)
    n = min(rows, 57)
    check(codes[:n], scales[:n], x[:n], "rows")
    assert (codes[n:] == MARK).all() and (scales[n:] == -1).all()


def test_values_at_the_edges():
    """Zeros, the smallest and largest bf16 values, NaN and infinities, each in a
    block of its own."""
    x = torch.zeros(1, 7 * 128, device="cuda")
    x[0, 128:256] = 3e38
    x[0, 256:384] = 1e-40
    x[0, 384], x[0, 390] = float("nan"), 5.0
    x[0, 512], x[0, 520] = float("-inf"), 5.0
    x[0, 640:768] = float("nan")
    x[0, 768:] = 448.0
    x = x.bfloat16()
    codes, scales = torch.zeros(1, 896, dtype=torch.uint8, device="cuda"), torch.zeros(1, 7, device="cuda")
    B.moe_quant_rows(x, codes, scales)
    v = F.e4m3(codes) * F.at_columns(scales, 896)
    assert (v[0, :128] == 0).all() and scales[0, 0] == 0
    assert ((v[0, 128:256] / x[0, 128:256].double() - 1).abs() <= 4 * F.U32).all()
    # 1e-40 / 448 is some 159 steps of the subnormals: a scale off by half a step
    assert ((v[0, 256:384] / x[0, 256:384].double() - 1).abs() <= F.UE4M3 + 1 / 159).all()
    assert torch.isnan(v[0, 384:512]).all() and torch.isnan(scales[0, 3])
    assert torch.isnan(v[0, 512]) and torch.isinf(scales[0, 4])
    assert torch.isnan(v[0, 640:768]).all()
    assert (v[0, 768:] == 448).all() and scales[0, 6] == 1


@pytest.mark.parametrize("E,N,K,halves", [(1, 16, 16, 1), (2, 128, 128, 1), (3, 144, 272, 1), (2, 16, 1040, 2),
                                          (4, 272, 144, 2), (1, 2048, 768, 2), (5, 384, 528, 1)])
def test_weights(E, N, K, halves):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    w = torch.randn(E, halves * N, K, generator=g, device="cuda").bfloat16()
    w[0, 0, :16] = 0
    nbn, nbk = F.blocks(N), F.blocks(K)
    codes = torch.full((E + 1, halves * N, K), MARK, dtype=torch.uint8, device="cuda")
    turned = torch.full((E + 1, K, halves * N), MARK, dtype=torch.uint8, device="cuda")
    scales = torch.full((E + 1, halves, nbn, nbk), -1.0, device="cuda")
    scales_t = torch.full((E + 1, nbk, halves, nbn), -1.0, device="cuda")
    B.moe_quant_weights(w, codes[:E], scales[:E], turned[:E], scales_t[:E], halves)
    for t, mark in ((codes, MARK), (turned, MARK), (scales, -1), (scales_t, -1)):
        assert (t[E] == mark).all()
    codes, turned, scales, scales_t = codes[:E], turned[:E], scales[:E], scales_t[:E]
    tall = torch.nn.functional.pad(w.double().view(E, halves, N, K), (0, nbk * 128 - K, 0, nbn * 128 - N))
    top = tall.abs().view(E, halves, nbn, 128, nbk, 128).amax((3, 5))
    R.inside(scales, top / 448, 4 * F.U32 * top, "scales")
    s = scales.double().repeat_interleave(128, 2).repeat_interleave(128, 3)[:, :, :N, :K]
    q = w.double().view(E, halves, N, K) / s
    tol = (F.UE4M3 * q.abs()).clamp(min=F.LEAST) + 4 * F.U32 * q.abs()
    R.inside(F.e4m3(codes).view(E, halves, N, K), q, tol, "codes")
    assert torch.equal(turned, codes.transpose(1, 2)) and torch.equal(scales_t, scales.permute(0, 3, 1, 2))
    alone, alone_scales = torch.zeros_like(codes), torch.zeros_like(scales)
    B.moe_quant_weights(w, alone, alone_scales, halves=halves)
    assert torch.equal(alone, codes) and torch.equal(alone_scales, scales)

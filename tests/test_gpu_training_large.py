"""The training and expert calls where an offset passes 32 bits, and at their
largest counts; checked on samples of rows."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

NONE, RELU, SILU, GELU, SWIGLU = range(5)
ROWS = 70001  # x 32768 columns of bf16: 4.6 GB


def normal(*shape, scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(scale)


def sample(n):
    return torch.tensor([0, 1, 255, 256, n // 2, n - 4465, n - 258, n - 2, n - 1], device="cuda")


def offsets_of(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("K,N,act", [(32768, 16, NONE), (32768, 48, GELU), (64, 32768, SWIGLU), (64, 32768, SILU)])
def test_product_rows(K, N, act):
    wide = 2 if act == SWIGLU else 1
    x, w = normal(ROWS, K), normal(1, wide * N, K, scale=K ** -0.5, seed=1)
    out = torch.empty(ROWS, N, dtype=torch.bfloat16, device="cuda")
    pre = torch.empty(ROWS, wide * N, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul(x, offsets_of([ROWS]), w, None, act, None, out, pre)
    at = sample(ROWS)
    y, dy, z, dz, _ = R.product(x[at], [0, len(at)], w, None, act, None)
    R.inside(out[at], y, dy, "out")
    R.inside(pre[at], z, dz, "preact")


@pytest.mark.parametrize("N,K,act", [(32768, 32, NONE), (64, 32768, SWIGLU)])
def test_dx_rows(N, K, act):
    wide = 2 if act == SWIGLU else 1
    dy, w = normal(ROWS, N), normal(1, N, K, scale=K ** -0.5, seed=1)
    z = normal(ROWS, wide * K, seed=2) if act else None
    dx = torch.empty(ROWS, wide * K, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul_dx(dy, offsets_of([ROWS]), w, act, z, dx)
    at = sample(ROWS)
    want, tol, _ = R.product_dx(dy[at], [0, len(at)], w, act, z[at] if act else None)
    R.inside(dx[at], want, tol, "dx")


def test_dw_rows():
    dy, x = normal(ROWS, 32768), normal(ROWS, 16, seed=1)
    dw, db = torch.empty(1, 32768, 16, device="cuda"), torch.empty(1, 32768, device="cuda")
    B.moe_expert_matmul_dw(dy, x, offsets_of([ROWS]), dw, db)
    at = torch.tensor([0, 31, 16383, 32640, 32767], device="cuda")
    want, tol, wb, tb = R.product_dw(dy[:, at].contiguous(), x, [0, ROWS], 1)
    R.inside(dw[:, at], want, tol, "dw")
    R.inside(db[:, at], wb, tb, "dbias")


def test_weights():
    """5.4 GB of weights, 10.7 GB of their gradients; the last experts checked."""
    E, N, K = 40, 8192, 8192
    w, x, dy = normal(E, N, K, scale=K ** -0.5), normal(2 * E, K, seed=1), normal(2 * E, N, seed=2)
    off = offsets_of([2] * E)
    out, dx = torch.empty_like(dy), torch.empty_like(x)
    dw = torch.empty(E, N, K, device="cuda")
    B.moe_expert_matmul(x, off, w, None, NONE, None, out)
    B.moe_expert_matmul_dx(dy, off, w, NONE, None, dx)
    B.moe_expert_matmul_dw(dy, x, off, dw)
    last, runs = slice(2 * E - 4, 2 * E), [0, 2, 4]
    y, tol, *_ = R.product(x[last], runs, w[-2:], None, NONE, None)
    R.inside(out[last], y, tol, "out")
    want, tol, _ = R.product_dx(dy[last], runs, w[-2:], NONE, None)
    R.inside(dx[last], want, tol, "dx")
    want, tol, *_ = R.product_dw(dy[last], x[last], runs, 2)
    R.inside(dw[-2:], want, tol, "dw")


@pytest.mark.parametrize("per", [0, 3])
def test_the_most_experts(per):
    """1024 runs, every third of `per` rows and one of 700."""
    lengths = [per if e % 3 == 0 else 0 for e in range(1024)]
    lengths[1000] = 700
    rows, K, N = sum(lengths), 48, 80
    x, w, dy = normal(rows, K), normal(1024, 2 * N, K, scale=K ** -0.5, seed=1), normal(rows, 2 * N, seed=2)
    off = offsets_of(lengths)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(1024, 2 * N, K, device="cuda")
    B.moe_expert_matmul(x, off, w, None, SWIGLU, None, out)
    B.moe_expert_matmul_dx(dy, off, w, NONE, None, dx)
    B.moe_expert_matmul_dw(dy, x, off, dw)
    y, tol, *_ = R.product(x, off.tolist(), w, None, SWIGLU, None)
    R.inside(out, y, tol, "out")
    want, tol, _ = R.product_dx(dy, off.tolist(), w, NONE, None)
    R.inside(dx, want, tol, "dx")
    want, tol, *_ = R.product_dw(dy, x, off.tolist(), 1024)
    R.inside(dw, want, tol, "dw")


@pytest.mark.parametrize("quant", [0, 1])
def test_combine_grad_rows(quant):
    T, H, k = 20001, 16384, 8
    rows = normal(T * k, H) if quant == 0 else torch.randint(-127, 128, (T * k, H), dtype=torch.int8, device="cuda")
    scales = torch.rand(T * k, device="cuda") if quant else None
    pos = torch.randperm(T * k, device="cuda").int()
    d_out, w = normal(T, H, seed=1), torch.rand(T, k, device="cuda")
    d_rows, d_w = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, k, device="cuda")
    B.moe_combine_grad(d_out, rows, scales, quant, pos, w, T, H, k, d_rows, d_w)
    at = sample(T)
    p = pos.view(T, k)[at].long()
    d = d_out[at].double()[:, None]
    v = rows[p].double() * (scales[p].double()[..., None] if quant else 1.0)
    want = d * w[at].double()[..., None]
    R.inside(d_rows[p], want, want.abs() * R.UBF16 * (1 + 2.0 ** -14), "d_rows")
    R.inside(d_w[at], (d * v).sum(2), (d * v).abs().sum(2) * (64 + 6 + 16 + 4) * R.U32, "d_w")


def test_balance_of_many_logits():
    T, E, k = (1 << 20) + 77, 1024, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty(T, E, device="cuda").normal_(generator=g)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    w, d_w = torch.rand(T, k, device="cuda"), torch.rand(T, k, device="cuda")
    out = B.moe_balance_loss(logits, idx, None, B.alloc_balance(T, T, E, k, "cuda"))
    d_loss, d_logits = torch.ones(1, device="cuda") * T, torch.empty_like(logits)
    B.moe_route_grad(logits, idx, w, d_w, None, d_loss, out, d_logits)
    sums = torch.zeros(E, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1 << 16):
        sums += logits[a:a + (1 << 16)].double().softmax(1).sum(0)
    counts = torch.bincount(idx.view(-1).long(), minlength=E)
    rel = (14.0 + E / 16 + 12 + T / 1024 + 16) * 2 * R.U32  # |logit| < 7: R.softmax_rel_bound's terms
    assert torch.equal(out.expert_counts[0].long(), counts) and out.tokens.item() == T
    R.inside(out.prob_sums[0], sums, sums * rel, "prob_sums")
    loss = E / (k * float(T) ** 2) * (counts * sums).sum()
    R.inside(out.loss[0], loss, loss * (rel + 4 * R.U32), "loss")
    at = sample(T)
    want, tol = R.route_grad(logits[at].double().softmax(1).cpu().numpy(), idx[at].cpu().numpy(), w[at].cpu().numpy(),
                             d_w[at].cpu().numpy(), np.ones(len(at), bool), d_loss.cpu().numpy(),
                             counts[None].cpu().numpy(), np.array([T]), T, E, k, rel)
    R.inside(d_logits[at].cpu(), want, tol, "d_logits")


def test_the_most_segments():
    T, E, k = 65535, 5, 2
    logits = torch.randn(T, E, device="cuda")
    idx = logits.topk(k, 1).indices.int()
    out = B.moe_balance_loss(logits, idx, None, B.alloc_balance(T, 1, E, k, "cuda"))
    p = logits.double().softmax(1)
    want = E / k * p.gather(1, idx.long()).sum(1)
    R.inside(out.loss, want, want * 40 * R.U32, "loss")
    assert (out.tokens == 1).all() and (out.expert_counts.sum(1) == k).all()
    d = torch.empty_like(logits)
    B.moe_route_grad(logits, idx, None, None, None, torch.ones(T, device="cuda"), out, d)
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, idx.long(), 1.0)
    mean = (p * hot).sum(1, keepdim=True)
    R.inside(d, E / k * p * (hot - mean), E / k * p * (hot + mean) * 60 * R.U32, "d_logits")

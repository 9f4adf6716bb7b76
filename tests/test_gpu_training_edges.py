"""The training and expert calls on values and states at their edges: NaN and
infinities, masked tokens whose output counts, sums that must come out exactly."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd.epgroup import EPGroup
from combine_fp32_router_amd.experts import ExpertMLP

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


@pytest.mark.parametrize("E,k", [(8, 2), (64, 4), (66, 2), (300, 3), (1024, 8)])
def test_masked_rows_stay_zero_for_any_loss_gradient(E, k):
    """A segment without live tokens may carry an infinite weight (one over its
    tokens, say): its rows, and a masked token's of any segment, are zeros."""
    T, seg = 70, 16
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = logits.topk(k, 1).indices.int()
    w, d_w = torch.rand(T, k, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    mask = (torch.rand(T, generator=g, device="cuda") < 0.6).to(torch.uint8)
    mask[16:32] = 0
    mask[32:34] = torch.tensor([1, 0])
    bal = B.moe_balance_loss(logits, idx, mask, B.alloc_balance(T, seg, E, k, "cuda"))
    plain, odd = torch.tensor([0.5, 0.0, 2.0, 1.0, 3.0], device="cuda"), torch.empty(5, device="cuda")
    odd.copy_(plain)
    odd[1], odd[2], odd[4] = float("inf"), float("nan"), -float("inf")
    for weights in (d_w, None):
        want, got = torch.empty_like(logits), torch.empty_like(logits)
        gates = w if weights is not None else None
        B.moe_route_grad(logits, idx, gates, weights, mask, plain, bal, want)
        B.moe_route_grad(logits, idx, gates, weights, mask, odd, bal, got)
        assert not want[mask == 0].any() and not got[mask == 0].any()
        assert torch.equal(got[:16], want[:16]) and torch.equal(got[48:64], want[48:64])
        assert not torch.isfinite(got[32:48][mask[32:48] != 0]).all(1).any()


@pytest.mark.parametrize("E,k", [(8, 2), (33, 4), (64, 4), (256, 8), (300, 3), (515, 5), (1024, 8)])
def test_router_gradient_over_its_own_logits(E, k):
    """d_logits may be logits: the same bits as apart from them."""
    T, seg = 1001, 400
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = logits.topk(k, 1).indices.int()
    w, d_w = torch.rand(T, k, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8)
    bal = B.moe_balance_loss(logits, idx, mask, B.alloc_balance(T, seg, E, k, "cuda"))
    d_loss, apart = torch.randn(3, generator=g, device="cuda") * T, torch.empty_like(logits)
    B.moe_route_grad(logits, idx, w, d_w, mask, d_loss, bal, apart)
    B.moe_route_grad(logits, idx, w, d_w, mask, d_loss, bal, logits)
    assert torch.equal(apart, logits)


@pytest.mark.parametrize("E,k", [(8, 2), (33, 4), (256, 8), (300, 3)])
def test_masked_tokens_keep_their_gates_if_asked(E, k):
    """masked_gates: a masked row has the gate weights' part alone, a live one
    the same bits as without."""
    T, seg = 333, 100
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = logits.topk(k, 1).indices.int()
    w, d_w = torch.rand(T, k, generator=g, device="cuda"), torch.randn(T, k, generator=g, device="cuda")
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    logits[mask == 0] = float("nan")  # not in the loss: not read
    bal = B.moe_balance_loss(logits, idx, mask, B.alloc_balance(T, seg, E, k, "cuda"))
    d_loss = torch.tensor([1.0, 20.0, -3.0, 4.0], device="cuda")
    plain, gates, got, only = (torch.empty_like(logits) for _ in range(4))
    B.moe_route_grad(logits, idx, w, d_w, mask, d_loss, bal, plain)
    B.moe_route_grad(None, idx, w, d_w, None, None, None, gates)
    B.moe_route_grad(logits, idx, w, d_w, mask, d_loss, bal, got, masked_gates=True)
    B.moe_route_grad(None, idx, w, d_w, mask, None, None, only, masked_gates=True)
    want, tol = R.route_grad(np.zeros((T, E)), idx.cpu().numpy(), w.cpu().numpy(), d_w.cpu().numpy(), np.ones(T, bool),
                             None, None, None, T, E, k, 0.0)
    R.inside(gates.cpu(), want, tol, "gates")
    off = mask == 0
    assert torch.equal(got[~off], plain[~off]) and torch.equal(only, gates)
    assert torch.equal(got[off], gates[off]) and gates[off].any() and not plain[off].any()


def test_a_layer_gives_masked_tokens_their_gates_if_asked():
    """With masked_gates the logits' gradient of a layer is that of its output
    for every token, and of the balance loss for the live ones."""
    T, H, E, k = 200, 64, 8, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    mlp = ExpertMLP(normal(g, E, 96, H, scale=H ** -0.5), normal(g, E, H, 48, scale=0.15), SWIGLU, max_rows=400, train=True)
    group = EPGroup(T, H, E, k, 4, experts=mlp)
    logits, x, d_out = torch.randn(T, E, generator=g, device="cuda"), normal(g, T, H), normal(g, T, H)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    bal, d_loss = B.alloc_balance(T, T, E, k, "cuda"), torch.full((1,), 50.0, device="cuda")
    out, plain, got, alone = torch.empty_like(x), *(torch.empty_like(logits) for _ in range(3))
    group.run(logits, x, out, balance=bal, token_mask=mask)
    group.backward(d_out, None, plain, d_loss=d_loss)
    group.backward(d_out, None, got, d_loss=d_loss, masked_gates=True)
    group.run(logits, x, out)
    group.backward(d_out, None, alone)
    off = mask == 0
    assert torch.equal(got[~off], plain[~off]) and torch.equal(got[off], alone[off]) and not plain[off].any()
    # the gates' part, from the returned rows: <d_out, d out / d logits>
    rows = torch.zeros(T, k, H, dtype=torch.float64, device="cuda")
    for s, (a, b) in enumerate(group.bounds):
        at = group.views[s].pos[:(b - a) * k].long()
        rows[a:b] = group.send_rows(s, 0).view(torch.bfloat16).view(-1, H)[at].double().view(b - a, k, H)
    z = logits.double().requires_grad_()
    gate = z.gather(1, group.idx[:T].long()).softmax(1)
    want, = torch.autograd.grad(((gate[..., None] * rows).sum(1) * d_out.double()).sum(), z)
    size = (rows * d_out.double()[:, None]).abs().sum(2).sum(1, keepdim=True).expand_as(want)
    R.inside(alone, want, size * (H + k + 24) * 2 * R.U32, "gates")


@pytest.mark.parametrize("T,E,seg", [((1 << 20) + 77, 16, 1 << 21), (1 << 19, 64, 1 << 18), (300001, 256, 150001),
                                     (200003, 300, 200003), (60001, 1024, 60001), (5000, 8, 250)])
def test_probability_sums_of_long_segments(T, E, seg):
    """The bound of a sum of probabilities by what a lane adds: a block has the
    batch's 512th part, in 16s, at least 32 tokens, or a short segment, and
    shares it over its waves and, up to 256 experts, their four groups of lanes."""
    seg = min(seg, T)
    tokens = min(max(32, -(-T // 512) + 15 & ~15), seg)
    if seg <= 256 and (T >= (16 if E <= 256 else 128) * seg or seg * E <= 32768):
        tokens = seg
    waves = (16 if tokens == seg and E <= 256 else 8 if E <= 512 else 4) * (4 if E <= 256 else 1)
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = torch.randint(0, E, (T, 2), generator=g, device="cuda").int()
    out = B.moe_balance_loss(logits, idx, None, B.alloc_balance(T, seg, E, 2, "cuda"))
    S = -(-T // seg)
    sums = torch.stack([logits[s * seg:(s + 1) * seg].double().softmax(1).sum(0) for s in range(S)])
    spread = (logits.amax() - logits.amin()).item()
    rel = (spread + E / 16 + 12 + 2 * -(-tokens // (2 * waves)) + 1) * 2 * R.U32  # R.softmax_rel_bound's terms
    R.inside(out.prob_sums, sums, sums * rel, "prob_sums")
    assert torch.equal(out.expert_counts.sum(1), 2 * out.tokens) and out.tokens.sum() == T


def test_a_group_keeps_the_device_it_was_made_on():
    """`cuda` names the device that is current when the group is made, not
    whichever is current when it runs."""
    group = EPGroup(16, 32, 4, 2, 2, device="cuda")
    assert group.device == group.idx.device == torch.device("cuda", torch.cuda.current_device())

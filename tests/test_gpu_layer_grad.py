"""A whole layer forward and backward -- router, balance loss, pack, exchange,
regroup, experts, return and combine, then every gradient -- against its
64-bit form.  A value of the reference carries a bound on how far the layer's
roundings (bf16 rows, fp32 sums, the payload's codes) may move it."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd.driver import capture
from combine_fp32_router_amd.epgroup import EPGroup
from combine_fp32_router_amd.experts import ExpertMLP

pytestmark = pytest.mark.gpu

SLOPE2 = {0: 0.0, 1: 0.0, 2: 0.5, 3: 0.8}  # bounds of the second derivatives (relu: away from 0)


class V:
    """A value and a bound on the error of its computed counterpart."""

    def __init__(self, v, err=0.0):
        self.v = v
        self.err = err if torch.is_tensor(err) else torch.full_like(v, err)

    def size(self):
        return self.v.abs() + self.err

    def bf16(self):
        return V(self.v, self.err + R.UBF16 * self.size())

    def __matmul__(self, w):
        n = self.v.shape[-1]
        return V(self.v @ w, self.err @ w.abs() + n * R.U32 * (self.size() @ w.abs()))

    def plus(self, b):
        return V(self.v + b, self.err + R.U32 * (self.size() + b.abs()))

    def times(self, o):
        return V(self.v * o.v, self.size() * o.err + self.err * o.v.abs() + 2 * R.U32 * self.size() * o.size())

    def rows(self, at):
        return V(self.v[at], self.err[at])

    def put(self, at, o):
        self.v[at], self.err[at] = o.v, o.err

    def columns(self, a, b):
        return V(self.v[:, a:b], self.err[:, a:b])


def act(z, a):
    if a == B.MOE_ACT_SWIGLU:
        n = z.v.shape[1] // 2
        return act(z.columns(0, n), B.MOE_ACT_SILU).times(z.columns(n, 2 * n))
    y, slope = R.act64(z.v, a)
    return V(y, slope * z.err + R.act_noise(z.v))


def slope(z, a):
    s = R.slope64(z.v, a)
    err = SLOPE2[a] * z.err + R.act_noise(z.v)
    if a == B.MOE_ACT_RELU:  # either side of 0
        err = torch.where(z.v.abs() <= z.err, torch.ones_like(err), torch.zeros_like(err))
    return V(s, err)


def through(g, z, a):
    """The gradient g of act(z) as that of z."""
    if a == B.MOE_ACT_SWIGLU:
        n = z.v.shape[1] // 2
        zg, zu = z.columns(0, n), z.columns(n, 2 * n)
        p, q = g.times(zu).times(slope(zg, B.MOE_ACT_SILU)), g.times(act(zg, B.MOE_ACT_SILU))
        return V(torch.cat([p.v, q.v], 1), torch.cat([p.err, q.err], 1))
    return g.times(slope(z, a))


def exact_rows(T, H, quant, g):
    """Rows that the payload holds exactly: its scale comes out as 1."""
    if quant == 0:
        return torch.randn(T, H, generator=g, device="cuda").bfloat16(), 1.0
    if quant == 3:
        x = (torch.randn(T, H, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn).float()
        top = 448.0
    else:
        top = 127.0 if quant == 1 else 7.0
        x = (torch.randn(T, H, generator=g, device="cuda") * top / 2).round().clamp(-top, top)
    x[:, 0] = top
    return x.bfloat16(), {1: 63.0, 2: 3.5, 3: 60.0}[quant]


def returned_rows(grp, quant, at, source):
    """Values of the returned rows `at` (int64 [n]) of a source, in 64 bits."""
    n, H = grp.source_rows, grp.H
    raw, sc = grp.send_rows(source, quant), grp.send_scales_of(source).double()
    if quant == 0:
        return raw.view(torch.bfloat16).view(n, H)[at].double()
    if quant == 3:
        codes = raw.view(torch.float8_e4m3fn).view(n, H).double()
    elif quant == 1:
        codes = raw.view(torch.int8).view(n, H).double()
    else:
        b = raw.view(n, H // 2).int()
        pair = torch.stack([b & 15, b >> 4], -1).view(n, H)
        codes = (pair - 16 * (pair > 7).int()).double()
    return codes[at] * sc[at, None]


def code_step(y, quant):
    """Half a step of a row's code, with its size's own error."""
    top = (y.v.abs() + y.err).amax(1, keepdim=True)
    if quant == 0:
        return torch.zeros_like(y.v)
    if quant == 3:
        return y.size() * 2.0 ** -4 + top / 448 * 2.0 ** -10
    return (top / (127 if quant == 1 else 7) * 0.5 * (1 + 2.0 ** -20)).expand_as(y.v)


# T, H, I, E, k, R, act, quant, capacity factor, biases, masked share
CASES = [(96, 64, 48, 8, 2, 4, B.MOE_ACT_SWIGLU, 0, None, True, 0.0),
         (257, 128, 96, 16, 4, 8, B.MOE_ACT_GELU, 0, None, True, 0.2),
         (200, 96, 64, 8, 2, 2, B.MOE_ACT_RELU, 0, 1.0, False, 0.0),
         (150, 64, 80, 8, 3, 4, B.MOE_ACT_SILU, 1, None, True, 0.1),
         (150, 64, 80, 8, 3, 4, B.MOE_ACT_SWIGLU, 2, None, False, 0.0),
         (150, 64, 80, 8, 3, 1, B.MOE_ACT_SWIGLU, 3, 1.25, True, 0.0),
         (5, 64, 16, 16, 2, 8, B.MOE_ACT_SWIGLU, 0, None, True, 0.0),
         (1, 16, 16, 1, 1, 1, B.MOE_ACT_NONE, 0, None, True, 0.0),
         (1500, 256, 128, 4, 2, 2, B.MOE_ACT_SWIGLU, 0, None, True, 0.1)]


def make(T, H, I, E, k, Rn, a, quant, biases, masked, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x, size = exact_rows(T, H, quant, g) if T else (torch.empty(0, H, dtype=torch.bfloat16, device="cuda"), 1.0)
    wide = 2 if a == B.MOE_ACT_SWIGLU else 1
    w_up = (rand(E, wide * I, H) / (size * H ** 0.5)).bfloat16()
    w_down = (rand(E, H, I) / I ** 0.5).bfloat16()
    b_up, b_down = (rand(E, wide * I) * 0.1, rand(E, H) * 0.1) if biases else (None, None)
    logits = rand(T, E)
    mask = (torch.rand(T, generator=g, device="cuda") >= masked).to(torch.uint8) if masked else None
    d_out = rand(T, H).bfloat16()
    rows = Rn * -(-T // Rn) * k
    mlp = ExpertMLP(w_up, w_down, a, b_up, b_down, max_rows=rows, train=True)
    return EPGroup(T, H, E, k, Rn, experts=mlp), mlp, x, logits, mask, d_out


@pytest.mark.parametrize("T,H,I,E,k,Rn,a,quant,cf,biases,masked", CASES)
def test_layer_and_its_gradients(T, H, I, E, k, Rn, a, quant, cf, biases, masked):
    grp, mlp, x, logits, mask, d_out = make(T, H, I, E, k, Rn, a, quant, biases, masked)
    seg = max(1, T // 2)
    bal = B.alloc_balance(T, seg, E, k, "cuda")
    S = bal.loss.numel()
    d_loss = torch.linspace(0.5, 2.0, S, device="cuda")
    out, d_x = torch.empty_like(x), torch.empty_like(x)
    d_logits = torch.empty_like(logits)
    grads = mlp.alloc_grads()
    grp.run(logits, x, out, quant=quant, capacity_factor=cf, balance=bal, token_mask=mask)
    grp.backward(d_out, d_x, d_logits, grads, d_loss)
    torch.cuda.synchronize()

    idx, w = grp.idx[:T].long(), grp.w[:T].double()
    top = logits.double().topk(k, 1)
    assert torch.equal(idx, top.indices)
    R.inside(w, top.values.softmax(1), 4 * R.U32 * torch.ones_like(w), "gates")
    kept, rows, at = torch.zeros(T, k, dtype=torch.bool, device="cuda"), [], []
    got = torch.zeros(T, k, H, dtype=torch.float64, device="cuda")
    for s, (t0, t1) in enumerate(grp.bounds):
        if t1 > t0:
            p = grp.views[s].pos[:(t1 - t0) * k].view(-1, k).long()
            kept[t0:t1] = p >= 0
            got[t0:t1] = returned_rows(grp, quant, p.clamp(min=0).reshape(-1), s).view(-1, k, H)
    assert (cf is not None) or bool(kept.all())

    # forward, slot by slot
    slot_t, slot_j = kept.nonzero(as_tuple=True)
    e_of = idx[slot_t, slot_j]
    n, wide = len(slot_t), mlp.wide
    zeros = lambda c: V(torch.zeros(n, c, dtype=torch.float64, device="cuda"))  # noqa: E731
    z, h, y = zeros(wide * I), zeros(I), zeros(H)
    wu, wd = mlp.w_up.double(), mlp.w_down.double()
    for e in range(E):
        r = (e_of == e).nonzero()[:, 0]
        ze = V(x[slot_t[r]].double()) @ wu[e].T
        ze = ze.plus(mlp.b_up[e].double()) if biases else ze
        he = act(ze, a).bf16()
        ye = he @ wd[e].T
        ye = (ye.plus(mlp.b_down[e].double()) if biases else ye).bf16()
        z.put(r, ze.bf16()), h.put(r, he), y.put(r, ye)
    slots = got[slot_t, slot_j]
    R.inside(slots, y.v, y.err + code_step(y, quant), "returned rows")
    want = (got * (w * kept)[..., None]).sum(1)
    size = (got * (w * kept)[..., None]).abs().sum(1)
    R.inside(out, want, size * (k + 4) * R.U32 + R.UBF16 * size * (1 + 2.0 ** -10), "out")

    # balance loss and the router
    lg, im = logits.cpu().numpy(), idx.cpu().numpy()
    mk = None if mask is None else mask.cpu().numpy()
    loss, counts, sums, tokens, prob = R.balance(lg, im, mk, seg, E, k)
    rel = R.softmax_rel_bound(lg, mk, E, T)
    assert np.array_equal(bal.expert_counts.cpu().numpy(), counts) and np.array_equal(bal.tokens.cpu().numpy(), tokens)
    R.inside(bal.loss, torch.as_tensor(loss).cuda(), torch.as_tensor(np.abs(loss) * 2 * rel + 1e-30).cuda(), "loss")
    d = d_out.double()
    d_w = (got * d[:, None]).sum(2) * kept
    d_w_size = (got * d[:, None]).abs().sum(2)
    R.inside(grp.d_w[:T], d_w, d_w_size * (H + 8) * R.U32, "d_w")
    live = np.ones(T, bool) if mk is None else mk != 0
    dl, tol = R.route_grad(prob, im, grp.w[:T].cpu().numpy(), grp.d_w[:T].cpu().numpy(), live, d_loss.cpu().numpy(),
                           counts, tokens, seg, E, k, rel)
    R.inside(d_logits, torch.as_tensor(dl).cuda(), torch.as_tensor(tol).cuda() + 1e-30, "d_logits")

    # the experts and the rows
    dy = V(d[slot_t] * w[slot_t, slot_j, None])
    dy = V(dy.v, R.U32 * dy.v.abs()).bf16()
    dx = zeros(H)
    f64 = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    want_g = {f: V(f64(getattr(grads, f))) for f in grads._fields if getattr(grads, f) is not None}
    for e in range(E):
        r = (e_of == e).nonzero()[:, 0]
        if not len(r):
            continue
        dye, ze, he = dy.rows(r), z.rows(r), h.rows(r)
        dz = through(dye @ wd[e], ze, a).bf16()
        dx.put(r, (dz @ wu[e]).bf16())
        xe = V(x[slot_t[r]].double())
        for f, p, q in (("w_down", dye, he), ("w_up", dz, xe)):
            v = p.v.T @ q.v
            err = p.size().T @ q.err + p.err.T @ q.v.abs() + len(r) * R.U32 * (p.size().T @ q.size())
            want_g[f].v[e], want_g[f].err[e] = v, err
        for f, p in (("b_down", dye), ("b_up", dz)):
            if f in want_g:
                want_g[f].v[e], want_g[f].err[e] = p.v.sum(0), p.err.sum(0) + len(r) * R.U32 * p.size().sum(0)
    for f, v in want_g.items():
        R.inside(getattr(grads, f), v.v, v.err, f)
    want = V(f64(x))
    want.v.index_add_(0, slot_t, dx.v)
    want.err.index_add_(0, slot_t, dx.err + (k + 4) * R.U32 * dx.size())
    want = want.bf16()
    R.inside(d_x, want.v, want.err, "d_x")


@pytest.mark.parametrize("quant", [0, 1])
def test_layer_and_its_gradients_in_a_graph(quant):
    T, H, E, k, Rn = 120, 64, 8, 2, 4
    grp, mlp, x, logits, _, d_out = make(T, H, 48, E, k, Rn, B.MOE_ACT_SWIGLU, quant, True, 0.0)
    bal = B.alloc_balance(T, T, E, k, "cuda")
    d_loss = torch.ones(1, device="cuda")
    grads = mlp.alloc_grads()
    outs = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(logits), *grads, bal.loss]

    def step():
        grp.run(logits, x, outs[0], quant=quant, balance=bal)
        grp.backward(d_out, outs[1], outs[2], grads, d_loss)

    graph = capture(step)
    for s in range(3):
        g = torch.Generator(device="cuda").manual_seed(s)
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        d_out.copy_(torch.randn(T, H, generator=g, device="cuda"))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        first = [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        for p, q in zip(first, outs):
            assert torch.equal(p, q)


def test_accumulating_and_partial_gradients():
    """Twice the gradients of two equal steps; rows or parameters alone."""
    T, H, E, k, Rn = 64, 64, 8, 2, 2
    grp, mlp, x, logits, _, d_out = make(T, H, 32, E, k, Rn, B.MOE_ACT_SILU, 0, True, 0.0)
    out, d_logits = torch.empty_like(x), torch.empty_like(logits)
    one, two = mlp.alloc_grads(), mlp.alloc_grads()
    d_x, d_x2 = torch.empty_like(x), torch.empty_like(x)
    grp.run(logits, x, out)
    grp.backward(d_out, d_x, d_logits, one)
    grp.backward(d_out, None, d_logits, two)
    grp.backward(d_out, d_x2, d_logits, two, accumulate=True)
    grp.backward(d_out, None, d_logits)
    torch.cuda.synchronize()
    assert torch.equal(d_x, d_x2)
    for p, q in zip(one, two):
        assert torch.equal(2 * p, q)


def test_no_tokens():
    """Nothing to do but zero gradients."""
    grp, mlp, x, logits, _, d_out = make(0, 32, 16, 4, 2, 2, B.MOE_ACT_SWIGLU, 0, True, 0.0)
    bal = B.alloc_balance(0, 1, 4, 2, "cuda")
    grads = mlp.alloc_grads()
    for quant in (0, 1):
        for g in grads:
            g.fill_(3.0)
        grp.run(logits, x, torch.empty_like(x), quant=quant, balance=bal)
        grp.backward(d_out, torch.empty_like(x), torch.empty_like(logits), grads, torch.ones(1, device="cuda"))
        torch.cuda.synchronize()
        assert not any(g.any() for g in grads) and bal.loss.item() == 0 and not bal.expert_counts.any()

"""moe_balance_loss and moe_route_grad against their 64-bit forms."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd import inputs as I

pytestmark = pytest.mark.gpu

# T, E, k, seg, masked share
CASES = [(1, 1, 1, 1, 0.0), (1, 8, 2, 1, 0.0), (1, 8, 2, 1, 1.0), (17, 7, 7, 5, 0.3), (256, 8, 2, 256, 0.0),
         (300, 16, 4, 300, 0.2), (257, 17, 3, 64, 0.0), (1000, 33, 16, 999, 0.5), (4096, 64, 8, 4096, 0.1),
         (70, 66, 2, 7, 0.4), (2049, 128, 8, 700, 0.9), (5000, 256, 8, 5000, 0.0), (777, 255, 8, 400, 0.1),
         (3001, 260, 8, 1500, 0.1), (512, 512, 1, 512, 0.0), (1200, 513, 16, 601, 0.2), (999, 1024, 16, 999, 0.0),
         (640, 1023, 5, 64, 1.0), (20000, 64, 4, 1, 0.1),
         (1172, 995, 15, 235, 0.9), (700, 1024, 4, 140, 0.0), (4000, 256, 8, 250, 0.1)]


def draw(T, E, k, masked, seed=0):
    wl = I.Workload("b", T=T, H=16, E=E, k=k, R=1, zipf_s=0.7, seed=seed)
    rng = np.random.default_rng(seed)
    logits = I.make_logits(wl)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    w = np.take_along_axis(logits, idx, axis=1).astype(np.float64)
    w = np.exp(w - w.max(axis=1, keepdims=True))
    w = (w / w.sum(axis=1, keepdims=True)).astype(np.float32)
    mask = None if masked == 0 else (rng.random(T) >= masked).astype(np.uint8)
    d_w = rng.standard_normal((T, k)).astype(np.float32)
    return logits, idx, w, mask, d_w, rng


def adds(T, seg):
    """Terms a lane adds: a block takes at most max(T / 1024 + 16, 256) tokens."""
    return max(-(-T // 1024) + 16, 256)


def run_loss(logits, idx, mask, seg, stream=None):
    T, E = logits.shape
    out = B.alloc_balance(T, seg, E, idx.shape[1], "cuda")
    for t in out[:4]:
        t.fill_(-7)
    return B.moe_balance_loss(R.dev(logits), R.dev(idx), None if mask is None else R.dev(mask), out, stream)


@pytest.mark.parametrize("T,E,k,seg,masked", CASES)
def test_balance_loss(T, E, k, seg, masked):
    logits, idx, _, mask, _, _ = draw(T, E, k, masked)
    if mask is not None:  # padding may hold anything
        logits[mask == 0] = np.nan
        idx[mask == 0] = 2 ** 31 - 1
    out = run_loss(logits, idx, mask, seg)
    torch.cuda.synchronize()
    loss, counts, sums, tokens, _ = R.balance(logits, idx, mask, seg, E, k)
    rel = R.softmax_rel_bound(logits, mask, E, adds(T, seg))
    assert np.array_equal(out.expert_counts.cpu().numpy(), counts)
    assert np.array_equal(out.tokens.cpu().numpy(), tokens)
    R.inside(out.prob_sums.cpu(), sums, sums * rel, "prob_sums")
    R.inside(out.loss.cpu(), loss, loss * (rel + 4 * R.U32), "loss")


@pytest.mark.parametrize("parts", ["both", "gates", "loss"])
@pytest.mark.parametrize("T,E,k,seg,masked", CASES)
def test_route_grad(T, E, k, seg, masked, parts):
    logits, idx, w, mask, d_w, rng = draw(T, E, k, masked, seed=3)
    S = -(-T // seg)
    d_loss = rng.standard_normal(S).astype(np.float32) * np.float32(T / S)
    live = np.ones(T, bool) if mask is None else mask != 0
    rel = R.softmax_rel_bound(logits, mask, E, 0)
    _, counts, _, tokens, p = R.balance(logits, idx, mask, seg, E, k)
    if mask is not None:
        logits[~live] = np.nan
        w[~live], d_w[~live] = np.inf, np.nan
    bal = run_loss(logits, idx, mask, seg)
    d_logits = torch.full((T, E), -7.0, device="cuda")
    gates, loss = parts != "loss", parts != "gates"
    B.moe_route_grad(R.dev(logits) if loss else None, R.dev(idx), R.dev(w) if gates else None,
                     R.dev(d_w) if gates else None, None if mask is None else R.dev(mask),
                     R.dev(d_loss) if loss else None, bal if loss else None, d_logits)
    torch.cuda.synchronize()
    w, d_w = np.where(live[:, None], w, 0), np.where(live[:, None], d_w, 0)
    want, tol = R.route_grad(p, idx, w, d_w if gates else None, live, d_loss if loss else None, counts, tokens,
                             seg, E, k, rel)
    got = d_logits.cpu()
    R.inside(got, want, tol, "d_logits")
    assert not got[torch.from_numpy(~live)].any()


def test_minus_infinity_and_lowest_logits():
    """Experts switched off by -inf or the type's lowest value have probability
    and gradient 0, and leave the others as they are."""
    logits, idx, w, _, d_w, _ = draw(200, 24, 4, 0.0)
    off = np.arange(24) % 3 == 1
    for low in (-np.inf, np.finfo(np.float32).min):
        z = np.where(off, np.float32(low), logits).astype(np.float32)
        ids = np.argsort(-z, axis=1, kind="stable")[:, :4].astype(np.int32)
        bal = run_loss(z, ids, None, 100)
        d_logits = torch.empty(200, 24, device="cuda")
        d_loss = torch.ones(2, device="cuda")
        B.moe_route_grad(R.dev(z), R.dev(ids), None, None, None, d_loss, bal, d_logits)
        torch.cuda.synchronize()
        loss, counts, sums, tokens, p = R.balance(z, ids, None, 100, 24, 4)
        rel = R.softmax_rel_bound(logits, None, 24, 256)
        R.inside(bal.prob_sums.cpu(), sums, sums * rel, "prob_sums")
        R.inside(bal.loss.cpu(), loss, loss * rel + 4 * R.U32 * loss, "loss")
        want, tol = R.route_grad(p, ids, None, None, np.ones(200, bool), np.ones(2), counts, tokens, 100, 24, 4, rel)
        R.inside(d_logits.cpu(), want, tol, "d_logits")
        assert not d_logits.cpu()[:, torch.from_numpy(off)].any()


def test_route_grad_repeated_and_foreign_ids():
    """An id that occurs twice gets both contributions, one outside [0, E) none."""
    _, idx, w, _, d_w, _ = draw(65, 20, 4, 0.0)
    idx[:, 2] = idx[:, 0]
    idx[::2, 3] = -1
    idx[1::2, 3] = 20
    d_logits = torch.empty(65, 20, device="cuda")
    B.moe_route_grad(None, R.dev(idx), R.dev(w), R.dev(d_w), None, None, None, d_logits)
    want, tol = R.route_grad(None, idx, w, d_w, np.ones(65, bool), None, None, None, 65, 20, 4, 0.0)
    R.inside(d_logits.cpu(), want, tol, "d_logits")


def test_unaligned_rows():
    """Arrays on 4-byte boundaries only, in place for the gradient."""
    logits, idx, w, _, d_w, _ = draw(130, 64, 8, 0.0)
    room = torch.empty(130 * 64 + 1, device="cuda")
    z = room[1:].view(130, 64)
    z.copy_(torch.from_numpy(logits))
    bal = B.moe_balance_loss(z, R.dev(idx), None, B.alloc_balance(130, 50, 64, 8, "cuda"))
    _, counts, sums, tokens, p = R.balance(logits, idx, None, 50, 64, 8)
    rel = R.softmax_rel_bound(logits, None, 64, 256)
    R.inside(bal.prob_sums.cpu(), sums, sums * rel, "prob_sums")
    d_loss = np.full(3, 2.0, np.float32)
    B.moe_route_grad(z, R.dev(idx), R.dev(w), R.dev(d_w), None, R.dev(d_loss), bal, z)
    want, tol = R.route_grad(p, idx, w, d_w, np.ones(130, bool), d_loss, counts, tokens, 50, 64, 8, rel)
    R.inside(z.cpu(), want, tol, "d_logits in place")


def test_gradient_agrees_with_differences():
    """The reference's own gradient against central differences of its loss
    (counts held), so that formula and loss belong together."""
    logits, idx, _, _, _, rng = draw(12, 6, 2, 0.0)
    _, counts, _, tokens, p = R.balance(logits, idx, None, 12, 6, 2)
    want, _ = R.route_grad(p, idx, None, None, np.ones(12, bool), np.ones(1), counts, tokens, 12, 6, 2, 0.0)
    h = 1e-4
    for _ in range(20):
        t, e = rng.integers(12), rng.integers(6)
        up, down = logits.astype(np.float64), logits.astype(np.float64)
        up[t, e] += h
        down[t, e] -= h
        slope = (R.balance(up, idx, None, 12, 6, 2)[0] - R.balance(down, idx, None, 12, 6, 2)[0]) / (2 * h)
        # the third derivative of the loss is below E / T: h^2 of it, and 64-bit noise over h
        assert abs(slope[0] - want[t, e]) <= h * h + 1e-15 / h


def test_empty_batch_and_same_bits_twice():
    out = B.alloc_balance(0, 5, 8, 2, "cuda")
    for t in out[:4]:
        t.fill_(-7)
    B.moe_balance_loss(torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"), None, out)
    for t in out[:4]:
        assert not t.any()
    logits, idx, _, _, _, _ = draw(30000, 100, 4, 0.0)
    a, b = run_loss(logits, idx, None, 30000), run_loss(logits, idx, None, 30000)
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x, y)


def test_balance_on_a_stream_and_in_a_graph():
    """Captured once (loss and gradient) and replayed on new logits, with
    eager calls of the same sizes between the replays."""
    T, E, k, seg = 3000, 64, 4, 1000
    sets = [draw(T, E, k, 0.0, seed=s) for s in range(3)]
    z, ids, w, d_w = (R.dev(a) for a in (sets[0][0], sets[0][1], sets[0][2], sets[0][4]))
    d_loss = torch.ones(3, device="cuda")
    bal, grad = B.alloc_balance(T, seg, E, k, "cuda"), torch.empty(T, E, device="cuda")

    def both(bal, grad):
        B.moe_balance_loss(z, ids, None, bal)
        B.moe_route_grad(z, ids, w, d_w, None, d_loss, bal, grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(bal, grad)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(bal, grad)
    bal2, grad2 = B.alloc_balance(T, seg, E, k, "cuda"), torch.empty_like(grad)
    for s in (1, 2, 0, 1):
        for t, a in ((z, sets[s][0]), (ids, sets[s][1]), (w, sets[s][2]), (d_w, sets[s][4])):
            t.copy_(torch.from_numpy(a))
        graph.replay()
        both(bal2, grad2)
        torch.cuda.synchronize()
        assert torch.equal(grad, grad2)
        for a, b in zip(bal[:4], bal2[:4]):
            assert torch.equal(a, b)

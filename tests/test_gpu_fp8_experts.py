"""Experts with E4M3 rows and weights, alone, in a group and between two norms:
every step against its 64-bit form, from what the step before it left."""
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B
from combine_fp32_router_amd.driver import capture
from combine_fp32_router_amd.epgroup import EPGroup
from combine_fp32_router_amd.experts import ExpertMLP8
from test_gpu_fp8_products import GELU, NONE, RELU, SILU, SWIGLU, coded_rows, normal, offsets_of

pytestmark = pytest.mark.gpu


def make(g, E, H, I, act, biases, rows, train):
    wide = 2 if act == SWIGLU else 1
    b = (normal(g, E, wide * I, scale=0.1, dtype=torch.float32), normal(g, E, H, scale=0.1, dtype=torch.float32)) \
        if biases else (None, None)
    return ExpertMLP8(normal(g, E, wide * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5), act, *b,
                      max_rows=rows, train=train)


def rows64(codes, scales, halves=1):
    """Values and peaks of coded rows [rows, halves * n]; scales [rows, halves, blocks],
    [rows, blocks], or one a row."""
    rows, n = codes.shape[0], codes.shape[1] // halves
    if scales.dim() == 1:
        s = scales.double()[:, None].expand(rows, n)
    else:
        s = F.at_columns(scales.view(rows, halves, -1), n).reshape(rows, halves * n)
    return F.e4m3(codes) * s, F.peaks(codes, s)


def weights64(coded, halves):
    codes, scales = coded  # [E, halves * N, K], [E, halves, blocks, blocks]
    E, wide_n, K = codes.shape
    s = scales.view(E * halves, F.blocks(wide_n // halves), -1).double().repeat_interleave(128, 1)
    s = F.at_columns(s[:, :wide_n // halves], K).reshape(E, wide_n, K)
    return F.e4m3(codes) * s, F.peaks(codes, s)


def transposed64(coded, halves):
    codes, scales = coded  # [E, K, halves * N], [E, blocks of K, halves, blocks of N]
    E, K, wide_n = codes.shape
    s = scales.view(E, -1, halves, scales.shape[-1]).double().repeat_interleave(128, 1)[:, :K]
    s = F.at_columns(s, wide_n // halves).reshape(E, K, wide_n)
    return F.e4m3(codes) * s, F.peaks(codes, s)


def half_step(w, codes_of):
    """Half a code's step, by the scale of whose block it is (at most top / 448)."""
    return w.abs() * F.UE4M3 * (1 + 2.0 ** -20) + codes_of * F.LEAST


def check_forward(mlp, coded, off, out, residual):
    n = coded[0].shape[0]
    x64, xp = rows64(*coded)
    y, dy, z, dz, w = F.product(x64, xp, off.tolist(), *weights64(mlp.up8, mlp.wide), mlp.b_up, mlp.act, None)
    h8, hs = mlp.hidden8[0][:n], mlp.hidden8[1][:n]
    F.check_codes(h8[w], hs[w], y[w], dy[w], "hidden")
    if mlp.train:
        R.inside(mlp.hidden[:n][w], y[w], F.bf16(y, dy)[w], "hidden")
        R.inside(mlp.preact[:n][w], z[w], F.bf16(z, dz)[w], "preact")
    h64, hp = rows64(h8, hs)
    h64, hp = torch.where(w[:, None], h64, 0.0), torch.where(w[:, None], hp, 0.0)
    y, dy, *_ = F.product(h64, hp, off.tolist(), *weights64(mlp.down8, 1), mlp.b_down, NONE, residual)
    R.inside(out[w], y[w], F.bf16(y, dy)[w], "out")
    return w


def check_backward(mlp, d_out, x, off, d_x, grads, w):
    """After backward(d_out, x, off, d_x, grads) of copies of them."""
    n, act = x.shape[0], mlp.act
    clean = lambda t: torch.where(w[:, None], t, torch.zeros_like(t))  # noqa: E731
    d8 = [t[:n] for t in mlp.x8]
    F.check_codes(d8[0][w], d8[1][w], d_out.double()[w], 0 * d_out.double()[w], "d_out")
    d64, dp = (clean(t) for t in rows64(*d8))
    z = clean(mlp.preact[:n])
    dz, tol, _ = F.product_dx(d64, dp, off.tolist(), *transposed64(mlp.down8_t, 1), act, z)
    dz8, dzs = (t[:n] for t in mlp.d_preact8)
    if d_x is not None:
        part = lambda t: t[w].view(-1, mlp.wide, mlp.I)  # noqa: E731
        F.check_codes(part(dz8), dzs[w], part(dz), part(tol), "d_preact")
        dz64, dzp = (clean(t) for t in rows64(dz8, dzs, mlp.wide))
        dx, dx_tol, _ = F.product_dx(dz64, dzp, off.tolist(), *transposed64(mlp.up8_t, mlp.wide), NONE, None)
        R.inside(d_x[w], dx[w], F.bf16(dx, dx_tol)[w], "d_x")
    if grads is not None:
        R.inside(mlp.d_preact[:n][w], dz[w], F.bf16(dz, tol)[w], "d_preact")
        dw, tw, db, tb = R.product_dw(clean(d_out), clean(mlp.hidden[:n]), off.tolist(), mlp.E)
        R.inside(grads.w_down, dw, tw, "w_down")
        if grads.b_down is not None:
            R.inside(grads.b_down, db, tb, "b_down")
        dw, tw, db, tb = R.product_dw(clean(mlp.d_preact[:n]), clean(x), off.tolist(), mlp.E)
        R.inside(grads.w_up, dw, tw, "w_up")
        if grads.b_up is not None:
            R.inside(grads.b_up, db, tb, "b_up")


# run lengths, H, I, act, biases, residual, train; what comes in: bf16 rows, codes with a
# scale each 128 or each row
CASES = [([1], 16, 16, NONE, True, True, True, "bf16"), ([1, 0, 3], 128, 272, SWIGLU, True, False, False, "row"),
         ([70, 0, 129, 1], 272, 144, SWIGLU, True, True, True, "block"), ([33, 300], 1040, 528, GELU, False, False, True, "bf16"),
         ([5] * 40, 256, 384, SWIGLU, False, True, False, "bf16"), ([257, 0, 700], 528, 1040, SILU, True, False, True, "row"),
         ([1] * 8 + [0] * 8, 2048, 768, SWIGLU, False, False, False, "row"), ([0, 0], 64, 64, SWIGLU, True, False, True, "block"),
         ([1500, 900], 1024, 2064, SWIGLU, False, False, True, "bf16"), ([40, 2], 64, 80, RELU, True, True, True, "row")]


@pytest.mark.parametrize("lengths,H,I,act,biases,residual,train,kind", CASES,
                         ids=[f"r{sum(c[0])}H{c[1]}I{c[2]}a{c[3]}{c[7]}" for c in CASES])
def test_experts_step_by_step(lengths, H, I, act, biases, residual, train, kind):
    g = torch.Generator(device="cuda").manual_seed(11)
    rows = sum(lengths) + 3  # three of no run
    mlp = make(g, len(lengths), H, I, act, biases, rows, train)
    for w, coded, halves in ((mlp.w_up, mlp.up8, mlp.wide), (mlp.w_down, mlp.down8, 1)):
        got = weights64(coded, halves)[0]
        top = w.double().abs().amax((1, 2), keepdim=True) / 448
        R.inside(got, w.double(), half_step(w.double(), top), "weights")
    off = offsets_of(lengths)
    if kind == "bf16":
        x = normal(g, rows, H)
        given = {}
    else:
        x, xs, x64, _ = coded_rows(g, rows, H, kind == "row")
        given = {"scales": xs}
    res = normal(g, rows, H) if residual else None
    out = torch.full((rows, H), 5.0, dtype=torch.bfloat16, device="cuda")
    mlp.forward(x, off, out, res, **given)
    torch.cuda.synchronize()
    coded = (x, xs) if given else tuple(t[:rows] for t in mlp.x8)
    w = check_forward(mlp, tuple(torch.where(w_like(t, off, rows), t.view(torch.uint8) if t.element_size() == 1 else t,
                                             torch.zeros_like(t.view(torch.uint8) if t.element_size() == 1 else t))
                                 for t in coded), off, out, res)
    assert (out[~w] == 5.0).all()
    if not train:
        assert mlp.hidden is None
        return
    d_out, x16 = normal(g, rows, H), x if kind == "bf16" else x64.bfloat16()
    grads, d_x = mlp.alloc_grads(), torch.full_like(out, 5.0)
    mlp.backward(d_out, x16, off, d_x, grads)
    check_backward(mlp, d_out, x16, off, d_x, grads, w)
    assert (d_x[~w] == 5.0).all()
    # either half of it alone, and in place of d_out: the same bits
    only, again = mlp.alloc_grads(), d_out.clone()
    mlp.backward(d_out, x16, off, None, only)
    mlp.backward(again, x16, off, again, None)
    for p, q in zip(grads, only):
        assert p is None or torch.equal(p, q)
    assert torch.equal(again[w], d_x[w]) and torch.equal(again[~w], d_out[~w])


def w_like(t, off, rows):
    """Which rows are of a run, for a tensor of rows."""
    live = torch.zeros(rows, dtype=torch.bool, device=t.device)
    live[:int(off[-1])] = True
    return live.view(-1, *[1] * (t.dim() - 1))


def test_weights_are_taken_again():
    g = torch.Generator(device="cuda").manual_seed(5)
    mlp = make(g, 2, 64, 48, SILU, False, 20, True)
    other = make(g, 2, 64, 48, SILU, False, 20, True)
    x, off = normal(g, 20, 64), offsets_of([9, 11])
    want, got = torch.empty_like(x), torch.empty_like(x)
    other.forward(x, off, want)
    mlp.forward(x, off, got)
    assert not torch.equal(want, got)
    mlp.w_up.copy_(other.w_up), mlp.w_down.copy_(other.w_down)
    mlp.quantize()
    mlp.forward(x, off, got)
    assert torch.equal(want, got)
    d_want, d_got = torch.empty_like(x), torch.empty_like(x)
    other.backward(x, x, off, d_want, None), mlp.backward(x, x, off, d_got, None)
    assert torch.equal(d_want, d_got)


# T, H, I, E, k, R, act, payload, train
GROUPS = [(96, 64, 48, 8, 2, 4, SWIGLU, 3, True), (257, 144, 96, 16, 4, 8, GELU, 3, True), (200, 96, 64, 8, 2, 2, SWIGLU, 3, False),
          (150, 128, 80, 8, 3, 4, SWIGLU, 0, True), (150, 64, 80, 8, 3, 1, SILU, 1, True), (1, 2048, 768, 32, 8, 1, SWIGLU, 3, False),
          (3, 16, 16, 8, 1, 8, NONE, 3, True)]


@pytest.mark.parametrize("T,H,I,E,k,Rn,act,quant,train", GROUPS)
def test_group(T, H, I, E, k, Rn, act, quant, train):
    g = torch.Generator(device="cuda").manual_seed(3)
    mlp = make(g, E, H, I, act, True, Rn * -(-T // Rn) * k, train)
    grp = EPGroup(T, H, E, k, Rn, experts=mlp)
    x, logits = normal(g, T, H), normal(g, T, E, dtype=torch.float32)
    out = torch.empty_like(x)
    grp.run(logits, x, out, quant=quant)
    torch.cuda.synchronize()
    off, M = grp.rl.group_offsets[:E + 1], grp.max_rows
    live = int(off[-1])
    assert live == T * k
    # the experts' rows: the tokens', by the row maps
    if quant == 3:
        coded = (grp.grouped.view(-1)[:M * H].view(M, H)[:live], grp.grouped_scales[:live])
        came = F.e4m3(coded[0]) * coded[1].double()[:, None]
        if train:
            R.inside(grp.expert_in[:live], came, F.bf16(came, came.abs() * R.U32), "rows for the gradients")
    else:
        coded = tuple(t[:live] for t in mlp.x8)
        came = grp.expert_in[:live].double()
        F.check_codes(*coded, came, 0 * came, "rows")
    order = grp.idx[:T].long().view(-1).argsort(stable=True)  # grouped order of one batch of all tokens
    sent = x.double()[order // k]
    top = sent.abs().amax(1, keepdim=True)
    step = {0: 0 * sent, 1: (top / 127 * 0.5).expand_as(sent), 3: half_step(sent, top / 448)}[quant]
    R.inside(came, sent, step * (1 + 2.0 ** -10) + (R.UBF16 * 1.01 * sent.abs() if quant == 1 else 0), "rows that came")
    sub = torch.zeros(M, dtype=torch.bool, device="cuda")
    sub[:live] = True
    check_forward(mlp, coded, off, grp.expert_out[:live], None)
    # back to the tokens
    y = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
    y[order] = grp.expert_out[:live].double()
    top = y.abs().amax(1, keepdim=True)
    step = {0: 0 * y, 1: (top / 127 * 0.5).expand_as(y), 3: half_step(y, top / 448)}[quant] * (1 + 2.0 ** -10)
    w = grp.w[:T].double()[..., None]
    want, tol = (y.view(T, k, H) * w).sum(1), (step.view(T, k, H) * w).sum(1)
    size = ((y.abs() + step).view(T, k, H) * w).sum(1)
    R.inside(out, want, F.bf16(want, tol + (k + 4) * R.U32 * size), "out")
    if not train:
        return
    d_out, d_x, d_logits = normal(g, T, H), torch.empty_like(x), torch.empty_like(logits)
    grads = mlp.alloc_grads()
    grp.backward(d_out, d_x, d_logits, grads)
    torch.cuda.synchronize()
    d_rows = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
    d_rows = (d_out.double()[:, None] * w).reshape(T * k, H)[order]
    got = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
    d8 = F.e4m3(mlp.x8[0][:live]) * F.at_columns(mlp.x8[1][:live], H)
    R.inside(d8, d_rows, half_step(d_rows, d_rows.abs().amax(1, keepdim=True) / 448) * 1.01 + 1.1 * R.UBF16 * d_rows.abs(),
             "rows' gradients")
    d_rows16 = d_rows.bfloat16()  # (as the combine's gradient rounds it, but for ties of its fp32 product)
    got[order] = grp.d_rows[:live].double()
    want = got.view(T, k, H).sum(1)
    R.inside(d_x, want, F.bf16(want, (k + 4) * R.U32 * got.view(T, k, H).abs().sum(1)), "d_x")
    off_cpu = off.tolist()
    dz, tol, _ = F.product_dx(*(rows64(*[t[:live] for t in mlp.x8])), off_cpu, *transposed64(mlp.down8_t, 1), act, mlp.preact[:live])
    R.inside(mlp.d_preact[:live], dz, F.bf16(dz, tol), "d_preact")
    dx, tol, _ = F.product_dx(*rows64(mlp.d_preact8[0][:live], mlp.d_preact8[1][:live], mlp.wide), off_cpu,
                              *transposed64(mlp.up8_t, mlp.wide), NONE, None)
    R.inside(grp.d_rows[:live], dx, F.bf16(dx, tol), "rows' d_x")
    dw, tw, _, _ = R.product_dw(mlp.d_preact[:live], grp.expert_in[:live], off_cpu, E)
    R.inside(grads.w_up, dw, tw, "w_up")
    dw, tw, _, _ = R.product_dw(d_rows16, mlp.hidden[:live], off_cpu, E)
    tie = R.product_dw(d_rows16.abs(), mlp.hidden[:live].abs(), off_cpu, E)[0] * 2 * R.UBF16  # (a tie's other side)
    R.inside(grads.w_down, dw, tw + tie, "w_down")


@pytest.mark.parametrize("quant", [0, 1, 3])
def test_no_tokens(quant):
    """Nothing to do but zero gradients."""
    g = torch.Generator(device="cuda").manual_seed(4)
    mlp = make(g, 4, 32, 16, SWIGLU, True, 0, True)
    grp = EPGroup(0, 32, 4, 2, 2, experts=mlp)
    x, logits = normal(g, 0, 32), normal(g, 0, 4, dtype=torch.float32)
    grads = mlp.alloc_grads()
    for t in grads:
        t.fill_(3.0)
    grp.run(logits, x, torch.empty_like(x), quant=quant)
    grp.backward(x, torch.empty_like(x), torch.empty_like(logits), grads)
    torch.cuda.synchronize()
    assert not any(t.any() for t in grads)


def block(mlp, x, res, w1, w2, off, room):
    """norm -> codes -> experts with the residual -> norm, and all of it back from
    d_y: as a block of a network has them."""
    T, H = x.shape
    s, y, c, v, h, s2, y2 = room["forward"]
    B.moe_add_norm(x, res, w1, 1e-5, s, y, c, v)
    mlp.forward(c, off, h, scales=v)
    B.moe_add_norm(h, s, w2, 1e-5, s2, y2)
    d_y2, d_h, d_y, d_x, dw1, dw2, grads = room["backward"]
    B.moe_add_norm_grad(d_y2, None, s2, w2, 1e-5, d_h, dw2)
    mlp.backward(d_h, y, off, d_y, grads)
    B.moe_add_norm_grad(d_y, d_h, s, w1, 1e-5, d_x, dw1)


def block_room(mlp, g, T, H):
    rows = lambda: torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    codes = torch.zeros(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros(T, F.blocks(H), device="cuda")
    f = lambda: torch.zeros(H, device="cuda")  # noqa: E731
    return {"forward": (rows(), rows(), codes, v, rows(), rows(), rows()),
            "backward": (normal(g, T, H), rows(), rows(), rows(), f(), f(), mlp.alloc_grads())}


@pytest.mark.parametrize("T,H,I,act", [(1, 64, 32, SWIGLU), (77, 272, 144, SWIGLU), (600, 528, 1040, GELU)])
def test_between_two_norms(T, H, I, act):
    g = torch.Generator(device="cuda").manual_seed(T)
    mlp = make(g, 1, H, I, act, True, T, True)
    x, res, off = normal(g, T, H), normal(g, T, H, scale=2.0), offsets_of([T])
    w1, w2 = normal(g, H, dtype=torch.float32), normal(g, H, dtype=torch.float32)
    room = block_room(mlp, g, T, H)
    block(mlp, x, res, w1, w2, off, room)
    torch.cuda.synchronize()
    s, y, c, v, h, s2, y2 = room["forward"]
    d_y2, d_h, d_y, d_x, dw1, dw2, grads = room["backward"]
    want_s, want_y, tol = F.norm(x, res, w1, 1e-5)
    R.inside(s, want_s, F.bf16(want_s, 0 * want_s), "sum")
    R.inside(y, want_y, F.bf16(want_y, tol), "y")
    F.check_codes(c, v, want_y, tol, "y")
    w = check_forward(mlp, (c, v), off, h, None)
    want_s, want_y, tol = F.norm(h, s, w2, 1e-5)
    R.inside(s2, want_s, F.bf16(want_s, 0 * want_s), "second sum")
    R.inside(y2, want_y, F.bf16(want_y, tol), "second y")
    want, tol, want_w, tol_w = F.norm_grad(d_y2, None, s2, w2, 1e-5)
    R.inside(d_h, want, F.bf16(want, tol), "d_h")
    R.inside(dw2, want_w, tol_w, "d_weight")
    check_backward(mlp, d_h, y, off, d_y, grads, w)
    want, tol, want_w, tol_w = F.norm_grad(d_y, d_h, s, w1, 1e-5)
    R.inside(d_x, want, F.bf16(want, tol), "d_x")
    R.inside(dw1, want_w, tol_w, "d_weight of the first")


def test_between_two_norms_in_a_graph():
    """Replays with the program's own work between them, and other inputs."""
    T, H, I = 200, 272, 144
    g = torch.Generator(device="cuda").manual_seed(9)
    mlp, mine = make(g, 1, H, I, SWIGLU, True, T, True), torch.Generator(device="cuda")
    x, res, off = normal(g, T, H), normal(g, T, H), offsets_of([T])
    w1, w2 = normal(g, H, dtype=torch.float32), normal(g, H, dtype=torch.float32)
    room = block_room(mlp, g, T, H)
    graph = capture(lambda: block(mlp, x, res, w1, w2, off, room))
    outs = [t for t in (*room["forward"], *room["backward"][1:6], *room["backward"][6]) if t is not None]
    outs = [t.view(torch.uint8) if t.element_size() == 1 else t for t in outs]
    for seed in range(3):
        mine.manual_seed(seed)
        x.copy_(normal(mine, T, H)), res.copy_(normal(mine, T, H))
        room["backward"][0].copy_(normal(mine, T, H))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        first = [o.clone() for o in outs]
        block(mlp, x, res, w1, w2, off, room)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, outs))


def test_two_layers_on_two_streams():
    """Two experts' calls at once, each with its own buffers and stream: what each
    gives alone."""
    g = torch.Generator(device="cuda").manual_seed(13)
    layers = [make(g, 4, 528, 272, SWIGLU, True, 900, True) for _ in range(2)]
    x, off = normal(g, 900, 528), offsets_of([300, 0, 599, 1])
    want, got = [torch.empty_like(x) for _ in layers], [torch.empty_like(x) for _ in layers]
    d_want, d_got = [torch.empty_like(x) for _ in layers], [torch.empty_like(x) for _ in layers]
    for m, o, d in zip(layers, want, d_want):
        m.forward(x, off, o), m.backward(x, x, off, d, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(4):
        for m, o, d, s in zip(layers, got, d_got, streams):
            m.forward(x, off, o, stream=s), m.backward(x, x, off, d, None, stream=s)
    torch.cuda.synchronize()
    for p, q in zip(want + d_want, got + d_got):
        assert torch.equal(p, q)

"""Cases for measuring the layer's training and expert operators: the router's balance loss with the router's
gradient, the combine's gradient, the experts' products and the experts' gradients.

Each case runs either in plain torch operations (`own` false) or through the package's calls (`own` true) on
the same inputs.  Rows and weights are bf16, router tensors and weight gradients fp32."""
import math
import random

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "swiglu")  # in the order of the package's MOE_ACT_* codes
QUANTS = ("bf16", "int8")  # payloads of the rows that the combine's gradient reads


def listed():
    return [
        # one short sequence through a small router: latency alone counts
        dict(name="balance 256x8", op="balance", tokens=256, experts=8, k=2, seg=256, masked=0.0),
        # a training batch of four sequences, padded at random places
        dict(name="balance 16384x256 masked", op="balance", tokens=16384, experts=256, k=8, seg=4096, masked=0.1),
        # a long batch as one segment over many experts
        dict(name="balance 131072x512", op="balance", tokens=131072, experts=512, k=8, seg=131072, masked=0.0),
        # a short odd batch with a capacity that drops slots
        dict(name="combine grad 33x528", op="combine_grad", tokens=33, hidden=528, k=3, quant="bf16", dropped=0.2),
        # one chunk of a batch whose rows came back as int8 codes
        dict(name="combine grad 4096x2048 int8", op="combine_grad", tokens=4096, hidden=2048, k=8, quant="int8", dropped=0.1),
        # a large chunk of wide bf16 rows
        dict(name="combine grad 8192x7168", op="combine_grad", tokens=8192, hidden=7168, k=8, quant="bf16", dropped=0.0),
        # serving: one token at its eight experts, one row each, of the 32 a GPU holds
        dict(name="product 1 token", op="product", rows=8, experts=32, inner=7168, outer=2048, act="swiglu",
             bias=False, residual=False, keep=False, spread="single"),
        # an uneven batch over many experts: down projection with bias and residual
        dict(name="product 4099 rows of 64", op="product", rows=4099, experts=64, inner=1024, outer=4096, act="none",
             bias=True, residual=True, keep=False, spread="uneven"),
        # training: gated up projection of a large batch, its pre-activations kept
        dict(name="product 16384x7168", op="product", rows=16384, experts=8, inner=7168, outer=2048, act="swiglu",
             bias=False, residual=False, keep=True, spread="uneven"),
        # a short odd batch through the gradients of a small product with bias
        dict(name="gradient 515x272", op="gradient", rows=515, experts=8, inner=272, outer=512, act="gelu",
             bias=True, spread="uneven"),
        # one chunk's gradients at the experts of a narrow model
        dict(name="gradient 8192x768", op="gradient", rows=8192, experts=8, inner=768, outer=2048, act="swiglu",
             bias=False, spread="uneven"),
        # gradients of the down projection for a large batch
        dict(name="gradient 16384x2048", op="gradient", rows=16384, experts=8, inner=2048, outer=7168, act="swiglu",
             bias=False, spread="uneven"),
    ]


def _log_int(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("balance", "combine_grad", "product", "product", "gradient"))
    if op == "balance":
        experts = _log_int(rng, 4, 1024)
        tokens = _log_int(rng, 1, min(131072, 131072 * 512 // experts))
        seg = tokens if rng.random() < 0.5 else max(1, -(-tokens // rng.randint(2, 9)))
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, min(experts, 16)), seg=seg,
                    masked=rng.choice((0.0, 0.0, 0.15, 0.9)))
    if op == "combine_grad":
        hidden, k = _log_int(rng, 16, 8192, 16), rng.randint(1, 16)
        tokens = _log_int(rng, 1, 8192 * 7168 * 8 // (hidden * k) if hidden * k > 65536 else 32768)
        return dict(op=op, tokens=tokens, hidden=hidden, k=k, quant=rng.choice(QUANTS), dropped=rng.choice((0.0, 0.1, 0.5)))
    experts, inner, outer = _log_int(rng, 1, 64), _log_int(rng, 32, 8192, 16), _log_int(rng, 32, 8192, 16)
    act = rng.choice(ACTS)
    rows = _log_int(rng, 1, 16384)
    wide = 2 if op == "product" and act == "swiglu" else 1
    if op == "gradient":
        while rows * inner * outer > 16384 * 2048 * 7168 or experts * inner * outer > 8 * 2048 * 7168:
            rows, experts, outer = (rows + 1) // 2, (experts + 1) // 2, max(32, outer // 32 * 16)
    while rows * inner * outer * wide > 16384 * 7168 * 2048 * 2 or experts * inner * outer * wide > 32 * 7168 * 2048 * 2:
        rows, experts = (rows + 1) // 2, (experts + 1) // 2
    more = dict(bias=rng.random() < 0.5, spread="uneven" if rows > experts or rng.random() < 0.5 else "single")
    if op == "product":
        more.update(residual=rng.random() < 0.5, keep=rng.random() < 0.5)
    return dict(op=op, rows=rows, experts=experts, inner=inner, outer=outer, act=act, **more)


def _row_counts(case, seed):
    """Rows of each expert's run, a list that sums to `rows`: one row each for the first few experts of a shuffle
    ("single"), or drawn with uneven odds ("uneven"; a few experts get none)."""
    rng = random.Random(seed)
    experts, rows = case["experts"], case["rows"]
    if case["spread"] == "single":
        took = set(rng.sample(range(experts), rows))
        return [int(e in took) for e in range(experts)]
    odds = [math.exp(0.7 * rng.gauss(0, 1)) * (rng.random() > 0.05) + 1e-9 for _ in range(experts)]
    counts = [int(rows * o / sum(odds)) for o in odds]
    counts[rng.randrange(experts)] += rows - sum(counts)
    return counts


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        out = torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)
        return out.mul_(scale) if scale != 1.0 else out

    s = dict(case=case, kept={})
    if case["op"] == "balance":
        T, E, k, seg = case["tokens"], case["experts"], case["k"], case["seg"]
        S = -(-T // seg)
        favour = -0.5 * torch.arange(1, E + 1, dtype=torch.float32, device=dev).log()
        s["logits"] = normal(T, E, dtype=torch.float32) + favour
        top = s["logits"].topk(k, dim=1)
        s["idx"], s["w"] = top.indices.int(), top.values.softmax(1)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = (torch.rand(T, generator=g, device=dev) >= case["masked"]).to(torch.uint8)
        s["d_w"] = normal(T, k, scale=1e-3 / T, dtype=torch.float32)
        s["d_loss"] = torch.full((S,), 0.01 / S, device=dev)
        s["d_logits"] = torch.zeros(T, E, device=dev)
    elif case["op"] == "combine_grad":
        T, H, k = case["tokens"], case["hidden"], case["k"]
        kept = torch.rand(T * k, generator=g, device=dev) >= case["dropped"]
        order = torch.randperm(T * k, generator=g, device=dev)
        slots = order[kept[order]]  # slot held by each row
        n = slots.numel()
        s["pos"] = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
        s["pos"][slots] = torch.arange(n, dtype=torch.int32, device=dev)
        s["row_src"] = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
        s["row_src"][:n] = slots.int()
        s["w"] = torch.rand(T, k, generator=g, device=dev).add_(0.05)
        s["w"] /= s["w"].sum(1, keepdim=True)
        s["d_out"] = normal(T, H, scale=1e-2)
        rows = normal(T * k, H, dtype=torch.bfloat16 if case["quant"] == "bf16" else torch.float32)
        s["scales"] = None
        if case["quant"] == "int8":
            s["scales"] = rows.abs().amax(1) / 127
            rows = (rows / s["scales"][:, None]).round_().clamp_(-127, 127).to(torch.int8)
        s["rows"] = rows
        s["d_rows"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device=dev)
        s["d_w"] = torch.zeros(T, k, device=dev)
    else:
        E, K, N, rows = case["experts"], case["inner"], case["outer"], case["rows"]
        counts = _row_counts(case, seed)
        s["counts"] = counts
        s["offsets"] = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device=dev)
        wide = 2 if case["act"] == "swiglu" else 1
        if case["op"] == "product":
            s["x"] = normal(rows, K)
            s["weight"] = normal(E, wide * N, K, scale=K ** -0.5)
            s["bias"] = normal(E, wide * N, scale=0.1, dtype=torch.float32) if case["bias"] else None
            s["residual"] = normal(rows, N) if case["residual"] else None
            s["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=dev)
            s["preact"] = torch.zeros(rows, wide * N, dtype=torch.bfloat16, device=dev) if case["keep"] else None
        else:
            s["dy"] = normal(rows, N, scale=1e-2)
            s["weight"] = normal(E, N, K, scale=K ** -0.5)
            s["preact"] = normal(rows, wide * K) if case["act"] != "none" else None
            s["x"] = normal(rows, K)
            s["dx"] = torch.zeros(rows, wide * K, dtype=torch.bfloat16, device=dev)
            s["dw"] = torch.zeros(E, N, K, device=dev)
            s["db"] = torch.zeros(E, N, device=dev) if case["bias"] else None
    return s


def run(s):
    if own:
        return _own[s["case"]["op"]](s)
    return _plain[s["case"]["op"]](s)


# ---- the package's calls


def _own_balance(s):
    from combine_fp32_router_amd import binding as B

    c = s["case"]
    if "balance" not in s["kept"]:
        s["kept"]["balance"] = B.alloc_balance(c["tokens"], c["seg"], c["experts"], c["k"], s["logits"].device)
    b = B.moe_balance_loss(s["logits"], s["idx"], s["mask"], s["kept"]["balance"])
    B.moe_route_grad(s["logits"], s["idx"], s["w"], s["d_w"], s["mask"], s["d_loss"], b, s["d_logits"])
    return dict(loss=b.loss, counts=b.expert_counts, prob_sums=b.prob_sums, tokens=b.tokens, d_logits=s["d_logits"])


def _own_combine_grad(s):
    from combine_fp32_router_amd import binding as B

    c = s["case"]
    B.moe_combine_grad(s["d_out"], s["rows"], s["scales"], QUANTS.index(c["quant"]), s["pos"], s["w"], c["tokens"],
                       c["hidden"], c["k"], s["d_rows"], s["d_w"])
    return dict(d_rows=s["d_rows"], d_w=s["d_w"])


def _own_product(s):
    from combine_fp32_router_amd import binding as B

    B.moe_expert_matmul(s["x"], s["offsets"], s["weight"], s["bias"], ACTS.index(s["case"]["act"]), s["residual"],
                        s["out"], s["preact"])
    return dict(out=s["out"], preact=s["preact"])


def _own_gradient(s):
    from combine_fp32_router_amd import binding as B

    B.moe_expert_matmul_dx(s["dy"], s["offsets"], s["weight"], ACTS.index(s["case"]["act"]), s["preact"], s["dx"])
    B.moe_expert_matmul_dw(s["dy"], s["x"], s["offsets"], s["dw"], s["db"])
    return dict(dx=s["dx"], dw=s["dw"], db=s["db"])


# ---- the plain forms, in 32 bits, rounded once


def _plain_balance(s):
    c, logits = s["case"], s["logits"]
    T, E, k, seg = c["tokens"], c["experts"], c["k"], c["seg"]
    S = -(-T // seg)
    live = torch.ones(T, dtype=torch.uint8, device=logits.device) if s["mask"] is None else s["mask"]
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * live[:, None]
    prob_sums = torch.nn.functional.pad(p, (0, 0, 0, S * seg - T)).view(S, seg, E).sum(1)
    part = torch.arange(T, device=logits.device) // seg
    tokens = torch.zeros(S, dtype=torch.int32, device=logits.device).scatter_add_(0, part, live.int())
    counts = torch.zeros(S * E, dtype=torch.int32, device=logits.device)
    counts.scatter_add_(0, (part[:, None] * E + s["idx"]).view(-1), live.int()[:, None].expand(T, k).reshape(-1))
    counts = counts.view(S, E)
    scale = E / (k * tokens.float().clamp(min=1) ** 2)
    loss = scale * (counts * prob_sums).sum(1)
    load = counts[part].float()
    d = (s["d_loss"] * scale)[part][:, None] * p * (load - (load * p).sum(1, keepdim=True))
    d_gate = s["w"] * (s["d_w"] - (s["w"] * s["d_w"]).sum(1, keepdim=True)) * live[:, None]
    d = d.scatter_add(1, s["idx"].long(), d_gate)
    return dict(loss=loss, counts=counts, prob_sums=prob_sums, tokens=tokens, d_logits=d)


def _plain_combine_grad(s):
    c = s["case"]
    T, H, k = c["tokens"], c["hidden"], c["k"]
    kept = s["pos"].view(T, k) >= 0
    at = s["pos"].clamp(min=0).long()
    rows = s["rows"][at].float()
    if s["scales"] is not None:
        rows *= s["scales"][at][:, None]
    d_out = s["d_out"].float()
    d_w = (rows.view(T, k, H) * d_out[:, None, :]).sum(2) * kept
    src = s["row_src"].clamp(min=0).long()
    d_rows = d_out[src // k] * (s["w"].view(-1)[src] * (s["row_src"] >= 0))[:, None]
    return dict(d_rows=d_rows.bfloat16(), d_w=d_w)


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _act_gradient(z, g, act):
    """What a gradient g of act(z) gives for z."""
    if act == "relu":
        return g * (z > 0)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return g * sig * (1 + z * (1 - sig))
    if act == "gelu":
        return g * (0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        sig = 1 / (1 + torch.exp(-gate))
        return torch.cat([g * up * sig * (1 + gate * (1 - sig)), g * gate * sig], dim=1)
    return g


def _plain_product(s):
    parts = zip(s["x"].split(s["counts"]), s["weight"], [None] * len(s["counts"]) if s["bias"] is None else s["bias"])
    z = torch.cat([_affine(x.float(), w, b) for x, w, b in parts if len(x)])
    out = _act(z, s["case"]["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return dict(out=out.bfloat16(), preact=None if s["preact"] is None else z.bfloat16())


def _affine(x, w, b):
    z = x @ w.float().t()
    return z if b is None else z + b


def _plain_gradient(s):
    parts = list(zip(s["dy"].split(s["counts"]), s["x"].split(s["counts"]), s["weight"]))
    dx = torch.cat([d.float() @ w.float() for d, _, w in parts if len(d)])
    if s["preact"] is not None:
        dx = _act_gradient(s["preact"].float(), dx, s["case"]["act"])
    dw = torch.stack([d.float().t() @ x.float() for d, x, _ in parts])
    db = None if s["db"] is None else torch.stack([d.float().sum(0) for d, _, _ in parts])
    return dict(dx=dx.bfloat16(), dw=dw, db=db)


_own = dict(balance=_own_balance, combine_grad=_own_combine_grad, product=_own_product, gradient=_own_gradient)
_plain = dict(balance=_plain_balance, combine_grad=_plain_combine_grad, product=_plain_product,
              gradient=_plain_gradient)


# ---- what one pass cannot do without


def work(case):
    if case["op"] == "balance":
        T, E, k = case["tokens"], case["experts"], case["k"]
        S = -(-T // case["seg"])
        return dict(bytes=8 * T * E + 12 * T * k + T + 8 * S * E, flops=16 * T * E)
    if case["op"] == "combine_grad":
        T, H, k = case["tokens"], case["hidden"], case["k"]
        rows = T * k * (1 - case["dropped"])
        return dict(bytes=int(2 * T * H + rows * H * (2 + (2 if case["quant"] == "bf16" else 1)) + 12 * T * k),
                    flops=int(3 * rows * H))
    E, K, N, rows = case["experts"], case["inner"], case["outer"], case["rows"]
    wide = 2 if case["act"] == "swiglu" else 1
    weights = 2 * min(E, rows) * K * N
    if case["op"] == "product":
        moved = wide * weights + 2 * rows * (K + N) + 2 * rows * N * (case["residual"] + wide * case["keep"])
        return dict(bytes=moved, flops=2 * rows * K * N * wide)
    moved = weights + 4 * E * K * N + 2 * rows * (N + K) + 2 * rows * wide * K * (1 if case["act"] == "none" else 2)
    return dict(bytes=moved, flops=4 * rows * K * N)


# ---- the same from the definitions, in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(s, case)
    if case["op"] == "combine_grad":
        return _exact_combine_grad(s, case)
    bounds = [(e, sum(s["counts"][:e]), sum(s["counts"][:e + 1])) for e in range(case["experts"])]
    return (_exact_product if case["op"] == "product" else _exact_gradient)(s, case, bounds)


def _exact_balance(s, case):
    E, k, seg = case["experts"], case["k"], case["seg"]
    losses, counts, sums, live, grads = [], [], [], [], []
    for n, at in enumerate(range(0, case["tokens"], seg)):
        logits = s["logits"][at:at + seg].double()
        on = torch.ones(len(logits), dtype=torch.float64, device=logits.device)
        if s["mask"] is not None:
            on = s["mask"][at:at + seg].double()
        p = torch.softmax(logits, dim=1)
        ids = s["idx"][at:at + seg].long()
        c = torch.bincount(ids[on > 0].view(-1), minlength=E).double()
        mean, m = on @ p, on.sum().clamp(min=1)
        losses.append(E * (c / (k * m)) @ (mean / m))
        w, d_w = s["w"][at:at + seg].double(), s["d_w"][at:at + seg].double()
        # softmax's Jacobian, of the loss's slope c over all experts and of d_w over the chosen ones
        slope = s["d_loss"][n].double() * E * c / (k * m * m)
        d = p * slope - p * (p @ slope)[:, None]
        gate = w * d_w - w * (w * d_w).sum(1, keepdim=True)
        grads.append(on[:, None] * d.scatter_add(1, ids, gate))
        counts.append(c)
        sums.append(mean)
        live.append(on.sum())
    return dict(loss=torch.stack(losses), counts=None, prob_sums=torch.stack(sums), tokens=None,
                d_logits=torch.cat(grads))


def _exact_combine_grad(s, case):
    T, H, k = case["tokens"], case["hidden"], case["k"]
    d_out, w = s["d_out"].double(), s["w"].double()
    d_w = torch.zeros(T, k, dtype=torch.float64, device=w.device)
    d_rows = torch.zeros(T * k, H, dtype=torch.float64, device=w.device)
    for j in range(k):
        at = s["pos"].view(T, k)[:, j].long()
        t = (at >= 0).nonzero()[:, 0]
        rows = s["rows"][at[t]].double()
        if s["scales"] is not None:
            rows = rows * s["scales"][at[t]].double()[:, None]
        d_w[t, j] = torch.linalg.vecdot(rows, d_out[t])
        d_rows[at[t]] = d_out[t] * w[t, j, None]
    return dict(d_rows=d_rows, d_w=d_w)


def _exact_product(s, case, bounds):
    wide = 2 if case["act"] == "swiglu" else 1
    z = torch.zeros(case["rows"], wide * case["outer"], dtype=torch.float64, device=s["x"].device)
    for e, a, b in bounds:
        if b > a:
            z[a:b] = s["x"][a:b].double() @ s["weight"][e].double().T
            if s["bias"] is not None:
                z[a:b] += s["bias"][e].double()
    if case["act"] == "swiglu":
        y = torch.nn.functional.silu(z[:, :case["outer"]]) * z[:, case["outer"]:]
    else:
        y = dict(none=lambda v: v, relu=torch.relu, silu=torch.nn.functional.silu,
                 gelu=torch.nn.functional.gelu)[case["act"]](z)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return dict(out=y, preact=None if s["preact"] is None else z)


def _exact_gradient(s, case, bounds):
    E, K, N = case["experts"], case["inner"], case["outer"]
    dev = s["x"].device
    g = torch.zeros(case["rows"], K, dtype=torch.float64, device=dev)
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=dev)
    db = torch.zeros(E, N, dtype=torch.float64, device=dev)
    for e, a, b in bounds:
        if b > a:
            d = s["dy"][a:b].double()
            g[a:b] = d @ s["weight"][e].double()
            dw[e] = d.T @ s["x"][a:b].double()
            db[e] = d.sum(0)
    if s["preact"] is not None:
        z = s["preact"].double().requires_grad_()
        with torch.enable_grad():
            if case["act"] == "swiglu":
                y = torch.nn.functional.silu(z[:, :K]) * z[:, K:]
            else:
                y = dict(relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)[case["act"]](z)
            g, = torch.autograd.grad(y, z, g)
    return dict(dx=g, dw=dw, db=None if s["db"] is None else db)

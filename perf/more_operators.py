"""Cases for measuring the layer's operators around E4M3 rows: the residual's addition with the root-mean-square norm
and its gradient, rows and weights in E4M3 codes with a scale for each block of 128, the experts' products of such
rows and weights (alone, and two with the codes of the rows between them), and the gradient of their rows.

Each case runs either in plain torch operations (`own` false) or through the package's calls (`own` true) on the same
inputs.  A block's scale is its largest size / 448, a code is E4M3(value / scale).  The norm's and the quantisers' codes are
returned as E4M3 values (torch's float8_e4m3fn), with their fp32 scales beside them; a product's codes go into the next."""
import math
import random

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "swiglu")  # in the order of the package's MOE_ACT_* codes
BLOCK = 128
EPS = 1e-6


def listed():
    return [
        # serving: one token on its way into a layer's 8-bit products; latency alone counts
        dict(name="norm 1x7168", op="norm", tokens=1, hidden=7168, residual=True, y=False, codes="block"),
        # a short odd batch whose last block is short too, bf16 for the router and codes for the products
        dict(name="norm 33x528", op="norm", tokens=33, hidden=528, residual=True, y=True, codes="row"),
        # a training batch: sum, normed rows and their codes
        dict(name="norm 16384x7168", op="norm", tokens=16384, hidden=7168, residual=True, y=True, codes="block"),
        # gradients of a short odd batch
        dict(name="norm grad 515x2048", op="norm_grad", tokens=515, hidden=2048, stream=True),
        # gradients of a training batch
        dict(name="norm grad 16384x7168", op="norm_grad", tokens=16384, hidden=7168, stream=True),
        # one chunk's gradient rows on their way into a product
        dict(name="codes of rows 4099x7168", op="quant_rows", rows=4099, hidden=7168, halves=1),
        # after a training step: the gated up projections of eight experts, for the product and for its gradient
        dict(name="codes of weights 8x4096x7168", op="quant_weights", experts=8, outer=2048, inner=7168, halves=2),
        # serving: one token at its eight experts, one row each, of the 32 a GPU holds, rows as a payload brought them;
        # the gated up projection, and the down projection of its codes
        dict(name="products 1 token", op="product", rows=8, experts=32, inner=7168, outer=2048, act="swiglu", bias=False,
             residual=False, keep=False, scales="row", then=7168, spread="single"),
        # an uneven batch over many experts: down projection with bias and residual
        dict(name="product 4099 rows of 64", op="product", rows=4099, experts=64, inner=1024, outer=4096, act="none",
             bias=True, residual=True, keep=False, scales="block", then=0, spread="uneven"),
        # training: both projections of a large batch, pre-activations kept
        dict(name="products 16384x7168", op="product", rows=16384, experts=8, inner=7168, outer=2048, act="swiglu",
             bias=False, residual=False, keep=True, scales="block", then=7168, spread="uneven"),
        # a short odd batch through the gradient of a small product
        dict(name="gradient 515x272", op="gradient", rows=515, experts=8, inner=272, outer=512, act="gelu", halves=1,
             then=0, spread="uneven"),
        # gradients of a large batch's rows through the down projection and the gate, and on through the up projection
        dict(name="gradients 16384x2048", op="gradient", rows=16384, experts=8, inner=2048, outer=7168, act="swiglu",
             halves=1, then=7168, spread="uneven"),
    ]


def _log_int(rng, low, high, step=1):
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "quant_rows", "quant_weights", "product", "product", "product", "gradient"))
    if op in ("norm", "norm_grad", "quant_rows"):
        hidden = _log_int(rng, 16, 16384, 16)
        rows = _log_int(rng, 1, min(65536, 16384 * 7168 // hidden))
        if op == "norm":
            y = rng.random() < 0.6
            return dict(op=op, tokens=rows, hidden=hidden, residual=rng.random() < 0.7, y=y,
                        codes=rng.choice(("block", "row") + ("none",) * y))
        if op == "norm_grad":
            return dict(op=op, tokens=rows, hidden=hidden, stream=rng.random() < 0.7)
        halves = rng.choice((1, 1, 2))
        return dict(op=op, rows=rows, hidden=-(-hidden // (16 * halves)) * 16 * halves, halves=halves)
    experts, inner, outer = _log_int(rng, 1, 64), _log_int(rng, 32, 8192, 16), _log_int(rng, 32, 8192, 16)
    if op == "quant_weights":
        halves = rng.choice((1, 2))
        while experts * inner * outer * halves > 8 * 4096 * 7168:
            experts, outer = (experts + 1) // 2, max(32, outer // 32 * 16)
        return dict(op=op, experts=experts, outer=outer, inner=inner, halves=halves)
    act, rows = rng.choice(ACTS), _log_int(rng, 1, 16384)
    halves = rng.choice((1, 2)) if op == "gradient" and act == "none" else 1
    wide = 2 if act == "swiglu" else halves
    then = _log_int(rng, 32, 8192, 16) if rng.random() < 0.4 else 0
    if op == "product":
        cost = inner * outer * wide + outer * then
    else:
        cost = inner * outer * halves + inner * then * (2 if act == "swiglu" else 1)
    while rows * cost > 16384 * 7168 * 2048 * 3 or experts * cost > 32 * 7168 * 2048 * 3:
        rows, experts = (rows + 1) // 2, (experts + 1) // 2
    spread = "uneven" if rows > experts or rng.random() < 0.5 else "single"
    more = dict(then=then, spread=spread)
    if op == "gradient":
        return dict(op=op, rows=rows, experts=experts, inner=inner, outer=outer, act=act, halves=halves, **more)
    return dict(op=op, rows=rows, experts=experts, inner=inner, outer=outer, act=act, bias=rng.random() < 0.5,
                residual=rng.random() < 0.5, keep=rng.random() < 0.5, scales=rng.choice(("block", "row")), **more)


def _row_counts(case, seed):
    """Rows of each expert's run, a list that sums to `rows`: one row each for a few experts ("single"), or drawn with
    uneven odds ("uneven"; a few experts get none)."""
    rng = random.Random(seed)
    experts, rows = case["experts"], case["rows"]
    if case["spread"] == "single":
        took = set(rng.sample(range(experts), rows))
        return [int(e in took) for e in range(experts)]
    odds = [math.exp(0.7 * rng.gauss(0, 1)) * (rng.random() > 0.05) + 1e-9 for _ in range(experts)]
    counts = [int(rows * o / sum(odds)) for o in odds]
    counts[rng.randrange(experts)] += rows - sum(counts)
    return counts


def _blocks(n):
    return -(-n // BLOCK)


def _coded(x, rows, cols):
    """x [..., R, C] fp32 in blocks of rows x cols: (E4M3 codes, scales [..., blocks of R, blocks of C])."""
    R, C = x.shape[-2:]
    nr, nc = -(-R // rows), -(-C // cols)
    tall = torch.nn.functional.pad(x, (0, nc * cols - C, 0, nr * rows - R))
    tall = tall.view(*x.shape[:-2], nr, rows, nc, cols)
    scales = tall.abs().amax((-3, -1)) / 448
    codes = tall / torch.where(scales > 0, scales, 1)[..., :, None, :, None]
    codes = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(*x.shape[:-2], nr * rows, nc * cols)
    return codes[..., :R, :C].contiguous(), scales


def _coded_weights(normal, experts, halves, outer, inner, turned=False):
    """Codes [experts, halves * outer, inner] with a scale for each 128 x 128 of a half; turned: [experts, outer, halves *
    inner], as a gradient's product reads them."""
    codes, scales = [], []
    for _ in range(experts):
        c, v = _coded(normal(halves, outer, inner, scale=(halves * inner) ** -0.5).float(), BLOCK, BLOCK)
        c = c.view(torch.uint8)
        codes.append(c.transpose(0, 1).reshape(outer, -1) if turned else c.view(halves * outer, inner))
        scales.append(v.transpose(0, 1) if turned else v)
    return torch.stack(codes).view(torch.float8_e4m3fn), torch.stack(scales).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        out = torch.empty(shape, dtype=dtype, device=dev).normal_(generator=g)
        return out.mul_(scale) if scale != 1.0 else out

    def room(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=dev)

    s = dict(case=case, kept={})
    if case["op"] == "norm":
        T, H = case["tokens"], case["hidden"]
        s["x"] = normal(T, H)
        s["residual"] = normal(T, H, scale=2.0) if case["residual"] else None
        s["weight"] = normal(H, scale=0.1, dtype=torch.float32) + 1
        s["sum"] = room(T, H) if case["residual"] else None
        s["y"] = room(T, H) if case["y"] else None
        s["codes"] = s["scales"] = None
        if case["codes"] != "none":
            s["codes"] = room(T, H, dtype=torch.uint8).view(torch.float8_e4m3fn)
            shape = (T, _blocks(H)) if case["codes"] == "block" else (T,)
            s["scales"] = room(*shape, dtype=torch.float32)
    elif case["op"] == "norm_grad":
        T, H = case["tokens"], case["hidden"]
        s["sum"], s["d_y"] = normal(T, H, scale=2.0), normal(T, H, scale=1e-2)
        s["d_sum"] = normal(T, H, scale=1e-2) if case["stream"] else None
        s["weight"] = normal(H, scale=0.1, dtype=torch.float32) + 1
        s["d_x"], s["d_weight"] = room(T, H), room(H, dtype=torch.float32)
    elif case["op"] == "quant_rows":
        rows, H, halves = case["rows"], case["hidden"], case["halves"]
        s["x"] = normal(rows, H, scale=1e-2) * torch.exp(normal(rows, 1, dtype=torch.float32)).bfloat16()
        s["codes"] = room(rows, H, dtype=torch.uint8).view(torch.float8_e4m3fn)
        nb = _blocks(H // halves)
        s["scales"] = room(rows, nb, dtype=torch.float32) if halves == 1 else room(rows, 2, nb, dtype=torch.float32)
    elif case["op"] == "quant_weights":
        E, N, K, halves = case["experts"], case["outer"], case["inner"], case["halves"]
        s["w"] = normal(E, halves * N, K, scale=K ** -0.5)
        s["codes"] = room(E, halves * N, K, dtype=torch.uint8).view(torch.float8_e4m3fn)
        s["scales"] = room(E, halves, _blocks(N), _blocks(K), dtype=torch.float32)
        s["codes_t"] = room(E, K, halves * N, dtype=torch.uint8).view(torch.float8_e4m3fn)
        s["scales_t"] = room(E, _blocks(K), halves, _blocks(N), dtype=torch.float32)
    else:
        E, K, N, rows = case["experts"], case["inner"], case["outer"], case["rows"]
        counts = _row_counts(case, seed)
        s["counts"] = counts
        s["offsets"] = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device=dev)
        wide = 2 if case["act"] == "swiglu" else 1
        if case["op"] == "product":
            s["x"], s["x_scales"] = _coded(normal(rows, K).float(), 1, K if case["scales"] == "row" else BLOCK)
            if case["scales"] == "row":
                s["x_scales"] = s["x_scales"][:, 0].contiguous()
            s["w"], s["w_scales"] = _coded_weights(normal, E, wide, N, K)
            s["bias"] = normal(E, wide * N, scale=0.1, dtype=torch.float32) if case["bias"] else None
            s["preact"] = room(rows, wide * N) if case["keep"] else None
            s["out"] = room(rows, case["then"] or N)
            s["residual"] = normal(rows, case["then"] or N) if case["residual"] else None
            if case["then"]:
                s["w2"], s["w2_scales"] = _coded_weights(normal, E, 1, case["then"], N)
                s["codes"] = room(rows, N, dtype=torch.uint8).view(torch.float8_e4m3fn)
                s["scales"] = room(rows, _blocks(N), dtype=torch.float32)
        else:
            h = case["halves"]
            s["dy"], s["dy_scales"] = _coded(normal(rows * h, N, scale=1e-2).float(), 1, BLOCK)
            s["dy"] = s["dy"].view(rows, h * N)
            s["dy_scales"] = s["dy_scales"].view(rows, h, _blocks(N)) if h == 2 else s["dy_scales"]
            s["w_t"], s["w_t_scales"] = _coded_weights(normal, E, h, K, N, turned=True)
            s["preact"] = normal(rows, wide * K) if case["act"] != "none" else None
            s["dx"] = room(rows, wide * K)
            if case["then"]:
                s["w2_t"], s["w2_t_scales"] = _coded_weights(normal, E, wide, case["then"], K, turned=True)
                s["codes"] = room(rows, wide * K, dtype=torch.uint8).view(torch.float8_e4m3fn)
                s["scales"] = room(rows, _blocks(K), dtype=torch.float32) if wide == 1 else \
                    room(rows, 2, _blocks(K), dtype=torch.float32)
                s["out"] = room(rows, case["then"])
    return s


def run(s):
    if own:
        return _own[s["case"]["op"]](s)
    return _plain[s["case"]["op"]](s)


# ---- the package's calls


def _own_norm(s):
    from combine_fp32_router_amd import binding as B

    B.moe_add_norm(s["x"], s["residual"], s["weight"], EPS, s["sum"], s["y"], s["codes"], s["scales"])
    return {k: s[k] for k in ("sum", "y", "codes", "scales")}


def _own_norm_grad(s):
    from combine_fp32_router_amd import binding as B

    B.moe_add_norm_grad(s["d_y"], s["d_sum"], s["sum"], s["weight"], EPS, s["d_x"], s["d_weight"])
    return {k: s[k] for k in ("d_x", "d_weight")}


def _own_quant_rows(s):
    from combine_fp32_router_amd import binding as B

    B.moe_quant_rows(s["x"], s["codes"], s["scales"], halves=s["case"]["halves"])
    return {k: s[k] for k in ("codes", "scales")}


def _own_quant_weights(s):
    from combine_fp32_router_amd import binding as B

    B.moe_quant_weights(s["w"], s["codes"], s["scales"], s["codes_t"], s["scales_t"], halves=s["case"]["halves"])
    return {k: s[k] for k in ("codes", "scales", "codes_t", "scales_t")}


def _own_product(s):
    from combine_fp32_router_amd import binding as B

    act = ACTS.index(s["case"]["act"])
    if s["case"]["then"]:
        B.moe_expert_matmul_fp8(s["x"], s["x_scales"], s["offsets"], s["w"], s["w_scales"], s["bias"], act, None, None,
                                s["codes"], s["scales"], s["preact"])
        B.moe_expert_matmul_fp8(s["codes"], s["scales"], s["offsets"], s["w2"], s["w2_scales"], None, B.MOE_ACT_NONE,
                                s["residual"], s["out"])
    else:
        B.moe_expert_matmul_fp8(s["x"], s["x_scales"], s["offsets"], s["w"], s["w_scales"], s["bias"], act, s["residual"],
                                s["out"], preact=s["preact"])
    return {k: s[k] for k in ("out", "preact")}


def _own_gradient(s):
    from combine_fp32_router_amd import binding as B

    codes = (s["codes"], s["scales"]) if s["case"]["then"] else (None, None)
    B.moe_expert_matmul_fp8_dx(s["dy"], s["dy_scales"], s["offsets"], s["w_t"], s["w_t_scales"],
                               ACTS.index(s["case"]["act"]), s["preact"], s["dx"], *codes)
    if not s["case"]["then"]:
        return dict(dx=s["dx"])
    B.moe_expert_matmul_fp8_dx(*codes, s["offsets"], s["w2_t"], s["w2_t_scales"], B.MOE_ACT_NONE, None, s["out"])
    return dict(dx=s["dx"], out=s["out"])


# ---- the plain forms, in 32 bits, rounded once


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * s["weight"]
    codes = scales = None
    if c["codes"] != "none":
        codes, scales = _coded(y, 1, c["hidden"] if c["codes"] == "row" else BLOCK)
        scales = scales[:, 0] if c["codes"] == "row" else scales
    return dict(sum=None if s["sum"] is None else x.bfloat16(), y=None if s["y"] is None else y.bfloat16(),
                codes=codes, scales=scales)


def _plain_norm_grad(s):
    x, d_y = s["sum"].float(), s["d_y"].float()
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    x = x * r
    g = d_y * s["weight"]
    d_x = r * (g - x * (g * x).mean(1, keepdim=True))
    if s["d_sum"] is not None:
        d_x = d_x + s["d_sum"].float()
    return dict(d_x=d_x.bfloat16(), d_weight=(d_y * x).sum(0))


def _plain_quant_rows(s):
    rows, H, halves = s["case"]["rows"], s["case"]["hidden"], s["case"]["halves"]
    codes, scales = _coded(s["x"].float().view(rows * halves, H // halves), 1, BLOCK)
    return dict(codes=codes.view(rows, H), scales=scales.view(s["scales"].shape))


def _plain_quant_weights(s):
    c = s["case"]
    E, N, K, halves = c["experts"], c["outer"], c["inner"], c["halves"]
    codes, scales = _coded(s["w"].float().view(E, halves, N, K), BLOCK, BLOCK)
    codes_t = codes.view(torch.uint8).permute(0, 3, 1, 2).reshape(E, K, halves * N).view(torch.float8_e4m3fn)
    return dict(codes=codes.view(E, halves * N, K), scales=scales, codes_t=codes_t,
                scales_t=scales.permute(0, 3, 1, 2).contiguous())


def _spread(scales, rows, cols, block_rows):
    """Scales [blocks of rows, blocks of cols] at every row and column."""
    if block_rows > 1:
        scales = scales.repeat_interleave(block_rows, -2)[..., :rows, :]
    return scales.repeat_interleave(BLOCK, -1)[..., :cols]


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


def _plain_rows(x, scales, w, w_scales, counts, halves, outer, inner):
    """fp32 rows [rows, inner] by their experts' weights [halves * outer, inner]."""
    x = x.float() * (scales[:, None] if scales.dim() == 1 else _spread(scales, len(x), inner, 1))
    parts = []
    for e, rows in enumerate(x.split(counts)):
        if len(rows):
            m = w[e].float().view(halves, outer, inner) * _spread(w_scales[e], outer, inner, BLOCK)
            parts.append(rows @ m.view(halves * outer, inner).t())
    return torch.cat(parts)


def _plain_product(s):
    c = s["case"]
    E, K, N, wide = c["experts"], c["inner"], c["outer"], 2 if c["act"] == "swiglu" else 1
    z = _plain_rows(s["x"], s["x_scales"], s["w"], s["w_scales"], s["counts"], wide, N, K)
    if s["bias"] is not None:
        at = torch.repeat_interleave(torch.arange(E, device=z.device), s["offsets"].diff(), output_size=len(z))
        z = z + s["bias"][at]
    y = _act(z, c["act"])
    if c["then"]:
        codes, scales = _coded(y, 1, BLOCK)
        y = _plain_rows(codes, scales, s["w2"], s["w2_scales"], s["counts"], 1, c["then"], N)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return dict(out=y.bfloat16(), preact=None if s["preact"] is None else z.bfloat16())


def _plain_back(dy, scales, w_t, w_t_scales, counts, halves, outer, inner):
    """fp32 rows [rows, halves * inner] by the transposed weights [outer, halves * inner]."""
    rows = len(dy)
    dy = dy.float().view(rows, halves, inner) * _spread(scales.view(rows, halves, -1), halves, inner, 1)
    parts = []
    for e, d in enumerate(dy.split(counts)):
        if len(d):
            m = w_t[e].float().view(outer, halves, inner).transpose(0, 1)
            m = m * _spread(w_t_scales[e].transpose(0, 1), outer, inner, BLOCK)
            parts.append(d.reshape(-1, halves * inner) @ m.transpose(0, 1).reshape(outer, halves * inner).t())
    return torch.cat(parts)


def _plain_gradient(s):
    c = s["case"]
    wide = 2 if c["act"] == "swiglu" else 1
    g = _plain_back(s["dy"], s["dy_scales"], s["w_t"], s["w_t_scales"], s["counts"], c["halves"], c["inner"], c["outer"])
    if s["preact"] is not None:
        g = _act_gradient(s["preact"].float(), g, c["act"])
    if not c["then"]:
        return dict(dx=g.bfloat16())
    codes, scales = _coded(g.view(-1, c["inner"]), 1, BLOCK)
    out = _plain_back(codes.view(c["rows"], -1), scales, s["w2_t"], s["w2_t_scales"], s["counts"], wide, c["then"],
                      c["inner"])
    return dict(dx=g.bfloat16(), out=out.bfloat16())


_own = dict(norm=_own_norm, norm_grad=_own_norm_grad, quant_rows=_own_quant_rows, quant_weights=_own_quant_weights,
            product=_own_product, gradient=_own_gradient)
_plain = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, quant_rows=_plain_quant_rows,
              quant_weights=_plain_quant_weights, product=_plain_product, gradient=_plain_gradient)


# ---- what one pass cannot do without


def work(case):
    op = case["op"]
    if case["op"] == "norm":
        n, T = case["tokens"] * case["hidden"], case["tokens"]
        moved = n * (2 + 4 * case["residual"] + 2 * case["y"] + (case["codes"] != "none")) + 4 * case["hidden"]
        return dict(bytes=moved + 4 * T * (_blocks(case["hidden"]) if case["codes"] == "block" else 1), flops=6 * n)
    if case["op"] == "norm_grad":
        n = case["tokens"] * case["hidden"]
        return dict(bytes=n * (6 + 2 * case["stream"]) + 8 * case["hidden"], flops=12 * n)
    if case["op"] == "quant_rows":
        n = case["rows"] * case["hidden"]
        return dict(bytes=3 * n + 4 * case["rows"] * case["halves"] * _blocks(case["hidden"] // case["halves"]), flops=2 * n)
    if case["op"] == "quant_weights":
        n = case["experts"] * case["halves"] * case["outer"] * case["inner"]
        return dict(bytes=4 * n + 8 * case["experts"] * case["halves"] * _blocks(case["outer"]) * _blocks(case["inner"]),
                    flops=2 * n)
    E, K, N, rows = case["experts"], case["inner"], case["outer"], case["rows"]
    wide = 2 if case["act"] == "swiglu" else 1
    then = case["then"]
    if op == "product":
        weights = wide * (K * N + 4 * _blocks(K) * _blocks(N)) + then * N + 4 * _blocks(then) * _blocks(N)
        taken = K + 4 * (_blocks(K) if case["scales"] == "block" else 1) + 2 * (then or N) * case["residual"]
        made = 2 * (then or N) + 2 * wide * N * case["keep"]
        return dict(bytes=min(E, rows) * weights + rows * (taken + made), flops=2 * rows * (K * N * wide + N * then))
    h = case["halves"]
    weights = h * (K * N + 4 * _blocks(K) * _blocks(N)) + wide * (then * K + 4 * _blocks(then) * _blocks(K))
    moved = h * (N + 4 * _blocks(N)) + 2 * wide * K * (1 if case["act"] == "none" else 2) + 2 * then
    return dict(bytes=min(E, rows) * weights + rows * moved, flops=2 * rows * (K * N * h + K * then * wide))


# ---- the same from the definitions, in 64 bits (a code's value before its rounding)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact[case["op"]](s, case)


def _exact_codes(v, block):
    """v [rows, n] in blocks of `block`: (v / its block's scale, scales)."""
    at = torch.arange(v.shape[1], device=v.device) // block
    tops = torch.zeros(v.shape[0], int(at[-1]) + 1, dtype=v.dtype, device=v.device)
    tops = tops.scatter_reduce(1, at.expand_as(v), v.abs(), "amax")
    scales = tops / 448
    quotient = v / scales[:, at]
    return torch.where(scales[:, at] > 0, quotient, torch.zeros_like(v)), scales


def _exact_norm(s, case):
    x = s["x"].double()
    if s["residual"] is not None:
        x = x.add(s["residual"].double())
    size = torch.linalg.vector_norm(x, dim=1, keepdim=True).square() / case["hidden"]
    y = torch.rsqrt(size + EPS) * x * s["weight"].double()
    codes = scales = None
    if case["codes"] == "block":
        codes, scales = _exact_codes(y, BLOCK)
    elif case["codes"] == "row":
        codes, scales = _exact_codes(y, case["hidden"])
        scales = scales.flatten()
    return dict(sum=None if s["sum"] is None else x, y=None if s["y"] is None else y, codes=codes, scales=scales)


def _exact_norm_grad(s, case):
    # from autograd, of the norm as it is defined
    x = s["sum"].double().requires_grad_()
    w = s["weight"].double().requires_grad_()
    with torch.enable_grad():
        y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w
    d_x, d_w = torch.autograd.grad(y, (x, w), s["d_y"].double())
    if s["d_sum"] is not None:
        d_x += s["d_sum"].double()
    return dict(d_x=d_x, d_weight=d_w)


def _exact_quant_rows(s, case):
    parts = [_exact_codes(x, BLOCK) for x in s["x"].double().chunk(case["halves"], dim=1)]
    codes = torch.cat([c for c, _ in parts], 1)
    scales = parts[0][1] if len(parts) == 1 else torch.stack([v for _, v in parts], 1)
    return dict(codes=codes, scales=scales)


def _exact_quant_weights(s, case):
    E, N, K, halves = case["experts"], case["outer"], case["inner"], case["halves"]
    codes = torch.zeros(E, halves, N, K, dtype=torch.float64, device=s["w"].device)
    scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device=s["w"].device)
    w = s["w"].view(E, halves, N, K)
    for i, n in enumerate(range(0, N, BLOCK)):
        tall = w[:, :, n:n + BLOCK].double()
        for j, k in enumerate(range(0, K, BLOCK)):
            part = tall[..., k:k + BLOCK]
            scale = part.abs().flatten(2).max(2).values / 448
            scales[:, :, i, j] = scale
            codes[:, :, n:n + BLOCK, k:k + BLOCK] = part / scale[..., None, None].clamp(min=1e-300)
    turned = codes.permute(0, 3, 1, 2).reshape(E, K, halves * N)
    return dict(codes=codes.reshape(E, halves * N, K), scales=scales, codes_t=turned, scales_t=scales.permute(0, 3, 1, 2))


def _exact_weights(codes, scales):
    """codes [R, C] with a scale for each 128 x 128."""
    R, C = codes.shape
    at = [torch.arange(n, device=codes.device) // BLOCK for n in (R, C)]
    return codes.double() * scales.double()[at[0]][:, at[1]]


def _exact_rounded(v):
    """The coded rows v [rows, n] in 64 bits: each value over its scale rounded to the nearest E4M3 number (three bits behind
    the first, steps of 2^-9 below 2^-6; ties to even)."""
    q, scales = _exact_codes(v, BLOCK)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    at = torch.arange(v.shape[1], device=v.device) // BLOCK
    return torch.round(q / step) * step * scales[:, at]


def _exact_product(s, case):
    K, N, gated = case["inner"], case["outer"], case["act"] == "swiglu"
    scales = s["x_scales"].double().view(case["rows"], -1)
    at = torch.arange(K, device=scales.device) // BLOCK * (case["scales"] == "block")
    x = s["x"].double() * scales[:, at]
    z = torch.zeros(case["rows"], N * (1 + gated), dtype=torch.float64, device=x.device)
    for e, n in enumerate(s["counts"]):
        a = sum(s["counts"][:e])
        for half in range(1 + gated if n else 0):
            cols = slice(half * N, (half + 1) * N)
            z[a:a + n, cols] = x[a:a + n] @ _exact_weights(s["w"][e][cols], s["w_scales"][e][half]).T
        if n and s["bias"] is not None:
            z[a:a + n] += s["bias"][e].double()
    if gated:
        y = torch.nn.functional.silu(z[:, :N]) * z[:, N:]
    else:
        y = dict(none=lambda v: v, relu=torch.relu, silu=torch.nn.functional.silu,
                 gelu=torch.nn.functional.gelu)[case["act"]](z)
    if case["then"]:
        h = _exact_rounded(y)
        y = torch.zeros(case["rows"], case["then"], dtype=torch.float64, device=x.device)
        for e, n in enumerate(s["counts"]):
            if n:
                a = sum(s["counts"][:e])
                y[a:a + n] = h[a:a + n] @ _exact_weights(s["w2"][e], s["w2_scales"][e][0]).T
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return dict(out=y, preact=None if s["preact"] is None else z)


def _exact_gradient(s, case):
    K, N, h, then = case["inner"], case["outer"], case["halves"], case["then"]
    dev = s["dy"].device
    g = torch.zeros(case["rows"], K, dtype=torch.float64, device=dev)
    at = torch.arange(N, device=dev) // BLOCK
    for half in range(h):
        cols = slice(half * N, (half + 1) * N)
        scales = s["dy_scales"].view(case["rows"], h, -1)[:, half].double()
        dy = s["dy"][:, cols].double() * scales[:, at]
        for e, n in enumerate(s["counts"]):
            if n:
                a = sum(s["counts"][:e])
                g[a:a + n] += dy[a:a + n] @ _exact_weights(s["w_t"][e][:, cols], s["w_t_scales"][e][:, half]).T
    if s["preact"] is not None:
        z = s["preact"].double().requires_grad_()
        with torch.enable_grad():
            if case["act"] == "swiglu":
                y = torch.nn.functional.silu(z[:, :K]) * z[:, K:]
            else:
                y = dict(relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)[case["act"]](z)
            g, = torch.autograd.grad(y, z, g)
    if not then:
        return dict(dx=g)
    out = torch.zeros(case["rows"], then, dtype=torch.float64, device=dev)
    for half, v in enumerate(g.split(K, dim=1)):
        v, cols = _exact_rounded(v), slice(half * K, (half + 1) * K)
        for e, n in enumerate(s["counts"]):
            if n:
                a = sum(s["counts"][:e])
                out[a:a + n] += v[a:a + n] @ _exact_weights(s["w2_t"][e][:, cols], s["w2_t_scales"][e][:, half]).T
    return dict(dx=g, out=out)


_exact = dict(norm=_exact_norm, norm_grad=_exact_norm_grad, quant_rows=_exact_quant_rows,
              quant_weights=_exact_quant_weights, product=_exact_product, gradient=_exact_gradient)

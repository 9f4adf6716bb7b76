"""The experts' products and their gradients against their 64-bit forms."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

NONE, RELU, SILU, GELU, SWIGLU = range(5)
CANARY = -7.0

# run lengths per expert, K, N, act, bias, residual, keep preact
PRODUCTS = [
    ([1], 16, 16, NONE, False, False, False), ([1], 7168, 512, SWIGLU, False, False, True),
    ([0, 1, 0, 0, 1, 1], 512, 48, SILU, True, False, True), ([8], 64, 128, GELU, True, True, True),
    ([15, 16, 17, 0, 33], 272, 144, SWIGLU, True, True, True), ([127, 128, 129, 1], 80, 272, RELU, True, True, False),
    ([255, 256, 257, 0, 0, 2], 512, 256, SWIGLU, False, False, True), ([300], 1040, 2064, NONE, True, True, False),
    ([64] * 8, 256, 768, SWIGLU, False, True, False), ([0, 0, 0], 64, 64, NONE, False, False, False),
    ([3] * 70, 128, 96, GELU, True, False, True), ([513, 5], 1024, 1040, SILU, False, False, False),
    ([1000, 24, 0, 700], 2048, 768, SWIGLU, True, False, True), ([40, 9, 31], 4096, 1024, NONE, False, True, False),
    ([2, 0, 3, 1, 1, 1], 2048, 2048, SWIGLU, True, True, False), ([129] * 3, 48, 32, SWIGLU, True, False, True)]


def offsets_of(lengths, base=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + base, dtype=torch.int32, device="cuda")


def normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def check_product(lengths, K, N, act, bias, residual, keep, base=0, spare=3, rows=None, scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, wide = len(lengths), 2 if act == SWIGLU else 1
    rows = sum(lengths) + spare if rows is None else rows
    x, w = normal(g, rows, K, scale=scale), normal(g, E, wide * N, K, scale=K ** -0.5)
    b = normal(g, E, wide * N, dtype=torch.float32) if bias else None
    res = normal(g, rows, N) if residual else None
    out = torch.full((rows, N), CANARY, dtype=torch.bfloat16, device="cuda")
    pre = torch.full((rows, wide * N), CANARY, dtype=torch.bfloat16, device="cuda") if keep else None
    off = offsets_of(lengths, base)
    B.moe_expert_matmul(x, off, w, b, act, res, out, pre)
    torch.cuda.synchronize()
    y, dy, z, dz, written = R.product(x, off.tolist(), w, b, act, res)
    R.inside(out[written], y[written], dy[written], "out")
    assert (out[~written] == CANARY).all()
    if keep:
        R.inside(pre[written], z[written], dz[written], "preact")
        assert (pre[~written] == CANARY).all()
    return x, w, b, res, off, out, pre


@pytest.mark.parametrize("case", PRODUCTS, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}a{c[3]}" for c in PRODUCTS])
def test_product(case):
    check_product(*case)


@pytest.mark.parametrize("n", [1, 2, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 200])
@pytest.mark.parametrize("act", [NONE, SWIGLU])
def test_run_lengths(n, act):
    """One run of every length around the tiles' edges, beside an empty one."""
    check_product([0, n], 144, 80, act, True, True, True, seed=n)


# Runs around the tiles' edges, with enough rows for the 256- and (MANY) the
# 128-column tiles rather than the kernel for few rows.
EDGES = [127, 128, 129, 1, 255, 256, 257, 0, 64, 65, 2, 3000]
MANY = [130, 1, 0, 64, 1200, 105]
TILED = [(EDGES, 80, 2064, NONE, True, True, True), (EDGES, 272, 1040, SWIGLU, True, True, True),
         (EDGES, 144, 2064, GELU, False, False, True), (EDGES, 528, 1040, SWIGLU, False, False, False),
         (MANY, 528, 2064, SILU, True, True, True), (MANY, 1040, 1040, SWIGLU, True, False, True),
         (MANY, 1040, 1200, RELU, False, True, False), ([0, 1500, 0], 1040, 1040, SWIGLU, True, True, True)]


@pytest.mark.parametrize("case", TILED, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}a{c[3]}" for c in TILED])
def test_tiled_product(case):
    check_product(*case, base=7)


@pytest.mark.parametrize("K", [48, 64, 80, 112, 128, 144, 192, 272])
def test_tiled_reduced_lengths(K):
    check_product(EDGES, K, 2064, NONE, False, False, False, seed=K)


def tile_shape(lengths, rows, columns):
    """The tiles (rows, columns) that a call of these outputs takes: the smallest
    of which at most 256 come out."""
    live = min(rows, len(lengths))
    for h, c in ((64, 128), (64, 256), (128, 128), (128, 256), (256, 128)):
        if ((rows - live) // h + live) * -(-columns // c) <= 256:
            return h, c
    return 256, 256


# runs, columns (gate and up ones both), the tiles they take
SHAPES = [(EDGES, 368, (64, 128)), (EDGES, 752, (64, 256)), ([5000, 0, 130, 140], 640, (128, 128)),
          (EDGES, 1248, (128, 256)), ([12000, 0, 65, 1], 640, (256, 128)), (EDGES, 2064, (256, 256)),
          ([5000, 1, 129, 128], 640, (128, 128)), ([77] * 40, 256, (64, 128)), ([0, 8000, 1, 200, 63], 1152, (256, 256))]


@pytest.mark.parametrize("lengths,columns,shape", SHAPES, ids=[f"r{sum(s[0])}N{s[1]}" for s in SHAPES])
def test_every_tile_shape(lengths, columns, shape):
    rows = sum(lengths)
    assert tile_shape(lengths, rows, columns) == shape
    check_product(lengths, 1040, columns, SILU, True, True, True, spare=0)
    check_product(lengths, 1040, columns // 32 * 16, SWIGLU, True, False, True, spare=0)
    check_dx(lengths, columns, 528, GELU, spare=0)
    check_dx(lengths, columns, 272, SWIGLU, spare=0)


# 17 tiles of 256 columns: of 21 or 16 whole ones of 256 rows, 101 or 16 are the
# last round's, which are cut to a half or a quarter; some pieces lie behind
# their run's end
@pytest.mark.parametrize("lengths", [[5000, 0, 200, 1], [3900, 150], [260, 3584, 140, 70]], ids=["halves", "quarters", "odd"])
def test_last_round_in_pieces(lengths):
    check_product(lengths, 144, 4112, SILU, True, True, True)
    check_product(lengths, 144, 2064, SWIGLU, True, False, True)
    check_dx(lengths, 4112, 144, GELU)


# few tiles (cut to 64 rows), some (to 128), many; and more runs than are ordered
CUTS = [([900], 272, 528), ([1500], 2560, 2560), ([0, 40, 1700, 3, 64], 1040, 1296), ([200, 300, 1000], 2064, 1040),
        ([65] * 70, 144, 272), ([700], 4112, 4112)]


@pytest.mark.parametrize("lengths,K,N", CUTS, ids=[f"E{len(s[0])}r{sum(s[0])}K{s[1]}N{s[2]}" for s in CUTS])
def test_cut_tiles_of_dw(lengths, K, N):
    test_dw(lengths, K, N, NONE)


def test_tiled_runs_are_cut_and_nan_stays():
    check_product(EDGES, 144, 2064, SILU, True, True, True, rows=3333)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = normal(g, 4000, 144), normal(g, 3, 2064, 144)
    x[1777], x[3990:] = float("nan"), float("nan")
    out = torch.zeros(4000, 2064, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul(x, offsets_of([1777, 1, 2212]), w, None, NONE, None, out)
    assert torch.isnan(out).any(1).nonzero()[:, 0].tolist() == [1777]
    y, dy, *_ = R.product(x, [0, 1777, 1778, 3990], w, None, NONE, out)
    x[1777] = 0
    B.moe_expert_matmul(x, offsets_of([1777, 1, 2212]), w, None, NONE, out, out)  # residual in place
    keep = torch.arange(3990, device="cuda") != 1777
    R.inside(out[:3990][keep], y[:3990][keep], dy[:3990][keep], "in place")


@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 112, 128, 144, 272, 528, 1040])
def test_reduced_lengths(K):
    check_product([70, 6], K, 112, SILU, False, True, False, seed=K)


@pytest.mark.parametrize("n", [3, 300])
def test_flat_numbering_starts_elsewhere(n):
    """Offsets of a rank's own experts: row 0 is row offsets[0]."""
    check_product([n, 0, 7, n], 128, 64, NONE, True, False, False, base=12345)


@pytest.mark.parametrize("rows", [5, 130, 299])
def test_runs_are_cut_at_the_buffer(rows):
    """Offsets past max_rows: the rows there are computed, none beyond."""
    check_product([100, 150, 400], 128, 64, RELU, False, True, True, rows=rows)


def test_large_values_and_saturation():
    """Pre-activations far out on both sides: sigmoid and erf saturate, nothing
    turns NaN."""
    for act in (RELU, SILU, GELU, SWIGLU):
        *_, out, pre = check_product([40, 300], 64, 64, act, True, False, True, scale=300.0)
        assert torch.isfinite(out[:340]).all() and torch.isfinite(pre[:340]).all()


def test_nan_stays_in_its_row():
    """A row of NaN (padding between runs of another caller, say) reaches no
    other row's output."""
    for n in (12, 400):
        g = torch.Generator(device="cuda").manual_seed(n)
        x, w = normal(g, n + 4, 80), normal(g, 2, 48, 80)
        x[3], x[n:] = float("nan"), float("nan")  # one row of a run, and the rows past the runs
        out = torch.zeros(n + 4, 48, dtype=torch.bfloat16, device="cuda")
        B.moe_expert_matmul(x, offsets_of([n // 2, n - n // 2]), w, None, NONE, None, out)
        bad = torch.isnan(out).any(1).nonzero()[:, 0].tolist()
        assert bad == [3]


def test_residual_in_place_and_alias_refusals():
    g = torch.Generator(device="cuda").manual_seed(3)
    for n in (9, 200):
        x, w, out = normal(g, n, 64), normal(g, 1, 96, 64, scale=0.125), normal(g, n, 96)
        off = offsets_of([n])
        y, dy, *_ = R.product(x, off.tolist(), w, None, GELU, out)
        B.moe_expert_matmul(x, off, w, None, GELU, out, out)
        R.inside(out, y, dy, "in place")


GRADIENTS = [
    ([1], 16, 16, NONE), ([5, 0, 2], 64, 128, GELU), ([127, 128, 129], 272, 144, SWIGLU), ([256, 0, 257, 31], 512, 272, SILU),
    ([300], 1040, 528, RELU), ([0, 0], 64, 64, SWIGLU), ([33] * 9, 768, 2048, SWIGLU), ([700, 1, 500], 256, 1024, SWIGLU),
    ([3, 1, 0, 4], 2048, 512, NONE), ([2100, 0, 129, 1, 64], 2064, 272, SWIGLU), ([700, 900], 1040, 4112, GELU)]


@pytest.mark.parametrize("lengths,K,N,act", GRADIENTS, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}a{c[3]}" for c in GRADIENTS])
def test_dx(lengths, K, N, act):
    check_dx(lengths, K, N, act)


def check_dx(lengths, K, N, act, spare=2):
    g = torch.Generator(device="cuda").manual_seed(7)
    E, wide, rows = len(lengths), 2 if act == SWIGLU else 1, sum(lengths) + spare
    dy, w = normal(g, rows, N), normal(g, E, N, K, scale=K ** -0.5)
    z = normal(g, rows, wide * K, scale=2.0) if act else None
    dx = torch.full((rows, wide * K), CANARY, dtype=torch.bfloat16, device="cuda")
    off = offsets_of(lengths, 99)
    want, tol, written = R.product_dx(dy, off.tolist(), w, act, z)
    B.moe_expert_matmul_dx(dy, off, w, act, z, dx)
    R.inside(dx[written], want[written], tol[written], "dx")
    assert (dx[~written] == CANARY).all()
    if act:  # in place of the pre-activations
        kept = z.clone()
        B.moe_expert_matmul_dx(dy, off, w, act, z, z)
        assert torch.equal(z[written], dx[written]) and torch.equal(z[~written], kept[~written])


@pytest.mark.parametrize("lengths,K,N,act", GRADIENTS, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}" for c in GRADIENTS])
def test_dw(lengths, K, N, act):
    g = torch.Generator(device="cuda").manual_seed(8)
    E, rows = len(lengths), sum(lengths) + 2
    dy, x = normal(g, rows, N), normal(g, rows, K)
    dy[sum(lengths):], x[sum(lengths):] = float("nan"), float("nan")  # rows of no run are not read
    off = offsets_of(lengths, 5)
    want, tol, db, tb = R.product_dw(dy, x, off.tolist(), E)
    dw, dbias = torch.full((E, N, K), CANARY, device="cuda"), torch.full((E, N), CANARY, device="cuda")
    B.moe_expert_matmul_dw(dy, x, off, dw, dbias)
    R.inside(dw, want, tol, "dw")
    R.inside(dbias, db, tb, "dbias")
    half = torch.full((E, N, K), CANARY, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul_dw(dy, x, off, half)
    R.inside(half, want, tol + R.UBF16 * (want.abs() + tol), "dw bf16")
    before, before_b = dw.clone(), dbias.clone()
    dw.add_(1.5), dbias.add_(1.5)
    B.moe_expert_matmul_dw(dy, x, off, dw, dbias, accumulate=True)
    R.inside(dw, before.double() + 1.5 + want, tol + 4 * R.U32 * (before.abs() + want.abs() + 1.5), "dw accumulated")
    R.inside(dbias, before_b.double() + 1.5 + db, tb + 4 * R.U32 * (before_b.abs() + db.abs() + 1.5), "dbias accumulated")


# few outputs and long sums, which several workgroups share
LONG_DX = [([130, 0, 70], 144, 8192, SWIGLU), ([1], 16, 4096, NONE), ([1200], 48, 6384, SILU), ([64, 1, 63, 65, 200], 272, 2064, GELU),
           ([3] * 20, 384, 16400, RELU)]
LONG = [([2000, 0, 100], 4096, 384, SILU, True, True, True), ([1900, 70, 1], 8192, 192, SWIGLU, True, True, True),
        ([8000], 8192, 48, NONE, False, False, False), ([900, 1100, 64], 6160, 368, GELU, True, False, True)]
LONG_DW = [([15000, 707], 192, 544, NONE), ([9, 30000, 0], 16, 16, NONE), ([8192], 1040, 272, NONE), ([0, 0, 9000], 128, 80, NONE)]


def workspace_of(name, lengths, spare, K, N):
    return B.expert_workspace_bytes("moe_expert_matmul_" + name, len(lengths), sum(lengths) + spare, K, N)


@pytest.mark.parametrize("case", LONG, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}a{c[3]}" for c in LONG])
def test_product_in_parts(case):
    lengths, K, N, act = case[:4]
    assert B.expert_workspace_bytes("moe_expert_matmul", len(lengths), sum(lengths) + 3, K, N, act) > 0
    x, w, b, res, off, out, pre = check_product(*case)
    space = torch.full((1 << 22,), float("nan"), device="cuda")
    again = torch.full_like(out, CANARY)
    B.moe_expert_matmul(x, off, w, b, act, res, again, pre, workspace=space)
    assert torch.equal(out, again)


@pytest.mark.parametrize("lengths,K,N,act", LONG_DX, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}a{c[3]}" for c in LONG_DX])
def test_dx_in_parts(lengths, K, N, act):
    assert workspace_of("dx", lengths, 2, K, N) > 0
    check_dx(lengths, K, N, act)


@pytest.mark.parametrize("lengths,K,N,act", LONG_DW, ids=[f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}" for c in LONG_DW])
def test_dw_in_parts(lengths, K, N, act):
    assert workspace_of("dw", lengths, 2, K, N) > 0
    test_dw(lengths, K, N, act)


def test_parts_with_workspaces_streams_and_a_graph():
    """The same bits with a workspace of the caller's (full of NaN, and nothing
    written behind it), on another stream, and replayed."""
    g = torch.Generator(device="cuda").manual_seed(11)
    lengths, K, N = [9000, 0, 1000], 144, 80
    E, rows, off = 3, 10000, offsets_of([9000, 0, 1000])
    dy, x, w = normal(g, rows, N), normal(g, rows, K), normal(g, E, 8192, K)
    long_dy = normal(g, 100, 8192)
    short = offsets_of([60, 0, 40])

    def outs():
        return (torch.zeros(E, N, K, device="cuda"), torch.zeros(E, N, device="cuda"),
                torch.zeros(100, K, dtype=torch.bfloat16, device="cuda"))

    def call(o, stream=None, spaces=(None, None)):
        B.moe_expert_matmul_dw(dy, x, off, o[0], o[1], stream=stream, workspace=spaces[0])
        B.moe_expert_matmul_dx(long_dy, short, w, NONE, None, o[2], stream=stream, workspace=spaces[1])

    first = outs()
    call(first)
    spaces = []
    for need in (workspace_of("dw", lengths, 0, K, N), workspace_of("dx", [60, 0, 40], 0, K, 8192)):
        assert need > 0 and need % 4 == 0
        spaces.append(torch.full((need // 4 + 64,), float("nan"), device="cuda"))
    used = [s[:-64].view(torch.uint8) for s in spaces]
    second, third, fourth = outs(), outs(), outs()
    call(second, None, used)
    assert all(torch.isnan(s[-64:]).all() for s in spaces)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(third, side)
    call(third, side.cuda_stream)
    side.synchronize()
    with torch.cuda.stream(side):
        call(fourth)
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            call(fourth)
    for s in range(3):
        for t in fourth:
            t.fill_(-7)
        graphs[s % 2].replay()
        torch.cuda.synchronize()
        for got in (second, third, fourth):
            assert all(torch.equal(p, q) for p, q in zip(first, got))
        again = outs()
        call(again)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_dw_without_rows():
    dw, db = torch.full((3, 32, 48), 2.0, device="cuda"), torch.full((3, 32), 2.0, device="cuda")
    none = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul_dw(*none, offsets_of([0, 0, 0]), dw, db, accumulate=True)
    assert (dw == 2).all() and (db == 2).all()
    B.moe_expert_matmul_dw(*none, offsets_of([0, 0, 0]), dw, db)
    assert not dw.any() and not db.any()


def test_products_agree_with_differences():
    """<dy, product(x + a) - product(x - a)> = 2 <dx, a>, and alike for the
    weights and the bias, on small integers where every step is exact."""
    g = torch.Generator(device="cuda").manual_seed(4)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").float()  # noqa: E731
    for lengths in ([3, 0, 5], [150, 0, 140]):
        rows, K, N, E = sum(lengths), 32, 48, 3
        off = offsets_of(lengths)
        x, a, w, c, b, h, dy = ints(rows, K), ints(rows, K), ints(E, N, K), ints(E, N, K), ints(E, N), ints(E, N), ints(rows, N)

        def out(x, w, b):
            o = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
            B.moe_expert_matmul(x.bfloat16(), off, w.bfloat16(), b, NONE, None, o)
            return o.double()

        dx = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
        B.moe_expert_matmul_dx(dy.bfloat16(), off, w.bfloat16(), NONE, None, dx)
        dw, db = torch.empty(E, N, K, device="cuda"), torch.empty(E, N, device="cuda")
        B.moe_expert_matmul_dw(dy.bfloat16(), x.bfloat16(), off, dw, db)
        d = dy.double()
        # |z| <= 32 * 2 + 2 and |dx| <= 48: integers below 256 are exact in bf16
        assert ((out(x + a, w, b) - out(x - a, w, b)) * d).sum() == 2 * (dx.double() * a.double()).sum()
        assert ((out(x, w + c, b) - out(x, w - c, b)) * d).sum() == 2 * (dw.double() * c.double()).sum()
        assert ((out(x, w, b + h) - out(x, w, b - h)) * d).sum() == 2 * (db.double() * h.double()).sum()


def test_experts_in_a_graph_and_same_bits():
    """Forward, dx and dw captured once and replayed on new rows and runs; each
    replay equals the eager calls bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(6)
    E, K, N, rows = 6, 256, 128, 500
    w1, w2 = normal(g, E, 2 * N, K, scale=K ** -0.5), normal(g, E, K, N, scale=N ** -0.5)
    x, dy = normal(g, rows, K), normal(g, rows, K)
    off = offsets_of([100, 0, 50, 200, 1, 149])

    def buffers():
        z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        return [z(rows, N), z(rows, 2 * N), z(rows, K), z(rows, 2 * N), z(E, K, N, dtype=torch.float32), z(rows, K)]

    def step(o):
        h, pre, y, dpre, dw2, dx = o
        B.moe_expert_matmul(x, off, w1, None, SWIGLU, None, h, pre)
        B.moe_expert_matmul(h, off, w2, None, NONE, None, y)
        B.moe_expert_matmul_dx(dy, off, w2, SWIGLU, pre, dpre)
        B.moe_expert_matmul_dw(dy, h, off, dw2)
        B.moe_expert_matmul_dx(dpre, off, w1, NONE, None, dx)

    a, b = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for lengths in ([100, 0, 50, 200, 1, 149], [0, 500, 0, 0, 0, 0], [1, 2, 3, 4, 5, 485]):
        off.copy_(offsets_of(lengths))
        x.copy_(normal(g, rows, K))
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        for p, q in zip(a, b):
            assert torch.equal(p, q)

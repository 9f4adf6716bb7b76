"""The products of E4M3 rows and weights and the gradient of their rows against
their 64-bit forms."""
import numpy as np
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

NONE, RELU, SILU, GELU, SWIGLU = range(5)
CANARY, MARK = -7.0, 77
EDGES = [127, 128, 129, 1, 255, 256, 257, 0, 64, 65, 2, 3000]
MANY = [130, 1, 0, 64, 1200, 105]

# run lengths per expert, K, N, act, bias, residual, keep preact, a scale for each row
PRODUCTS = [
    ([1], 16, 16, NONE, False, False, False, False), ([1], 7168, 512, SWIGLU, False, False, True, True),
    ([0, 1, 0, 0, 1, 1], 512, 48, SILU, True, False, True, False), ([8], 64, 128, GELU, True, True, True, True),
    ([15, 16, 17, 0, 33], 272, 144, SWIGLU, True, True, True, False),
    ([127, 128, 129, 1], 80, 272, RELU, True, True, False, False),
    ([255, 256, 257, 0, 0, 2], 512, 256, SWIGLU, False, False, True, False),
    ([300], 1040, 2064, NONE, True, True, False, True), ([64] * 8, 256, 768, SWIGLU, False, True, False, False),
    ([0, 0, 0], 64, 64, NONE, False, False, False, False), ([3] * 70, 128, 96, GELU, True, False, True, True),
    ([513, 5], 1024, 1040, SILU, False, False, False, False), ([1000, 24, 0, 700], 2048, 768, SWIGLU, True, False, True, False),
    ([40, 9, 31], 4096, 1024, NONE, False, True, False, True), ([2, 0, 3, 1, 1, 1], 2048, 2048, SWIGLU, True, True, False, False),
    ([129] * 3, 48, 32, SWIGLU, True, False, True, True), (EDGES, 80, 2064, NONE, True, True, True, False),
    (EDGES, 272, 1040, SWIGLU, True, True, True, False), (EDGES, 144, 2064, GELU, False, False, True, True),
    (MANY, 528, 2064, SILU, True, True, True, False), (MANY, 1040, 1040, SWIGLU, True, False, True, True),
    (MANY, 1040, 1200, RELU, False, True, False, False), ([0, 1500, 0], 1040, 1040, SWIGLU, True, True, True, False)]


def offsets_of(lengths, base=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]) + base, dtype=torch.int32, device="cuda")


def normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def coded_weights(g, E, wide, N, K):
    """E4M3 [E, wide * N, K], scales, the 64-bit values and their peaks."""
    codes, scales = F.coded(normal(g, E * wide, N, K, scale=K ** -0.5), 128, 128)
    return with_values(codes, scales, E, wide, N, K)


def with_values(codes, scales, E, wide, N, K):
    s = scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :N, :K]
    return (codes.view(torch.uint8).view(E, wide * N, K), scales.view(E, wide, F.blocks(N), F.blocks(K)),
            (F.e4m3(codes) * s).view(E, wide * N, K), F.peaks(codes, s).view(E, wide * N, -1))


def coded_rows(g, rows, K, row, scale=1.0):
    codes, scales = F.coded(normal(g, rows, K, scale=scale) * normal(g, rows, 1).exp(), 1, K if row else 128)
    s = scales.double().expand(rows, K) if row else F.at_columns(scales, K)
    return (codes.view(torch.uint8), scales[:, 0].contiguous() if row else scales, F.e4m3(codes) * s,
            F.peaks(codes, s))


def rooms(rows, n, halves=1):
    return (torch.full((rows, halves * n), CANARY, dtype=torch.bfloat16, device="cuda"),
            torch.full((rows, halves * n), MARK, dtype=torch.uint8, device="cuda"),
            torch.full((rows, halves, F.blocks(n)), CANARY, device="cuda"))


def check_product(lengths, K, N, act, bias, residual, keep, row, base=0, spare=3, rows=None, scale=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    E, wide = len(lengths), 2 if act == SWIGLU else 1
    rows = sum(lengths) + spare if rows is None else rows
    x, xs, x64, xp = coded_rows(g, rows, K, row, scale)
    w, ws, w64, wp = coded_weights(g, E, wide, N, K)
    b = normal(g, E, wide * N, dtype=torch.float32) if bias else None
    res = normal(g, rows, N) if residual else None
    out, codes, scales = rooms(rows, N)
    pre = torch.full((rows, wide * N), CANARY, dtype=torch.bfloat16, device="cuda") if keep else None
    off = offsets_of(lengths, base)
    B.moe_expert_matmul_fp8(x, xs, off, w, ws, b, act, res, out, codes, scales, pre)
    torch.cuda.synchronize()
    y, dy, z, dz, written = F.product(x64, xp, off.tolist(), w64, wp, b, act, res)
    R.inside(out[written], y[written], F.bf16(y, dy)[written], "out")
    F.check_codes(codes[written], scales[written, 0], y[written], dy[written], "out")
    assert (out[~written] == CANARY).all() and (codes[~written] == MARK).all() and (scales[~written] == CANARY).all()
    if keep:
        R.inside(pre[written], z[written], F.bf16(z, dz)[written], "preact")
        assert (pre[~written] == CANARY).all()
    only = torch.full_like(out, CANARY)  # one output at a time: the same bits
    B.moe_expert_matmul_fp8(x, xs, off, w, ws, b, act, res, only)
    assert torch.equal(only, out)
    _, c, s = rooms(rows, N)
    B.moe_expert_matmul_fp8(x, xs, off, w, ws, b, act, res, None, c, s[:, 0])
    assert torch.equal(c, codes) and torch.equal(s, scales)
    return x, xs, off, w, ws, b, res, out, codes, scales, pre


def ids(cases):
    return [f"E{len(c[0])}r{sum(c[0])}K{c[1]}N{c[2]}a{c[3]}" for c in cases]


@pytest.mark.parametrize("case", PRODUCTS, ids=ids(PRODUCTS))
def test_product(case):
    check_product(*case, base=7)


@pytest.mark.parametrize("n", [1, 2, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 200])
@pytest.mark.parametrize("act", [NONE, SWIGLU])
def test_run_lengths(n, act):
    """One run of every length around the tiles' edges, beside an empty one."""
    check_product([0, n], 144, 80, act, True, True, True, n % 2 == 0, seed=n)


@pytest.mark.parametrize("K", [16, 32, 112, 128, 144, 240, 256, 272, 400, 528, 1040])
def test_reduced_lengths(K):
    check_product([70, 6], K, 112, SILU, False, True, False, False, seed=K)
    check_product(EDGES, K, 2064, NONE, False, False, False, True, seed=K)


@pytest.mark.parametrize("rows", [5, 130, 299])
def test_runs_are_cut_at_the_buffer(rows):
    """Offsets past max_rows: the rows there are computed, none beyond."""
    check_product([100, 150, 400], 128, 64, RELU, False, True, True, False, rows=rows)


def test_large_values_and_saturation():
    for act in (RELU, SILU, GELU, SWIGLU):
        *_, out, _, _, pre = check_product([40, 300], 64, 64, act, True, False, True, False, scale=300.0)
        assert torch.isfinite(out[:340]).all() and torch.isfinite(pre[:340]).all()


# some rows an expert, 64 of them a tile: runs around its blocks of 16, and columns that
# end inside a group of 128
SOME = [1, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 0, 66, 127, 129, 130]


@pytest.mark.parametrize("K,N,act", [(16, 4112, NONE), (528, 2064, SWIGLU), (640, 2048, SILU), (2064, 1040, SWIGLU), (1040, 4096, GELU)])
@pytest.mark.parametrize("row", [False, True])
def test_some_rows_an_expert(K, N, act, row):
    check_product(SOME, K, N, act, True, True, True, row, base=3)


@pytest.mark.parametrize("K,N,act,halves", [(4112, 16, NONE, 1), (2064, 528, SWIGLU, 1), (2048, 640, NONE, 2), (1040, 400, GELU, 1),
                                            (4096, 1040, SWIGLU, 1), (2064, 528, NONE, 2)])
def test_some_rows_dx(K, N, act, halves):
    test_dx(SOME, K, N, act, halves)


@pytest.mark.parametrize("n", [12, 400, 3000])
def test_nan_stays_in_its_row(n):
    """A NaN code, or a NaN scale, of one row reaches no other row; NaN behind the
    runs reaches none."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x, xs, _, _ = coded_rows(g, n + 4, 272, False)
    w, ws, _, _ = coded_weights(g, 2, 1, 144, 272)
    x[3, 7], xs[5, 1] = 0x7F, float("nan")
    x[n:], xs[n:] = 0x7F, float("nan")
    out, codes, scales = rooms(n + 4, 144)
    B.moe_expert_matmul_fp8(x, xs, offsets_of([n // 2, n - n // 2]), w, ws, None, NONE, None, out, codes, scales[:, 0])
    assert torch.isnan(out).any(1).nonzero()[:, 0].tolist() == [3, 5]
    assert torch.isnan(scales).flatten(1).all(1).nonzero()[:, 0].tolist() == [3, 5]


def test_residual_in_place():
    g = torch.Generator(device="cuda").manual_seed(3)
    for n in (9, 200, 2000):
        x, xs, x64, xp = coded_rows(g, n, 192, False)
        w, ws, w64, wp = coded_weights(g, 1, 1, 96, 192)
        out, off = normal(g, n, 96), offsets_of([n])
        y, dy, *_ = F.product(x64, xp, off.tolist(), w64, wp, None, GELU, out)
        B.moe_expert_matmul_fp8(x, xs, off, w, ws, None, GELU, out, out)
        R.inside(out, y, F.bf16(y, dy), "in place")


GRADIENTS = [
    ([1], 16, 16, NONE, 1), ([5, 0, 2], 64, 128, GELU, 1), ([127, 128, 129], 272, 144, SWIGLU, 1),
    ([256, 0, 257, 31], 512, 272, SILU, 1), ([300], 1040, 528, RELU, 1), ([0, 0], 64, 64, SWIGLU, 1),
    ([33] * 9, 768, 2048, SWIGLU, 1), ([700, 1, 500], 256, 1024, SWIGLU, 1), ([3, 1, 0, 4], 2048, 512, NONE, 2),
    ([2100, 0, 129, 1, 64], 2064, 272, SWIGLU, 1), ([700, 900], 1040, 2064, GELU, 1), ([70, 3], 272, 144, NONE, 2),
    ([700, 20], 528, 16, NONE, 2), (EDGES, 1040, 272, NONE, 2), (EDGES, 272, 400, SWIGLU, 2)]


@pytest.mark.parametrize("lengths,K,N,act,halves", GRADIENTS, ids=[i + f"h{c[4]}" for i, c in zip(ids(GRADIENTS), GRADIENTS)])
def test_dx(lengths, K, N, act, halves):
    g = torch.Generator(device="cuda").manual_seed(7)
    E, wide, rows = len(lengths), 2 if act == SWIGLU else 1, sum(lengths) + 2
    dy, dys, dy64, dyp = coded_rows(g, rows * halves, N, False)
    dy, dys, dy64 = dy.view(rows, halves * N), dys.view(rows, halves, -1), dy64.view(rows, halves * N)
    dys = dys if halves == 2 else dys[:, 0]
    # weights [E, halves * N, K] and their transposes
    w, ws, w64, _ = coded_weights(g, E, halves, N, K)
    wt, wts = w.transpose(1, 2).contiguous(), ws.permute(0, 3, 1, 2).contiguous()
    across = ws.double().repeat_interleave(128, 2).repeat_interleave(128, 3)[:, :, :N, :K].reshape(E, halves * N, K)
    wtp = F.peaks(wt, across.transpose(1, 2))
    z = normal(g, rows, wide * K, scale=2.0) if act else None
    dx, codes, scales = rooms(rows, K, wide)
    off = offsets_of(lengths, 99)
    want, tol, written = F.product_dx(dy64, dyp.view(rows, -1), off.tolist(), w64.transpose(1, 2), wtp, act, z)
    B.moe_expert_matmul_fp8_dx(dy, dys, off, wt, wts, act, z, dx, codes, scales)
    R.inside(dx[written], want[written], F.bf16(want, tol)[written], "dx")
    n = int(written.sum())
    F.check_codes(codes[written].view(n, wide, K), scales[written], want[written].view(n, wide, K), tol[written].view(n, wide, K), "dx")
    assert (dx[~written] == CANARY).all() and (codes[~written] == MARK).all() and (scales[~written] == CANARY).all()
    _, c, s = rooms(rows, K, wide)
    B.moe_expert_matmul_fp8_dx(dy, dys, off, wt, wts, act, z, None, c, s)
    assert torch.equal(c, codes) and torch.equal(s, scales)
    if act:  # in place of the pre-activations
        kept = z.clone()
        B.moe_expert_matmul_fp8_dx(dy, dys, off, wt, wts, act, z, z)
        assert torch.equal(z[written], dx[written]) and torch.equal(z[~written], kept[~written])


def test_repeats_are_equal_and_captured_too():
    case = check_product([300, 0, 70, 1], 1040, 272, SWIGLU, True, True, True, False)
    x, xs, off, w, ws, b, res, out, codes, scales, pre = case
    outs = [torch.zeros_like(t) for t in (out, codes, scales, pre)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        B.moe_expert_matmul_fp8(x, xs, off, w, ws, b, SWIGLU, res, outs[0], outs[1], outs[2][:, 0], outs[3])
    n = 371
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, (out, codes, scales, pre)):
            assert torch.equal(got[:n], want[:n]) and (got[n:] == 0).all()


# Codes of four neighbouring exponents: no product of eight loses a bit, so the
# sums are fp32's alone, and one wrong or missing code of thousands shows.
@pytest.mark.parametrize("lengths,K,N,act", [([1, 0, 3], 2048, 272, NONE), ([70, 6], 1040, 144, SILU), ([300], 400, 528, NONE),
                                             (EDGES, 2064, 1040, SWIGLU), (MANY, 1040, 2064, NONE)])
def test_sums_of_near_codes(lengths, K, N, act):
    g = torch.Generator(device="cuda").manual_seed(K)
    E, wide, rows = len(lengths), 2 if act == SWIGLU else 1, sum(lengths)

    def codes(*shape):
        c = torch.randint(7 << 3, 11 << 3, shape, generator=g, device="cuda")
        return (c + 128 * torch.randint(0, 2, shape, generator=g, device="cuda")).to(torch.uint8)

    x, xs = codes(rows, K), torch.rand(rows, F.blocks(K), generator=g, device="cuda")
    w, ws = codes(E * wide, N, K), torch.rand(E * wide, F.blocks(N), F.blocks(K), generator=g, device="cuda") * K ** -0.5
    x64 = F.e4m3(x) * F.at_columns(xs, K)
    w, ws, w64, wp = with_values(w, ws, E, wide, N, K)
    off = offsets_of(lengths)
    y, dy, z, dz, _ = F.product(x64, 0 * F.peaks(x, F.at_columns(xs, K)), off.tolist(), w64, wp, None, act, None)
    out, codes_out, scales = rooms(rows, N)
    B.moe_expert_matmul_fp8(x, xs, off, w, ws, None, act, None, out, codes_out, scales[:, 0])
    R.inside(out, y, F.bf16(y, dy), "out")
    F.check_codes(codes_out, scales[:, 0], y, dy, "out")


# few rows an expert: with a workspace their coded results take another way, where the
# sums are long
@pytest.mark.parametrize("lengths,K,N,act", [([1], 400, 144, SILU), ([1, 0, 3, 16, 1], 1040, 272, SWIGLU), ([2] * 9, 272, 2064, NONE),
                                             ([1] * 8 + [0] * 24, 2064, 768, SWIGLU)])
def test_few_coded_rows_without_a_workspace(lengths, K, N, act):
    x, xs, off, w, ws, b, res, out, codes, scales, _ = check_product(lengths, K, N, act, True, True, False, False)
    rows, E = x.shape[0], len(lengths)
    need = B.expert_fp8_workspace_bytes("moe_expert_matmul_fp8", E, rows, K, N, act)
    assert need == (rows * N * 4 if K > 1000 else 0)
    _, c, s = rooms(rows, N)
    B._call("moe_expert_matmul_fp8", None, x, xs, xs.shape[1], off, w, ws, b, act, res, E, rows, K, N, None, c, s, None, None, None)
    assert torch.equal(c, codes) and torch.equal(s, scales)


@pytest.mark.parametrize("lengths,K,N,act,halves", [([1], 144, 400, SILU, 1), ([1, 0, 3, 16, 1], 272, 1040, SWIGLU, 1),
                                                    ([1] * 8 + [0] * 24, 2064, 768, NONE, 2), ([3, 2], 4096, 528, SWIGLU, 2)])
def test_few_coded_gradients_without_a_workspace(lengths, K, N, act, halves):
    g = torch.Generator(device="cuda").manual_seed(8)
    E, wide, rows = len(lengths), 2 if act == SWIGLU else 1, sum(lengths)
    dy, dys, *_ = coded_rows(g, rows * halves, N, False)
    dy, dys = dy.view(rows, halves * N), dys.view(rows, halves, -1)
    wt, wts, *_ = coded_weights(g, E, 1, K, halves * 16 * (N // 16))
    wts = torch.rand(E, F.blocks(K), halves, F.blocks(N), generator=g, device="cuda")
    z = normal(g, rows, wide * K) if act else None
    off = offsets_of(lengths)
    need = B.expert_fp8_workspace_bytes("moe_expert_matmul_fp8_dx", E, rows, K, N, act, halves)
    assert need == (rows * wide * K * 4 if halves * N > 1000 else 0)
    dx, codes, scales = rooms(rows, K, wide)
    B.moe_expert_matmul_fp8_dx(dy, dys, off, wt, wts, act, z, dx, codes, scales)
    dx2, c, s = rooms(rows, K, wide)
    B._call("moe_expert_matmul_fp8_dx", None, dy, dys, off, wt, wts, halves, act, z, E, rows, K, N, dx2, c, s, None, None)
    assert torch.equal(dx, dx2) and torch.equal(c, codes) and torch.equal(s, scales)

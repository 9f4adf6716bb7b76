"""The residual's addition with the norm, and its gradient, against their 64-bit
forms."""
import pytest
import torch

import fp8_ref as F
import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

CANARY = -7.0
SIZES = [(1, 16), (1, 128), (3, 48), (5, 144), (33, 528), (7, 1040), (515, 2048), (2100, 2064), (130, 4112), (1, 7168),
         (70, 8192), (5, 8208), (3, 16384), (4, 16400), (3, 32768), (2, 65536), (9000, 64)]


def normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def room(T, H, dtype=torch.bfloat16):
    """T rows, and one behind them that no call may write."""
    whole = torch.full((T + 1, H), CANARY, dtype=dtype, device="cuda") if dtype != torch.uint8 else \
        torch.full((T + 1, H), 77, dtype=dtype, device="cuda")
    return whole, whole[:T]


def check_norm(T, H, residual, weight, row, eps=1e-6, scale=1.0, x=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + H)
    x = normal(g, T, H, scale=scale) if x is None else x
    r = normal(g, T, H, scale=2 * scale) if residual else None
    w = normal(g, H, dtype=torch.float32) if weight else None
    (all_s, s), (all_y, y), (all_c, c) = room(T, H), room(T, H), room(T, H, torch.uint8)
    nb = 1 if row else F.blocks(H)
    all_v, v = room(T, nb, torch.float32)
    B.moe_add_norm(x, r, w, eps, s, y, c, v.reshape(-1) if row else v)
    want_s, want_y, tol = F.norm(x, r, w, eps)
    R.inside(s, want_s, F.bf16(want_s, 0 * want_s), "sum")
    R.inside(y, want_y, F.bf16(want_y, tol), "y")
    F.check_codes(c, v, want_y, tol, "y")
    for whole, mark in ((all_s, CANARY), (all_y, CANARY), (all_c, 77), (all_v, CANARY)):
        assert (whole[T] == mark).all()
    return x, r, w, s, y, c, v


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("row", [True, False])
def test_norm(T, H, row):
    check_norm(T, H, True, True, row)


@pytest.mark.parametrize("T,H", [(3, 48), (66, 7168)])
def test_norm_without(T, H):
    """No residual, no weight, fewer outputs: the same values."""
    x, _, _, s, y, c, v = check_norm(T, H, False, False, False)
    assert torch.equal(s, x)
    only = torch.zeros_like(y)
    B.moe_add_norm(x, None, None, 1e-6, None, only)
    assert torch.equal(only, y)
    codes, scales = torch.zeros_like(c), torch.zeros_like(v)
    B.moe_add_norm(x, None, None, 1e-6, None, None, codes.view(torch.float8_e4m3fn), scales)
    assert torch.equal(codes, c) and torch.equal(scales, v)


@pytest.mark.parametrize("scale", [1e-15, 1e15])
def test_norm_of_small_and_large_rows(scale):
    check_norm(20, 528, True, True, False, eps=0.0 if scale > 1 else 1e-35, scale=scale)


def test_norm_in_place():
    x, r, w, s, y, c, v = check_norm(50, 1040, True, True, False)
    a, b = x.clone(), r.clone()
    B.moe_add_norm(a, b, w, 1e-6, b, a)  # the stream in place, the normed rows over x
    assert torch.equal(a, y) and torch.equal(b, s)


@pytest.mark.parametrize("H", [144, 2064, 8208])
@pytest.mark.parametrize("row", [True, False])
def test_norm_of_zeros_and_of_nan(H, row):
    """A zero row has zero codes and scales; a NaN or an infinity shows in its own
    row and reaches no other."""
    x = torch.ones(9, H, device="cuda").bfloat16()
    x[2] = 0
    x[4, 5], x[6, H - 1] = float("nan"), float("inf")
    s, y, c = torch.zeros_like(x), torch.zeros_like(x), torch.zeros(9, H, dtype=torch.uint8, device="cuda")
    v = torch.zeros(9, device="cuda") if row else torch.zeros(9, F.blocks(H), device="cuda")
    B.moe_add_norm(x, None, None, 1e-6, s, y, c, v)
    assert torch.equal(s.view(torch.int16), x.view(torch.int16))
    assert (y[2] == 0).all() and (c[2] == 0).all() and (v[2] == 0).all()
    assert torch.isnan(y[4]).all() and torch.isnan(v[4]).all()
    assert torch.isnan(y[6, H - 1]) and torch.isnan(v[6]).any()  # the root of an infinity: zeros, and inf * 0
    fine = [0, 1, 3, 5, 7, 8]
    assert (y[fine] == 1).all() and torch.isfinite(v[fine]).all()
    values = F.e4m3(c) * (v[:, None] if row else F.at_columns(v, H))
    assert ((values[fine] - 1).abs() < 1e-5).all()


def test_repeats_are_equal_and_captured_too():
    x, r, w, s, y, c, v = check_norm(300, 2064, True, True, False)
    d_y, ds = x.flip(0).contiguous(), r.flip(0).contiguous()
    d_x, d_w = torch.zeros_like(x), torch.zeros(2064, device="cuda")
    B.moe_add_norm_grad(d_y, ds, s, w, 1e-6, d_x, d_w)
    outs = [torch.zeros_like(t) for t in (s, y, c, v, d_x, d_w)]
    work = torch.empty(B.add_norm_grad_workspace_bytes(300, 2064), dtype=torch.uint8, device="cuda")
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        B.moe_add_norm(x, r, w, 1e-6, *outs[:4])
        B.moe_add_norm_grad(d_y, ds, outs[0], w, 1e-6, outs[4], outs[5], workspace=work)
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, (s, y, c, v, d_x, d_w)):
            assert torch.equal(got, want)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("stream", [True, False])
def test_norm_grad(T, H, stream):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    s, d_y, w = normal(g, T, H, scale=2.0), normal(g, T, H), normal(g, H, dtype=torch.float32)
    ds = normal(g, T, H) if stream else None
    whole, d_x = room(T, H)
    d_w = torch.full((H,), CANARY, device="cuda")
    B.moe_add_norm_grad(d_y, ds, s, w, 1e-6, d_x, d_w)
    want, tol, want_w, tol_w = F.norm_grad(d_y, ds, s, w, 1e-6)
    R.inside(d_x, want, F.bf16(want, tol), "d_x")
    R.inside(d_w, want_w, tol_w, "d_weight")
    assert (whole[T] == CANARY).all()
    before = d_w.clone()
    B.moe_add_norm_grad(d_y, ds, s, w, 1e-6, d_x, d_w, accumulate=True)
    assert torch.equal(d_w, before + before) or ((d_w - 2 * before).abs() <= 2 * tol_w + 4 * F.U32 * before.abs()).all()
    kept = d_x.clone()
    for name in ("d_y", "d_sum", "sum"):  # in place of each, and without d_weight
        a = dict(d_y=d_y.clone(), d_sum=None if ds is None else ds.clone(), sum=s.clone())
        if a[name] is not None:
            B.moe_add_norm_grad(a["d_y"], a["d_sum"], a["sum"], w, 1e-6, a[name])
            assert torch.equal(a[name], kept), name


def test_norm_grad_without_weight_and_of_no_rows():
    g = torch.Generator(device="cuda").manual_seed(1)
    s, d_y = normal(g, 40, 272), normal(g, 40, 272)
    d_x, d_w = torch.zeros_like(s), torch.full((272,), CANARY, device="cuda")
    B.moe_add_norm_grad(d_y, None, s, None, 1e-6, d_x, d_w)
    want, tol, want_w, tol_w = F.norm_grad(d_y, None, s, None, 1e-6)
    R.inside(d_x, want, F.bf16(want, tol), "d_x")
    R.inside(d_w, want_w, tol_w, "d_weight")
    kept = d_w.clone()
    none = s[:0]
    B.moe_add_norm(none, none, None, 1e-6, none, none)
    B.moe_add_norm_grad(none, None, none, None, 1e-6, none, d_w, accumulate=True)
    assert torch.equal(d_w, kept)
    B.moe_add_norm_grad(none, None, none, None, 1e-6, none, d_w)
    assert (d_w == 0).all()


@pytest.mark.parametrize("H", [48, 272])
def test_norm_grad_against_differences(H):
    """The gradient of sum(y * d_y) against central differences of the 64-bit
    norm: their error is of the third derivative, below 1e-6 of the sizes here."""
    g = torch.Generator(device="cuda").manual_seed(H)
    s, d_y, w = normal(g, 4, H, scale=2.0), normal(g, 4, H), normal(g, H, dtype=torch.float32)
    d_x, d_w = torch.zeros_like(s), torch.zeros(H, device="cuda")
    B.moe_add_norm_grad(d_y, None, s, w, 1e-6, d_x, d_w)

    def loss(s64, w64):
        return (s64 * torch.rsqrt((s64 * s64).mean(1, keepdim=True) + 1e-6) * w64 * d_y.double()).sum()

    h = 1e-4
    for i in (0, 1, H // 2, H - 1):
        e = torch.zeros(4, H, dtype=torch.float64, device="cuda")
        e[2, i] = h
        num = (loss(s.double() + e, w.double()) - loss(s.double() - e, w.double())) / (2 * h)
        assert abs(num - d_x[2, i].double()) <= F.UBF16 * abs(num) + 1e-5
        e = torch.zeros(H, dtype=torch.float64, device="cuda")
        e[i] = h
        num = (loss(s.double(), w.double() + e) - loss(s.double(), w.double() - e)) / (2 * h)
        assert abs(num - d_w[i].double()) <= 1e-5

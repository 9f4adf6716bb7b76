"""moe_combine_grad against its 64-bit form, for every payload format."""
import numpy as np
import pytest
import torch

import training_ref as R
from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

# T, H, k, quant, dropped share
CASES = [(1, 16, 1, 0, 0.0), (1, 32, 16, 2, 0.0), (33, 528, 3, 0, 0.2), (100, 2048, 8, 1, 0.1), (64, 7168, 8, 0, 0.0),
         (50, 7168, 8, 1, 0.1), (50, 7168, 8, 2, 0.1), (50, 7168, 8, 3, 0.1), (7, 16, 16, 1, 0.5), (9, 48, 2, 3, 1.0),
         (5, 65536, 2, 0, 0.3), (5, 65536, 2, 1, 0.3), (5, 65536, 3, 2, 0.3), (3, 16384, 5, 0, 0.0), (3, 32768, 5, 0, 0.0),
         (3, 20000, 5, 3, 0.0), (2000, 1040, 7, 0, 0.1)]


def payload(T, H, k, quant, dropped, seed=0):
    """Random rows as codes, their scales, their values in 64 bits, and pos."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = T * k
    kept = torch.rand(n, generator=g, device="cuda") >= dropped
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots = kept.nonzero()[:, 0]
    pos[slots] = torch.randperm(len(slots), generator=g, device="cuda").int()
    scales = torch.rand(n, generator=g, device="cuda") + 0.01
    if quant == 0:
        rows = torch.randn(n, H, generator=g, device="cuda").bfloat16()
        return rows, None, rows.double(), pos
    if quant == 3:
        rows = (torch.randn(n, H, generator=g, device="cuda") * 50).to(torch.float8_e4m3fn)
        values = rows.double()
        rows = rows.view(torch.uint8)
    else:
        top = 127 if quant == 1 else 7
        codes = torch.randint(-top, top + 1, (n, H), generator=g, device="cuda")
        values = codes.double()
        rows = codes.to(torch.int8) if quant == 1 else ((codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)).to(torch.uint8)
    return rows, scales, values * scales.double()[:, None], pos


def reference(d_out, values, pos, w, T, H, k):
    at = pos.view(T, k).long()
    kept = at >= 0
    d = d_out.double()
    d_w, size = torch.zeros(T, k, dtype=torch.float64, device="cuda"), torch.zeros(T, k, dtype=torch.float64, device="cuda")
    rows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = kept[:, j].nonzero()[:, 0]
        v = values[at[t, j]]
        d_w[t, j], size[t, j] = (v * d[t]).sum(1), (v * d[t]).abs().sum(1)
        rows[at[t, j]] = d[t] * w.double()[t, j, None]
    return rows, d_w, size


@pytest.mark.parametrize("parts", ["both", "rows", "gates"])
@pytest.mark.parametrize("T,H,k,quant,dropped", CASES)
def test_combine_grad(T, H, k, quant, dropped, parts):
    rows, scales, values, pos = payload(T, H, k, quant, dropped)
    g = torch.Generator(device="cuda").manual_seed(5)
    d_out = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    w = torch.randn(T, k, generator=g, device="cuda")
    d_rows = torch.full((T * k, H), -7.0, dtype=torch.bfloat16, device="cuda") if parts != "gates" else None
    d_w = torch.full((T, k), -7.0, device="cuda") if parts != "rows" else None
    B.moe_combine_grad(d_out, rows if parts != "rows" else None, scales if parts != "rows" else None, quant, pos, w,
                       T, H, k, d_rows, d_w)
    torch.cuda.synchronize()
    want, want_w, size = reference(d_out, values, pos, w, T, H, k)
    if d_rows is not None:
        n = int((pos >= 0).sum())
        R.inside(d_rows[:n], want[:n], want[:n].abs() * R.UBF16 * (1 + 2.0 ** -14), "d_rows")
        assert (d_rows[n:] == -7).all()
    if d_w is not None:
        # a thread adds up to 64 products, then 6 steps over the wave and 16 over the waves
        R.inside(d_w, want_w, size * (64 + 6 + 16 + 4) * R.U32, "d_w")
        assert not d_w[pos.view(T, k) < 0].any()


@pytest.mark.parametrize("parts", ["both", "rows", "gates"])
@pytest.mark.parametrize("T,H,k,quant,dropped", [(1, 16, 16, 0, 0.0), (4097, 16, 10, 1, 0.5), (333, 32, 16, 2, 0.1), (50, 64, 7, 3, 0.2),
                                                 (1001, 48, 9, 0, 0.1), (77, 96, 12, 1, 0.1), (6, 256, 3, 2, 0.3), (500, 240, 16, 0, 0.0),
                                                 (30, 272, 5, 1, 0.1), (30000, 256, 8, 0, 0.1), (30000, 256, 8, 3, 0.1)])
def test_short_rows(T, H, k, quant, dropped, parts):
    test_combine_grad(T, H, k, quant, dropped, parts)


@pytest.mark.parametrize("parts", ["both", "rows", "gates"])
@pytest.mark.parametrize("quant", range(4))
def test_rows_past_the_last_level_cache(quant, parts):
    """More than 256 MiB of gradient rows."""
    test_combine_grad(2060, 8192, 8, quant, 0.01, parts)


def test_dropped_rows_are_not_read():
    """NaN in rows that no slot points to reaches nothing."""
    T, H, k = 40, 256, 4
    rows, _, values, pos = payload(T, H, k, 0, 0.5)
    n = int((pos >= 0).sum())
    rows[n:] = float("nan")
    d_out, w = torch.randn(T, H, device="cuda").bfloat16(), torch.rand(T, k, device="cuda")
    d_rows, d_w = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, k, device="cuda")
    B.moe_combine_grad(d_out, rows, None, 0, pos, w, T, H, k, d_rows, d_w)
    assert torch.isfinite(d_rows).all() and torch.isfinite(d_w).all()


def test_gradient_of_the_combine_itself():
    """<d_out, combine(rows + h a) - combine(rows - h a)> = 2 h <d_rows, a>, and
    alike for the weights, with h a power of two and exact bf16 inputs, so the
    combine's own outputs are the only roundings."""
    T, H, k = 32, 512, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda").float()  # noqa: E731
    rows, a = ints(T * k, H), ints(T * k, H)
    w, b = ints(T, k) / 4, ints(T, k) / 4
    d_out = ints(T, H)
    pos = torch.randperm(T * k, generator=g, device="cuda").int()
    d_rows, d_w = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, k, device="cuda")
    B.moe_combine_grad(d_out.bfloat16(), rows.bfloat16(), None, 0, pos, w, T, H, k, d_rows, d_w)

    def out(r, w):
        o = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        B.moe_combine(r.bfloat16(), None, 0, pos, w.contiguous(), T, H, k, o)
        return o.double()

    # small integers and quarters: every product and sum here is exact in bf16
    # (|values| <= 4 * 4 * 9 / 4 < 64 in quarters) and in fp32
    d = d_out.double()
    assert ((out(rows + a, w) - out(rows - a, w)) * d).sum() == 2 * (d_rows.double() * a.double()).sum()
    assert ((out(rows, w + b) - out(rows, w - b)) * d).sum() == 2 * (d_w.double() * b.double()).sum()


def test_combine_grad_in_a_graph():
    T, H, k = 300, 512, 4
    rows, scales, _, pos = payload(T, H, k, 1, 0.1)
    d_out, w = torch.randn(T, H, device="cuda").bfloat16(), torch.rand(T, k, device="cuda")
    outs = [(torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, k, device="cuda")) for _ in range(2)]
    call = lambda o: B.moe_combine_grad(d_out, rows, scales, 1, pos, w, T, H, k, *o)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs[0])
    for s in range(3):
        d_out.copy_(torch.randn(T, H, device="cuda"))
        w.copy_(torch.rand(T, k, device="cuda"))
        graph.replay()
        call(outs[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])

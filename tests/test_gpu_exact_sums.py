"""Long sums of -1, 0 and 1: every partial sum is a whole number below 2^24, so
exact in fp32 in any order, and one lost or doubled row or step shows.  (Against
bounds that grow with the number of terms a lost tail of random values does
not.)"""
import pytest
import torch

from combine_fp32_router_amd import binding as B

pytestmark = pytest.mark.gpu

NONE = B.MOE_ACT_NONE


def ints(g, *shape):
    """-1, 0 or 1, none of them 0 along the last rows and columns."""
    t = torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8)
    t[..., -1:, :] = 1 - 2 * (t[..., -1:, :] < 0).to(torch.int8)
    t[..., :, -1:] = 1 - 2 * (t[..., :, -1:] < 0).to(torch.int8)
    return t.bfloat16()


def offsets_of(lengths):
    return torch.tensor([sum(lengths[:e]) for e in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def product64(a, b):
    """a b^T of whole numbers, exact, as fp32."""
    return (a.double() @ b.double().T.contiguous()).float()


# runs, K, N: for few rows, whole tiles of every height, in parts
PRODUCTS = [([1], 65536, 64), ([3, 0, 17, 1], 8208, 80), ([40, 9], 4176, 528), ([64] * 4, 2064, 272),
            ([5000, 3], 4112, 640), ([700, 65, 0, 1], 2064, 1040), ([3000, 129], 8208, 2064),
            ([2000, 0, 100], 4112, 384), ([8000], 8208, 48), ([900, 1, 64], 6160, 368)]


@pytest.mark.parametrize("lengths,K,N", PRODUCTS, ids=[f"E{len(s[0])}r{sum(s[0])}K{s[1]}N{s[2]}" for s in PRODUCTS])
def test_product_and_dx(lengths, K, N):
    """dx is the same product with its weights the other way round."""
    g = torch.Generator(device="cuda").manual_seed(K)
    rows, E = sum(lengths), len(lengths)
    x, w, off = ints(g, rows, K), ints(g, E, N, K), offsets_of(lengths)
    want = torch.cat([product64(r, w[e]) for e, r in enumerate(x.split(lengths))]).bfloat16()
    out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul(x, off, w, None, NONE, None, out)
    assert torch.equal(out, want)
    back = w.transpose(1, 2).contiguous()
    dx = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul_dx(x, off, back, NONE, None, dx)
    assert torch.equal(dx, want)


# runs, K, N: whole tiles (of 256, 128, 64 rows, more runs than are ordered), then in parts;
# ends of a step of 64, of one row, of 63 and of a last part shorter than the others
GRADIENTS = [([3001], 2064, 2064), ([0, 40, 9000, 3, 64], 1040, 1296), ([700, 1, 4097], 1040, 4112), ([193] * 70, 144, 272),
             ([30000, 1, 63], 528, 1040),
             ([9, 30000, 0], 16, 16), ([15000, 707], 192, 544), ([8192], 1040, 272), ([8193], 144, 272), ([0, 0, 9023], 128, 80),
             ([16385, 1], 16, 48), ([70001], 64, 64), ([4096 + 64 * 5, 33], 80, 144)]


@pytest.mark.parametrize("lengths,K,N", GRADIENTS, ids=[f"E{len(s[0])}r{sum(s[0])}K{s[1]}N{s[2]}" for s in GRADIENTS])
def test_dw(lengths, K, N):
    g = torch.Generator(device="cuda").manual_seed(N)
    rows, E = sum(lengths), len(lengths)
    dy, x, off = ints(g, rows, N), ints(g, rows, K), offsets_of(lengths)
    parts = list(zip(dy.split(lengths), x.split(lengths)))
    want = torch.stack([product64(d.T.contiguous(), r.T.contiguous()) for d, r in parts])
    want_b = torch.stack([d.double().sum(0).float() for d, _ in parts])
    dw, db = torch.full((E, N, K), -7.0, device="cuda"), torch.full((E, N), -7.0, device="cuda")
    B.moe_expert_matmul_dw(dy, x, off, dw, db)
    assert torch.equal(dw, want) and torch.equal(db, want_b)
    half = torch.full((E, N, K), -7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_matmul_dw(dy, x, off, half)
    assert torch.equal(half, want.bfloat16())
    B.moe_expert_matmul_dw(dy, x, off, dw, db, accumulate=True)
    assert torch.equal(dw, 2 * want) and torch.equal(db, 2 * want_b)


def test_dw_past_32_bit_offsets():
    """70001 rows of 32768 columns: 4.6 GB."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, K, N = 70001, 16, 32768
    dy, x = ints(g, rows, N), ints(g, rows, K)
    dw, db = torch.empty(1, N, K, device="cuda"), torch.empty(1, N, device="cuda")
    B.moe_expert_matmul_dw(dy, x, offsets_of([rows]), dw, db)
    for a in (0, 16384 - 64, N - 128):
        d = dy[:, a:a + 128].contiguous()
        assert torch.equal(dw[0, a:a + 128], product64(d.T.contiguous(), x.T.contiguous()))
        assert torch.equal(db[0, a:a + 128], d.double().sum(0).float())


# T, H, k, quant
GATES = [(3, 65536, 2, 0), (3, 65536, 2, 1), (3, 65536, 3, 2), (3, 65536, 2, 3), (65, 7168, 8, 0), (65, 7168, 8, 1), (65, 1040, 5, 3),
         (101, 96, 16, 2), (101, 48, 9, 0), (2060, 8192, 8, 1)]


@pytest.mark.parametrize("T,H,k,quant", GATES)
def test_gates_of_the_combine(T, H, k, quant):
    """Rows, output gradients and scales all whole: the gate weights' gradients
    come out exactly."""
    g = torch.Generator(device="cuda").manual_seed(H)
    rows, d_out = ints(g, T * k, H), ints(g, T, H)
    scales = torch.randint(1, 4, (T * k,), generator=g, device="cuda").float() if quant else None
    values = rows.double() * (scales.double()[:, None] if quant else 1.0)
    if quant == 1:
        rows = rows.to(torch.int8)
    elif quant == 2:
        c = rows.to(torch.int8).int()
        rows = ((c[:, 0::2] & 15) | ((c[:, 1::2] & 15) << 4)).to(torch.uint8)
    elif quant == 3:
        rows = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    pos = torch.randperm(T * k, generator=g, device="cuda").int()
    d_w = torch.zeros(T, k, device="cuda")
    B.moe_combine_grad(d_out, rows, scales, quant, pos, torch.ones(T, k, device="cuda"), T, H, k, None, d_w)
    want = (values[pos.long()].view(T, k, H) * d_out.double()[:, None]).sum(2)
    assert torch.equal(d_w.double(), want)

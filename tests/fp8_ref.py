"""64-bit reference forms of the norm, of E4M3 codes and of the products of
coded rows and weights, with bounds on how far 32-bit arithmetic may be off.

u is half a step of fp32.  A value rounded to E4M3 is off by at most 2^-4 of its
size, or by half of the subnormals' step 2^-9."""
import torch

import training_ref as R

U32, UBF16, UE4M3, LEAST = R.U32, R.UBF16, 2.0 ** -4, 2.0 ** -10
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def e4m3(codes):
    """The values of codes (uint8 or float8_e4m3fn) in 64 bits."""
    return codes.view(torch.float8_e4m3fn).double()


def at_columns(scales, n):
    """Scales [..., blocks of n] at every one of n columns."""
    return scales.double().repeat_interleave(BLOCK, -1)[..., :n]


def tops(v):
    """Largest size of each block of v [..., n]."""
    n = v.shape[-1]
    v = torch.nn.functional.pad(v.abs(), (0, blocks(n) * BLOCK - n))
    return v.view(*v.shape[:-1], blocks(n), BLOCK).amax(-1)


def coded(x, rows=1, cols=BLOCK):
    """(codes, scales) of x [..., R, C] by blocks of rows x cols: some, not the
    kernel's."""
    r, c = x.shape[-2:]
    nr, nc = -(-r // rows), -(-c // cols)
    v = torch.nn.functional.pad(x.float(), (0, nc * cols - c, 0, nr * rows - r)).view(*x.shape[:-2], nr, rows, nc, cols)
    scales = v.abs().amax((-3, -1)) / 448
    v = (v / scales.clamp(min=1e-30)[..., :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    v = v.view(torch.uint8).reshape(*x.shape[:-2], nr * rows, nc * cols)[..., :r, :c].contiguous()
    return v.view(torch.float8_e4m3fn), scales


def check_codes(codes, scales, y, dy, what):
    """Codes of y (64 bits, known to dy) with a scale for each block of its last
    dimension, or scales of shape [rows, 1] for whole rows."""
    n = y.shape[-1]
    row = scales.shape[-1] == 1 and blocks(n) > 1
    top, off = (y.abs().amax(-1, keepdim=True), dy.amax(-1, keepdim=True)) if row else (tops(y), tops(dy))
    R.inside(scales, top / 448, off / 448 + 4 * U32 * (top + off) / 448, what + " scales")
    s = scales.double().expand(y.shape) if row else at_columns(scales, n)
    live = s > 0
    s = torch.where(live, s, 1.0)
    q, dq = y / s, dy / s + 4 * U32 * (y / s).abs()
    # (a quotient is at most 448, but for the noise of its scale)
    tol = dq + torch.maximum(UE4M3 * (q.abs() + dq), torch.full_like(q, LEAST))
    got = e4m3(codes)
    R.inside(got[live], q[live], tol[live], what + " codes")
    assert (got[~live] == 0).all() and (y.abs()[~live] <= dy[~live]).all(), what + " zeros"


def norm(x, residual, weight, eps):
    """(s, y, bound of y) in 64 bits.  A lane adds at most 64 squares, and sums of
    lanes meet in under 32 steps; the root halves what the mean is off."""
    s = x.double() if residual is None else x.double() + residual.double()
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    return s, y, (96 / 2 + 8) * U32 * y.abs()


def norm_grad(d_y, d_sum, s, weight, eps):
    """(d_x, its fp32 bound, d_weight, its bound)."""
    s, d_y = s.double(), d_y.double()
    n, T = s.shape[1], s.shape[0]
    r = torch.rsqrt((s * s).mean(1, keepdim=True) + eps)
    g = d_y if weight is None else d_y * weight.double()
    back, size = (g * s).mean(1, keepdim=True), (g * s).abs().mean(1, keepdim=True)
    d_x = r * g - s * r ** 3 * back
    rel = 96 / 2 + 8
    tol = U32 * (rel * (r * g).abs() + s.abs() * r ** 3 * (3 * rel * back.abs() + 104 * size))
    if d_sum is not None:
        d_x = d_x + d_sum.double()
        tol = tol + 2 * U32 * (d_x.abs() + tol)
    return d_x, tol, (d_y * s * r).sum(0), (rel + T + 64) * U32 * (d_y * s * r).abs().sum(0)


def peaks(codes, scales):
    """2^e of the largest exponent field among each 8 consecutive codes [..., n] (a
    subnormal's is -6), times their scale (scales [..., n])."""
    e = (codes.view(torch.uint8).int() >> 3 & 15).clamp(min=1) - 7
    return (torch.exp2(e.double()) * scales).unflatten(-1, (codes.shape[-1] // 8, 8)).amax(-1)


# What the matrix cores do with a product's codes, found by giving them every
# pair of codes: of each 8 consecutive products they keep the bits down to 2^-13
# of 2^(the largest sum of two exponent fields), and drop the rest towards zero.
# The largest product itself has six bits behind its first and loses nothing, so
# 8 products are off by less than 7 * 2^-13 * 2^(that sum), which the peaks of
# both sides' eight bound.  The sums of eights, and what a sum's last bit cannot
# hold (dropped or rounded, so 2 u), are fp32's, as are the scales and the blocks.
def _sums(x, xp, w, wp):
    z = x @ w.T
    return z, (x.abs() @ w.abs().T) * (2 * x.shape[1] + 8) * U32 + 7 * 2.0 ** -13 * (xp @ wp.T)


def product(x, xp, offsets, w, wp, bias, act, residual):
    """(y, its fp32 bound, z, its fp32 bound, written rows) of dequantised rows
    and weights (64 bits) with their peaks."""
    rows, E, wide_n = x.shape[0], w.shape[0], w.shape[1]
    z = torch.zeros(rows, wide_n, dtype=torch.float64, device=x.device)
    dz = torch.zeros_like(z)
    written = torch.zeros(rows, dtype=torch.bool, device=x.device)
    for e, a, b in R.runs(offsets, rows):
        if b <= a:
            continue
        z[a:b], dz[a:b] = _sums(x[a:b], xp[a:b], w[e], wp[e])
        if bias is not None:
            z[a:b] += bias.view(E, wide_n)[e].double()
            dz[a:b] += U32 * z[a:b].abs()
        written[a:b] = True
    if act == 4:
        N = wide_n // 2
        zg, zu = z[:, :N], z[:, N:]
        s, _ = R.act64(zg, 2)
        y = s * zu
        gate = 1.1 * dz[:, :N] + R.act_noise(zg)
        dy = gate * (zu.abs() + dz[:, N:]) + dz[:, N:] * (s.abs() + 1e-6)
    else:
        y, slope = R.act64(z, act)
        dy = slope * dz + (R.act_noise(z) if act in (2, 3) else 0.0)
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2 * U32 * y.abs()
    return y, dy, z, dz, written


def product_dx(dy, dyp, offsets, wt, wtp, act, z):
    """(dx, its fp32 bound, written rows); wt [E, K, N] in 64 bits."""
    rows, K = dy.shape[0], wt.shape[1]
    g = torch.zeros(rows, K, dtype=torch.float64, device=dy.device)
    dg = torch.zeros_like(g)
    written = torch.zeros(rows, dtype=torch.bool, device=dy.device)
    for e, a, b in R.runs(offsets, rows):
        if b > a:
            g[a:b], dg[a:b] = _sums(dy[a:b], dyp[a:b], wt[e], wtp[e])
            written[a:b] = True
    if act == 4:
        zg, zu = z[:, :K].double(), z[:, K:].double()
        a, b = zu * R.slope64(zg, 2), R.act64(zg, 2)[0]
        out = torch.cat([g * a, g * b], 1)
        tol = torch.cat([dg * a.abs() + g.abs() * R.act_noise(zg) * zu.abs(),
                         dg * b.abs() + g.abs() * R.act_noise(zg)], 1)
    elif act:
        a = R.slope64(z.double(), act)
        out, tol = g * a, dg * a.abs() + g.abs() * R.act_noise(z.double())
    else:
        out, tol = g, dg
    return out, tol + 4 * U32 * out.abs(), written


def bf16(y, dy):
    """The bound of y rounded to bf16."""
    return dy + UBF16 * (y.abs() + dy)

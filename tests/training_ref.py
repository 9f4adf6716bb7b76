"""64-bit reference forms of the training and expert operators, each with a
bound on how far a kernel in 32-bit arithmetic may be from it.

u is half a step of fp32 (2^-24); a sum of n terms taken in any order is off
by at most n u times the sum of the terms' sizes, and a value rounded once to
bf16 by at most 2^-8 of its size."""
import numpy as np
import torch

U32 = 2.0 ** -24
UBF16 = 2.0 ** -8


def dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).cuda()


def balance(logits, idx, mask, seg, E, k):
    """Per segment: loss, counts, prob_sums, live; and p [T, E] (0 where masked)."""
    T = logits.shape[0]
    live = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    z = np.zeros((T, E))
    z[live] = logits[live].astype(np.float64)
    p = np.exp(z - z.max(axis=1, keepdims=True)) if T else z
    p = p / p.sum(axis=1, keepdims=True) * live[:, None] if T else p
    S = max(1, -(-T // seg)) if T else 1
    counts, sums = np.zeros((S, E), np.int64), np.zeros((S, E))
    tokens, loss = np.zeros(S, np.int64), np.zeros(S)
    for s in range(S):
        at = slice(s * seg, min(T, (s + 1) * seg))
        ids = idx[at][live[at]].ravel()
        counts[s] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        sums[s] = p[at].sum(axis=0)
        tokens[s] = live[at].sum()
        if tokens[s]:
            loss[s] = E / (k * float(tokens[s]) ** 2) * (counts[s] * sums[s]).sum()
    return loss, counts, sums, tokens, p


def softmax_rel_bound(logits, mask, E, adds):
    """Relative bound of a probability, and of a sum of `adds` of them in a
    lane: the exponent's argument is rounded once (a relative error of its
    size in units of 2 u), expf and the division by a sum of E terms add
    their own roundings."""
    live = np.ones(len(logits), bool) if mask is None else np.asarray(mask) != 0
    z = logits[live].astype(np.float64)
    z = z[np.isfinite(z)]
    spread = z.max() - z.min() if z.size else 0.0
    return (min(spread, 110.0) + E / 16 + 12 + adds) * 2 * U32


def route_grad(p, idx, w, d_w, live, d_loss, counts, tokens, seg, E, k, rel):
    """d_logits and its bound; d_w or d_loss may be None.  `rel` bounds p."""
    T = idx.shape[0]
    d, tol = np.zeros((T, E)), np.zeros((T, E))
    if d_loss is not None:
        for s in range(len(d_loss)):
            at = slice(s * seg, min(T, (s + 1) * seg))
            if tokens[s] == 0:
                continue
            scale = float(d_loss[s]) * E / (k * float(tokens[s]) ** 2)
            c = counts[s].astype(np.float64)
            mean = (p[at] * c).sum(axis=1, keepdims=True)
            d[at] = scale * p[at] * (c - mean)
            tol[at] = abs(scale) * p[at] * (c + mean) * (2 * rel + (E / 16 + 16) * U32)
    if d_w is not None:
        w, d_w = w.astype(np.float64), d_w.astype(np.float64)
        g = w * (d_w - (w * d_w).sum(axis=1, keepdims=True))
        size = w * (np.abs(d_w) + np.abs(w * d_w).sum(axis=1, keepdims=True))
        for j in range(k):
            ok = (idx[:, j] >= 0) & (idx[:, j] < E)
            t = np.nonzero(ok)[0]
            d[t, idx[t, j]] += g[t, j]
            tol[t, idx[t, j]] += size[t, j] * (k + 8) * U32
    d[~live], tol[~live] = 0.0, 0.0
    return d, tol + 4 * U32 * np.abs(d)


def act64(z, act):
    """act(z) and a bound on its slope, elementwise (SwiGLU is handled apart)."""
    if act == 1:
        return z.clamp(min=0), 1.0
    if act == 2:
        return z * torch.sigmoid(z), 1.1
    if act == 3:
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5)), 1.13
    return z, 1.0


def slope64(z, act):
    if act == 1:
        return (z > 0).double()
    if act == 2:
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == 3:
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) / (2 * np.pi) ** 0.5
    return torch.ones_like(z)


# An activation evaluated in fp32 is off by a few u of its terms (1 + erf and
# 1 + z (1 - s) cancel, so the terms are bounded by 1 + |z|).
def act_noise(z):
    return 16 * U32 * (1 + z.abs())


def runs(offsets, rows):
    """(expert, first, end) of every run, cut at `rows`."""
    o = [min(max(int(v) - int(offsets[0]), 0), rows) for v in offsets]
    return [(e, o[e], max(o[e], o[e + 1])) for e in range(len(o) - 1)]


def product(x, offsets, w, bias, act, residual):
    """(out, its bound, z, its bound, written rows) in 64 bits on x's device."""
    rows, K = x.shape
    E, wide_n, _ = w.shape
    z = torch.zeros(rows, wide_n, dtype=torch.float64, device=x.device)
    dz = torch.zeros_like(z)
    written = torch.zeros(rows, dtype=torch.bool, device=x.device)
    for e, a, b in runs(offsets, rows):
        if b <= a:
            continue
        xe, we = x[a:b].double(), w[e].double()
        z[a:b], dz[a:b] = xe @ we.T, (xe.abs() @ we.abs().T) * (K * U32)
        if bias is not None:
            z[a:b] += bias.view(E, wide_n)[e].double()
            dz[a:b] += U32 * z[a:b].abs()
        written[a:b] = True
    if act == 4:
        N = wide_n // 2
        zg, zu = z[:, :N], z[:, N:]
        s, _ = act64(zg, 2)
        y = s * zu
        dy = (1.1 * dz[:, :N] + act_noise(zg)) * zu.abs() + dz[:, N:] * (s.abs() + 1e-6)
    else:
        y, slope = act64(z, act)
        dy = slope * dz + (act_noise(z) if act in (2, 3) else 0.0)
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2 * U32 * y.abs()
    return y, dy + UBF16 * (y.abs() + dy), z, dz + UBF16 * (z.abs() + dz), written


def product_dx(dy, offsets, w, act, z):
    rows = dy.shape[0]
    E, N, K = w.shape
    g = torch.zeros(rows, K, dtype=torch.float64, device=dy.device)
    dg = torch.zeros_like(g)
    written = torch.zeros(rows, dtype=torch.bool, device=dy.device)
    for e, a, b in runs(offsets, rows):
        if b > a:
            d, we = dy[a:b].double(), w[e].double()
            g[a:b], dg[a:b] = d @ we, (d.abs() @ we.abs()) * (N * U32)
            written[a:b] = True
    if act == 4:
        zg, zu = z[:, :K].double(), z[:, K:].double()
        a, b = zu * slope64(zg, 2), act64(zg, 2)[0]
        out = torch.cat([g * a, g * b], 1)
        tol = torch.cat([dg * a.abs() + g.abs() * act_noise(zg) * zu.abs(),
                         dg * b.abs() + g.abs() * act_noise(zg)], 1)
    elif act:
        a = slope64(z.double(), act)
        out, tol = g * a, dg * a.abs() + g.abs() * act_noise(z.double())
    else:
        out, tol = g, dg
    tol = tol + 4 * U32 * out.abs()
    return out, tol + UBF16 * (out.abs() + tol), written


def product_dw(dy, x, offsets, E):
    """(dw, its fp32 bound, db, its bound)."""
    rows, N, K = dy.shape[0], dy.shape[1], x.shape[1]
    dw = torch.zeros(E, N, K, dtype=torch.float64, device=dy.device)
    db = torch.zeros(E, N, dtype=torch.float64, device=dy.device)
    tw, tb = torch.zeros_like(dw), torch.zeros_like(db)
    for e, a, b in runs(offsets, rows):
        if b > a:
            d, xe = dy[a:b].double(), x[a:b].double()
            n = b - a
            dw[e], tw[e] = d.T @ xe, (d.abs().T @ xe.abs()) * (n * U32)
            db[e], tb[e] = d.sum(0), d.abs().sum(0) * (n * U32)
    return dw, tw, db, tb


def inside(got, want, tol, what):
    got, want, tol = (t.double() if isinstance(t, torch.Tensor) else torch.as_tensor(t).double()
                      for t in (got, want, tol))
    got = got.to(want.device)
    err = (got - want).abs()
    bad = ~(err <= tol + 1e-37)  # NaN counts as outside
    worst = (err / (tol + 1e-37)).max().item() if err.numel() else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {worst:.3g} x"

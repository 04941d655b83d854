"""Formulas in 64 bits of the operators of a fine-tuning step, with bounds on how far the kernels may be off.

A bound counts the roundings that the calls document: the output's (half a step: 2^-8 of the value in bf16, 2^-24 in
fp32), the two-term rank-wide intermediates' (2^-16 of each element), and n 2^-24 sum |a||b| for an fp32 sum of n
products; errors of an intermediate go through the products that follow."""
import math

import torch

F64 = torch.float64
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TERMS = 2.0 ** -16
U = 2.0 ** -24
# exp2, reciprocal and the error function's formula (1.5e-7), each against values near one, with room for their products
ACT = 2.0 ** -20


def d(t):
    return None if t is None else t.detach().cpu().to(F64)


def keep_mask(T, K, p, seed, offset):
    """[T, K] of 0 and 1: Philox-4x32-7 in Python integers' arithmetic (int64 with the products taken in halves)."""
    n = torch.arange(T * (K // 8), dtype=torch.int64)
    m = 0xFFFFFFFF

    def mul(a, w):
        lo, hi = (a & 0xFFFF) * w, (a >> 16) * w  # (both below 2^48)
        s = (hi & 0xFFFF) * 65536 + (lo & m)
        return ((hi >> 16) + (lo >> 32) + (s >> 32)) & m, s & m

    c = [n & m, n >> 32, torch.full_like(n, offset & m), torch.full_like(n, (offset >> 32) & m)]
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(7):
        h0, l0 = mul(c[0], 0xD2511F53)
        h1, l1 = mul(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    w = torch.stack(c, 1)
    bits = torch.stack((w & 0xFFFF, w >> 16), 2).reshape(T, K)
    return (bits >= round(65536 * p)).to(F64)


def kept_share(p):
    return 1.0 - round(65536 * p) / 65536


def within(got, want, bound, what):
    got, bound = d(got), bound.clamp_min(1e-38)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    off = (got - want).abs() / bound
    worst = float(off.max()) if off.numel() else 0.0
    print(f"{what}: at most {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.3f} times the bound at {tuple(torch.unravel_index(off.argmax(), off.shape))}"


def rank_pair(x, A, s):
    """t = s x A^T and the bound of its two terms."""
    t = s * (x @ A.T)
    return t, TERMS * t.abs() + (x.shape[1] + 2) * U * abs(s) * (x.abs() @ A.abs().T)


def linear(x, W, b, pairs):
    """x W^T + b + sum t B^T with pairs (t, its bound, B): the value before its rounding, and its bound."""
    y, e = x @ W.T, (x.shape[1] + sum(2 * p[2].shape[1] for p in pairs) + 2) * U * (x.abs() @ W.abs().T)
    for t, te, B in pairs:
        y, e = y + t @ B.T, e + te @ B.abs().T + (x.shape[1] + 4) * U * (t.abs() @ B.abs().T)
    if b is not None:
        y, e = y + b, e + U * b.abs() * 2
    return y, e


def rounded(v, e, dtype):
    """The bound of a value known to e when it is rounded to dtype."""
    return HALF[dtype] * (v.abs() + e) + e


def dropout(x, W, b, A, B, alpha, p, seed, offset, strength=1.0, request=1.0, dy=None):
    """{name: (value, bound before the output's rounding)}."""
    x, W, b, A, B, dy = (d(v) for v in (x, W, b, A, B, dy))
    R = A.shape[0]
    keep = keep_mask(*x.shape, p, seed, offset)
    s = alpha / R * strength * request / kept_share(p)
    xd = x * keep
    t, te = rank_pair(xd, A, s)
    out = {"y": linear(x, W, b, [(t, te, B)])}
    if dy is not None:
        u, ue = rank_pair(dy, B.T, s)
        base, be = linear(dy, W.T, None, [])
        ext, ee = linear(dy, torch.zeros_like(W.T), None, [(u, ue, A.T)])
        out["dx"] = (base + keep * ext, be + keep * ee + 2 * R * U * base.abs())
        T = x.shape[0]
        out["dA"] = (u.T @ xd, ue.T @ xd.abs() + 2 * (T + 70) * U * (u.abs().T @ xd.abs()))
        out["dB"] = (dy.T @ t, dy.abs().T @ te + 2 * (T + 70) * U * (dy.abs().T @ t.abs()))
    return out


def act(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def gated(x, Wg, Wu, gate, up, bg, bu, name, strength=1.0, request=1.0, dh=None):
    """As dropout(); act' and act'' are at most 1.2 in magnitude each (silu and both gelus), act(v) at most |v|."""
    x, Wg, Wu, bg, bu, dh = (d(v) for v in (x, Wg, Wu, bg, bu, dh))
    T, F = x.shape[0], Wg.shape[0]
    ad = []
    for a in (gate, up):
        if a is None or a["alpha"] * strength * request == 0:
            ad.append(None)
            continue
        A, B = d(a["A"]), d(a["B"])
        s = a["alpha"] / A.shape[0] * strength * request
        ad.append((A, B, s) + rank_pair(x, A, s))
    pairs = [[] if a is None else [(a[3], a[4], a[1])] for a in ad]
    g, ge = linear(x, Wg, bg, pairs[0])
    u, ue = linear(x, Wu, bu, pairs[1])
    a, da = act(g, name)
    ae = 1.2 * ge + ACT * (a.abs() + 1e-3 * g.abs())  # (the function's own error: relative, and absolute in the tails)
    de = 1.2 * ge + ACT * (1 + g.abs())
    out = {"h": (a * u, ae * u.abs() + (a.abs() + ae) * ue + 2 * U * (a * u).abs())}
    if dh is None:
        return out
    dg, du = dh * u * da, dh * a
    dge = dh.abs() * ((da.abs() + de) * ue + u.abs() * de) + 4 * U * dg.abs()
    due = dh.abs() * ae + 2 * U * du.abs()
    dge, due = rounded(dg, dge, torch.bfloat16), rounded(du, due, torch.bfloat16)  # (they are rounded for what follows)
    dx, dxe = dg @ Wg + du @ Wu, dge @ Wg.abs() + due @ Wu.abs()
    dxe = dxe + (2 * F + 600) * U * (dg.abs() @ Wg.abs() + du.abs() @ Wu.abs())
    for n, a, dd, dde in (("gate", ad[0], dg, dge), ("up", ad[1], du, due)):
        if a is None:
            continue
        A, B, s, t, te = a
        v, ve = rank_pair(dd, B.T, s)
        ve = ve + abs(s) * (dde @ B.abs())
        dx, dxe = dx + v @ A, dxe + ve @ A.abs() + (2 * F + 600) * U * (v.abs() @ A.abs())
        out["dA_" + n] = (v.T @ x, ve.T @ x.abs() + 2 * (T + 70) * U * (v.abs().T @ x.abs()))
        out["dB_" + n] = (dd.T @ t, dde.T @ t.abs() + dd.abs().T @ te + 2 * (T + 70) * U * (dd.abs().T @ t.abs()))
    out["dx"] = (dx, dxe)
    return out


def check(got, want, dtype, what):
    v, e = want
    within(got, v, rounded(v, e, dtype), what)

"""Plain 64-bit forms of the routed linear layer, its gradients and the AdamW step, for the tests, with
bounds on how far a correct kernel may be from them.

The bounds count roundings: a value rounded to bf16 is off by at most 2^-8 of it, to fp32 by 2^-24, and a
sum of n fp32 products by at most (n + 1) 2^-24 of the sum of their magnitudes."""
import numpy as np
import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24


def case(T, K, N, n, R, seed, layout="mixed", bias=True, ranks=False, tscale=True, none=0.2):
    """bf16 tensors of one routed layer on the CPU."""
    rng = np.random.default_rng(seed)

    def bf(shape, std):
        return torch.from_numpy(rng.standard_normal(shape) * std).to(torch.float32).to(torch.bfloat16)

    d = dict(x=bf((T, K), 1.0), W=bf((N, K), K ** -0.5), b=bf((N,), 0.2) if bias else None,
             A=bf((n, R, K), K ** -0.5), B=bf((n, N, R), 0.15), dy=bf((T, N), 1.0),
             scales=torch.from_numpy(rng.uniform(0.5, 2.0, n)).float(), ranks=None, token_scale=None)
    if layout == "mixed":
        ids = rng.integers(0, max(n, 1), T)
        ids[rng.random(T) < none] = -1
    else:  # requests of up to 90 tokens ("packed") or of several blocks of 128 ("long")
        most = 90 if layout == "packed" else 900
        ids = np.repeat(rng.integers(-1, max(n, 1), T), rng.integers(1, most, T))[:T]
    d["ids"] = torch.from_numpy(ids if n else np.full(T, -1)).to(torch.int32)
    if ranks:
        d["ranks"] = torch.from_numpy(rng.integers(1, R // 8 + 1, n) * 8).to(torch.int32)
        live = torch.arange(R)[None, :] < d["ranks"][:, None]
        d["A"] = d["A"] * live[:, :, None]
        d["B"] = d["B"] * live[:, None, :]
    if tscale:
        d["token_scale"] = torch.from_numpy(rng.uniform(0.25, 1.5, T)).float()
    return d


def _per_adapter(d):
    """(adapter, its tokens, their fp32 scales as float64) of every adapter in use."""
    ids = d["ids"].long()
    n = d["A"].shape[0]
    for a in sorted(set(ids.tolist())):
        if not 0 <= a < n:
            continue
        rows = (ids == a).nonzero().view(-1)
        s = d["scales"][a].expand(rows.numel())
        if d["token_scale"] is not None:
            s = s * d["token_scale"][rows]
        keep = s != 0
        if d["ranks"] is not None and d["ranks"][a] <= 0:
            keep &= False
        if keep.any():
            yield a, rows[keep], s[keep].double()[:, None]


def _slot(d, a):
    """The adapter's A and B in 64 bits, cut to its rank."""
    r = d["A"].shape[1] if d["ranks"] is None else min(int(d["ranks"][a]), d["A"].shape[1])
    return d["A"][a, :r].double(), d["B"][a, :, :r].double()


def forward(d):
    """(y, bound): the layer in 64 bits and how far each element of a correct bf16 result may be off."""
    x, W = d["x"].double(), d["W"].double()
    K = x.shape[1]
    y, mag = x @ W.T, x.abs() @ W.abs().T
    terms = torch.full((x.shape[0], 1), float(K), dtype=torch.float64)
    tb = torch.zeros_like(y)  # what the rounding of t~ and its own sum let through
    for a, rows, s in _per_adapter(d):
        A, B = _slot(d, a)
        t = (x[rows] @ A.T) * s
        tmag = (x[rows].abs() @ A.abs().T) * s.abs()
        y[rows] += t @ B.T
        mag[rows] += t.abs() @ B.abs().T
        terms[rows] += A.shape[0]
        tb[rows] += (t.abs() * U16 + tmag * (K + 3) * U32 * (1 + U16)) @ B.abs().T
    if d["b"] is not None:
        y += d["b"].double()
        mag += d["b"].double().abs()
    off = tb + (terms + 2) * U32 * (mag + tb)
    return y, off + U16 * (y.abs() + off)


def backward(d):
    """(dx, dA, dB) in 64 bits and their bounds."""
    x, dy, W = d["x"].double(), d["dy"].double(), d["W"].double()
    N, K = W.shape
    n, R, _ = d["A"].shape
    dx, mag = dy @ W, dy.abs() @ W.abs()
    terms = torch.full((x.shape[0], 1), float(N), dtype=torch.float64)
    ub = torch.zeros_like(dx)
    dA, bA = torch.zeros(n, R, K, dtype=torch.float64), torch.zeros(n, R, K, dtype=torch.float64)
    dB, bB = torch.zeros(n, N, R, dtype=torch.float64), torch.zeros(n, N, R, dtype=torch.float64)
    for a, rows, s in _per_adapter(d):
        A, B = _slot(d, a)
        r, c = A.shape[0], rows.numel()
        xa, dya = x[rows], dy[rows]
        u, t = (dya @ B) * s, (xa @ A.T) * s
        umag, tmag = (dya.abs() @ B.abs()) * s.abs(), (xa.abs() @ A.abs().T) * s.abs()
        dx[rows] += u @ A
        mag[rows] += u.abs() @ A.abs()
        terms[rows] += r
        ub[rows] += (u.abs() * U16 + umag * (N + 3) * U32 * (1 + U16)) @ A.abs()
        # hi + mid + lo: each rounded to bf16, and at most 2^-8 of the one before
        eu = u.abs() * U16 ** 3 + umag * (N + 3) * U32
        et = t.abs() * U16 ** 3 + tmag * (K + 3) * U32
        dA[a, :r] = u.T @ xa
        dB[a, :, :r] = dya.T @ t
        # 3 c products (hi, mid and lo apart) and the joins of the chunks, at most c of them
        bA[a, :r] = eu.T @ xa.abs() + (4 * c + 2) * U32 * ((u.abs() * (1 + 2 * U16) + eu).T @ xa.abs())
        bB[a, :, :r] = dya.abs().T @ et + (4 * c + 2) * U32 * (dya.abs().T @ (t.abs() * (1 + 2 * U16) + et))
    off = ub + (terms + 2) * U32 * (mag + ub)
    return (dx, dA, dB), (off + U16 * (dx.abs() + off), bA, bB)


def check(got, want, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bad = ~((g - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}: {g[bad][0].item()!r} for {want[bad][0].item()!r} "
                           f"(bound {bound.expand_as(want)[bad][0].item():.3e})")

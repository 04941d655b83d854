"""Cases and plain forms of the operators for many adapters beside one shared projection.

Three operators, used together where many low-rank adapters share a frozen base weight:

* ``fwd``   the linear layer whose tokens each name their adapter (serving: prompts and single
            tokens of many requests in one batch):
            y[t] = x[t] W^T + b + s_t (x[t] A_a^T) B_a^T,  a = token_adapter[t], s_t = scales[a] token_scale[t]
* ``bwd``   its gradients for an output gradient dy, the base frozen:
            u_t = s_t dy[t] B_a,  dx = dy W + u A_a,  dA_a = sum_t u_t^T x_t,  dB_a = sum_t dy_t^T (s_t x_t A_a^T)
* ``adamw`` one AdamW step over all adapters' tensors at once, the moments in 32 bits or as 8-bit
            floats (e4m3) with one fp32 scale per 256 elements

A token without an adapter (token_adapter -1) gets the base output. Layer sizes are this repository's own
workloads' (1536 / 8960 and 4096 / 14336 wide layers, ranks 16 to 64) or generic.
"""
import math

import torch

own = False
DEV = "cuda:0"
BLOCK = 256          # elements per scale of an 8-bit state
E4M3_MAX = 448.0
TINY = 2.0 ** -100   # a block of moments all below this holds zeros


def listed():
    return [
        # one request, one new token, on an attention projection: the smallest call, latency counts
        dict(name="fwd one token", op="fwd", T=1, K=1536, N=1536, n=4, R=16, layout="mixed", bias=True,
             ranks=False, tscale=False),
        # a decode batch: 64 requests, each with an adapter of its own, on the widest layer
        dict(name="fwd decode 64", op="fwd", T=64, K=4096, N=14336, n=64, R=16, layout="mixed", bias=False,
             ranks=False, tscale=False),
        # a larger decode batch of odd size; ranks 8 to 32 in slots of 32, a scale per request
        dict(name="fwd decode 203", op="fwd", T=203, K=1536, N=8960, n=32, R=32, layout="mixed", bias=True,
             ranks=True, tscale=True),
        # ragged prompts of 16 adapters packed one behind the other, on the FFN down layer
        dict(name="fwd prompts 4977", op="fwd", T=4977, K=8960, N=1536, n=16, R=64, layout="packed", bias=True,
             ranks=False, tscale=True),
        # the largest: the repository's 32760-token FFN up layer, its tokens shared by 8 adapters
        dict(name="fwd prompts 32760", op="fwd", T=32760, K=1536, N=8960, n=8, R=64, layout="packed", bias=False,
             ranks=False, tscale=False),
        # training: a small batch of four adapters on an attention projection
        dict(name="bwd 333", op="bwd", T=333, K=1536, N=1536, n=4, R=16, layout="packed", ranks=False, tscale=False),
        # training: eight adapters of ranks 8 to 32 on the FFN up layer
        dict(name="bwd 4352", op="bwd", T=4352, K=1536, N=8960, n=8, R=32, layout="packed", ranks=True, tscale=False),
        # training, the largest: 16 adapters of rank 64 on the FFN down layer, ragged
        dict(name="bwd 18871", op="bwd", T=18871, K=8960, N=1536, n=16, R=64, layout="packed", ranks=False,
             tscale=True),
        # the step over one layer's two tensors: latency counts
        dict(name="adamw32 one layer", op="adamw", layers=1, R=16, bits=32, grad="f32", master=False),
        # the step over a whole model's adapters (30 blocks of 6 projections): fp32 masters, bf16 copies
        dict(name="adamw32 model", op="adamw", layers=30, R=32, bits=32, grad="f32", master=True),
        # the same with 8-bit moments, small and whole
        dict(name="adamw8 one block", op="adamw", layers=2, R=8, bits=8, grad="bf16", master=False),
        dict(name="adamw8 model", op="adamw", layers=30, R=64, bits=8, grad="f32", master=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "adamw"])
    if op == "adamw":
        return dict(op="adamw", layers=rng.randint(1, 30), R=8 * rng.randint(1, 8), bits=rng.choice([8, 32]),
                    grad=rng.choice(["f32", "bf16"]), master=rng.random() < 0.5)
    K = 8 * _spread(rng, 16, 1120)
    N = _spread(rng, 100, 9000) if op == "fwd" else 8 * _spread(rng, 16, 1120)
    top = min(16000, int(1.4e11 / (K * N)) if op == "fwd" else int(1.2e11 / (K * N)))
    T = min(_spread(rng, 1, 16000), max(1, top))
    c = dict(op=op, T=T, K=K, N=N, n=_spread(rng, 1, 48), R=8 * rng.randint(1, 8),
             layout="mixed" if T <= 300 and rng.random() < 0.5 else "packed",
             ranks=rng.random() < 0.4, tscale=rng.random() < 0.5)
    if op == "fwd":
        c["bias"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------------------- inputs

def _routing(c, g):
    """Which adapter each token takes, -1 for none: "mixed" draws one per token (a decode batch), "packed"
    draws ragged requests that lie one behind the other."""
    T, n = c["T"], c["n"]
    if c["layout"] == "mixed":
        ids = torch.randint(0, n, (T,), generator=g, device=DEV, dtype=torch.int32)
        if T >= n:
            ids[:n] = torch.randperm(n, generator=g, device=DEV, dtype=torch.int32)  # every adapter is in use
        none = torch.rand((T,), generator=g, device=DEV) < (1 / 16 if T > 8 else 0.0)
        return torch.where(none, -1, ids).to(torch.int32)
    req = max(1, min(2 * n, T // 16))
    cuts = torch.randint(0, T + 1, (req - 1,), generator=g, device=DEV).sort().values
    seg = torch.searchsorted(cuts, torch.arange(T, device=DEV), right=True)
    which = torch.randperm(2 * n, generator=g, device=DEV)[:req] % n
    which = torch.where(torch.rand((req,), generator=g, device=DEV) < 1 / 16, -1, which)
    return which[seg].to(torch.int32)


def _shapes(c):
    """The adapter tensors of the case, A then B of each projection: four attention projections and the two
    FFN layers of each block (one attention projection alone for a single layer)."""
    R = c["R"]
    if c["layers"] == 1:
        return [(R, 1536), (1536, R)]
    block = [(R, 1536), (1536, R)] * 4 + [(R, 1536), (8960, R), (R, 8960), (1536, R)]
    return block * c["layers"]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(shape, std, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)

    if c["op"] == "adamw":
        return _prepare_adamw(c, g, normal)
    T, K, N, n, R = c["T"], c["K"], c["N"], c["n"], c["R"]
    st = dict(op=c["op"], x=normal((T, K), 1.0), W=normal((N, K), K ** -0.5), A=normal((n, R, K), K ** -0.5),
              B=normal((n, N, R), 0.02 ** 0.5), b=None, ranks=None, token_scale=None)
    st["scales"] = torch.rand((n,), generator=g, device=DEV) * 1.5 + 0.5
    st["token_adapter"] = _routing(c, g)
    if c["ranks"]:  # ranks that are multiples of 8; a slot is zero behind its adapter's rank
        st["ranks"] = (torch.randint(0, R // 8, (n,), generator=g, device=DEV, dtype=torch.int32) + 1) * 8
        live = torch.arange(R, device=DEV)[None, :] < st["ranks"][:, None]
        st["A"] *= live[:, :, None]
        st["B"] *= live[:, None, :]
    if c["tscale"]:
        st["token_scale"] = torch.rand((T,), generator=g, device=DEV) + 0.25
    if c["op"] == "fwd":
        if c["bias"]:
            st["b"] = normal((N,), 0.02 ** 0.5)
    else:
        st["dy"] = normal((T, N), 1.0)
    if own:
        import rank_gemm_lora_amd as rg
        if c["op"] == "fwd":
            need = rg.lora_linear_routed_workspace_size(T, K, N, n, R)
        else:
            need = rg.lora_linear_routed_bwd_workspace_size(T, K, N, n, R)
        st["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    return st


def _prepare_adamw(c, g, normal):
    # the program keeps its tensors in arenas (each tensor starts a new block of 256): parameters, masters,
    # gradients and moments; the tensors themselves are views
    shapes = _shapes(c)
    sizes = [a * b for a, b in shapes]
    starts, total = [], 0
    for k in sizes:
        starts.append(total)
        total += -(-k // BLOCK) * BLOCK
    live = torch.ones(total, device=DEV)
    for s, k in zip(starts, sizes):
        live[s + k:s + -(-k // BLOCK) * BLOCK] = 0  # (behind a tensor's end the arenas hold zeros)
    master = normal((total,), 0.05, torch.float32) * live
    # gradients and moments spread over several orders of magnitude, as between early and late layers
    size = torch.exp(torch.randn((total // BLOCK, 1), generator=g, device=DEV) * 1.5 - 7).expand(-1, BLOCK).reshape(-1)
    grad = normal((total,), 1.0, torch.float32) * size * live
    m = normal((total,), 0.3, torch.float32) * size * live
    v = (normal((total,), 1.0, torch.float32) * size).square() * live * 0.7 + 0.3 * size.square() * live
    st = dict(op="adamw", bits=c["bits"], step=100, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01,
              master=master if c["master"] else None, param=master.to(torch.bfloat16),
              grad=grad.to(torch.bfloat16) if c["grad"] == "bf16" else grad)
    if c["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        st["m"], st["m_scale"] = _pack(m, False)
        st["v"], st["v_scale"] = _pack(v.sqrt(), True)
    if own:
        import rank_gemm_lora_amd as rg

        def views(t):
            return None if t is None else [t[s:s + k] for s, k in zip(starts, sizes)]

        def block_views(t):
            return None if t is None else [t[s // BLOCK:s // BLOCK + -(-k // BLOCK)] for s, k in zip(starts, sizes)]

        # the optimizer over the tensors and the buffers that the backward calls leave their gradients in
        st["opt"] = rg.LoraAdamW(views(st["param"]), views(st["grad"]), master=views(st["master"]),
                                 state_bits=c["bits"], lr=st["lr"], betas=(st["beta1"], st["beta2"]), eps=st["eps"],
                                 weight_decay=st["wd"],
                                 state=dict(m=views(st["m"]), v=views(st["v"]), m_scale=block_views(st.get("m_scale")),
                                            v_scale=block_views(st.get("v_scale")), step=st["step"]))
    return st


# ----------------------------------------------------------------------------- the plain forms

def _pack(t, positive):
    """[n] fp32 -> (e4m3 [n], fp32 scale per 256): the scale is the block's largest magnitude / 448, a value
    becomes the e4m3 nearest to value * (448 / largest), ties to even. positive: a value above zero is kept
    above zero (at least the smallest e4m3), so that no root of a second moment is rounded down to none."""
    b = t.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    some = top >= TINY
    scale = torch.where(some, top / E4M3_MAX, 0.0)
    y = torch.where(some, b * (E4M3_MAX / torch.where(some, top, 1.0)), 0.0)
    q = y.to(torch.float8_e4m3fn)
    if positive:
        q = torch.where((q.view(torch.uint8) == 0) & (y > 0), 1, q.view(torch.uint8)).to(torch.uint8)
        q = q.view(torch.float8_e4m3fn)
    return q.view(-1), scale.view(-1)


def _unpack(q, scale):
    return (q.to(torch.float32).view(-1, BLOCK) * scale[:, None]).view(-1)


def _weights_of_tokens(st, dtype=torch.float32):
    """[T, n]: the scale of token t for adapter a, zero unless the token takes it."""
    ids, scales = st["token_adapter"].long(), st["scales"]
    one = ids[:, None] == torch.arange(scales.numel(), device=ids.device)
    s = scales[None, :] if st["token_scale"] is None else scales[None, :] * st["token_scale"][:, None]
    return torch.where(one, s, torch.zeros((), device=ids.device))


def _plain_fwd(st):
    x = st["x"].float()
    n, R, K = st["A"].shape
    T, N = x.shape[0], st["W"].shape[0]
    y = x @ st["W"].float().T
    t = (x @ st["A"].float().view(n * R, K).T).view(T, n, R) * _weights_of_tokens(st)[:, :, None]
    y += t.view(T, n * R) @ st["B"].float().transpose(1, 2).reshape(n * R, N)
    if st["b"] is not None:
        y += st["b"].float()
    return y.to(torch.bfloat16)


def _plain_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    n, R, K = st["A"].shape
    T, N = dy.shape
    w = _weights_of_tokens(st)[:, :, None]
    A = st["A"].float().view(n * R, K)
    B = st["B"].float().transpose(1, 2).reshape(n * R, N)
    u = ((dy @ B.T).view(T, n, R) * w).view(T, n * R)
    t = ((x @ A.T).view(T, n, R) * w).view(T, n * R)
    dx = dy @ st["W"].float() + u @ A
    dA = (u.T @ x).view(n, R, K)
    dB = (t.T @ dy).view(n, R, N).transpose(1, 2).contiguous()
    return dx.to(torch.bfloat16), dA, dB


def _plain_adamw(st):
    g = st["grad"].float()
    b1, b2, k = st["beta1"], st["beta2"], st["step"]
    eight = st["bits"] == 8
    f = lambda v: torch.tensor(v, dtype=torch.float64).float().item()  # noqa: E731  (each constant rounded to fp32 once)
    if eight:
        m, r = _unpack(st["m"], st["m_scale"]), _unpack(st["v"], st["v_scale"])
        v = r * r
    else:
        m, v = st["m"], st["v"]
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    r = v.sqrt()
    p = st["param"].float() if st["master"] is None else st["master"]
    p = p * f(1 - st["lr"] * st["wd"]) - (m / (r * f(1 / math.sqrt(1 - b2 ** k)) + f(st["eps"]))) * f(st["lr"] / (1 - b1 ** k))
    if st["master"] is not None:
        st["master"] = p
    st["param"] = p.to(torch.bfloat16)
    if eight:
        st["m"], st["m_scale"] = _pack(m, False)
        st["v"], st["v_scale"] = _pack(r, True)
    else:
        st["m"], st["v"] = m, v


def _adamw_outputs(st):
    return {k: st[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if st.get(k) is not None}


def run(state):
    st = state
    if st["op"] == "adamw":
        st["step"] += 1
        if own:
            st["opt"].step()
        else:
            _plain_adamw(st)
        return _adamw_outputs(st)
    if not own:
        return {"y": _plain_fwd(st)} if st["op"] == "fwd" else dict(zip(("dx", "dA", "dB"), _plain_bwd(st)))
    import rank_gemm_lora_amd as rg
    if st["op"] == "fwd":
        return {"y": rg.lora_linear_routed(st["x"], st["W"], st["b"], st["A"], st["B"], st["scales"],
                                           st["token_adapter"], token_scale=st["token_scale"], ranks=st["ranks"],
                                           workspace=st["ws"])}
    dx, dA, dB = rg.lora_linear_routed_backward(st["x"], st["W"], st["A"], st["B"], st["dy"], st["scales"],
                                                st["token_adapter"], token_scale=st["token_scale"],
                                                ranks=st["ranks"], workspace=st["ws"])
    return {"dx": dx, "dA": dA, "dB": dB}


def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(a * b for a, b in _shapes(c))
        grad = 4 if c["grad"] == "f32" else 2
        moments = 16 if c["bits"] == 32 else 4 + 16 / BLOCK            # both, read and written
        param = 4 + 4 + 2 if c["master"] else 2 + 2                    # (with a master the bf16 copy is only written)
        return {"bytes": n * (grad + moments + param), "flops": 14 * n}
    T, K, N, R = c["T"], c["K"], c["N"], c["R"]
    used = min(c["n"], T)
    adapters = used * R * (K + N) * 2
    side = 4 * T + (4 * T if c["tscale"] else 0) + 4 * c["n"]
    if c["op"] == "fwd":
        return {"bytes": 2 * (T * K + N * K + T * N) + adapters + side + (2 * N if c["bias"] else 0),
                "flops": 2 * T * (K * N + R * (K + N))}
    return {"bytes": 2 * (2 * T * K + N * K + T * N) + adapters + 4 * c["n"] * R * (K + N) + side,
            "flops": 2 * T * (K * N + 3 * R * K + 2 * R * N)}


# ----------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "adamw":
        return _exact_adamw(st)
    ids, d = st["token_adapter"], torch.float64
    x, W = st["x"].to(d), st["W"].to(d)
    s = torch.ones(ids.numel(), dtype=d, device=DEV) if st["token_scale"] is None else st["token_scale"].to(d)
    if st["op"] == "fwd":
        y = x @ W.T
        if st["b"] is not None:
            y = y + st["b"].to(d)
    else:
        dy = st["dy"].to(d)
        dx = dy @ W
        dA = torch.zeros(st["A"].shape, dtype=d, device=DEV)
        dB = torch.zeros(st["B"].shape, dtype=d, device=DEV)
    for a in range(st["A"].shape[0]):
        rows = (ids == a).nonzero().view(-1)
        if rows.numel() == 0:
            continue
        A, B = st["A"][a].to(d), st["B"][a].to(d)
        scale = (s[rows] * st["scales"][a].to(d))[:, None]
        t = (x[rows] @ A.T) * scale
        if st["op"] == "fwd":
            y[rows] += t @ B.T
        else:
            u = (dy[rows] @ B) * scale
            dx[rows] += u @ A
            dA[a] = u.T @ x[rows]
            dB[a] = dy[rows].T @ t
    return {"y": y} if st["op"] == "fwd" else {"dx": dx, "dA": dA, "dB": dB}


def _exact_adamw(st):
    d = torch.float64
    k = st["step"] + 1
    b1, b2 = st["beta1"], st["beta2"]
    eight = st["bits"] == 8
    g, m, v = st["grad"].to(d), st["m"].to(d), st["v"].to(d)
    if eight:
        m = m * st["m_scale"].to(d).repeat_interleave(BLOCK)
        v = (v * st["v_scale"].to(d).repeat_interleave(BLOCK)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = (st["param"] if st["master"] is None else st["master"]).to(d)
    p = p - st["lr"] * st["wd"] * p - st["lr"] * (m / (1 - b1 ** k)) / ((v / (1 - b2 ** k)).sqrt() + st["eps"])
    out = {"param": p}
    if st["master"] is not None:
        out["master"] = p
    if not eight:
        return dict(out, m=m, v=v)
    for name, t in (("m", m), ("v", v.sqrt())):
        top = t.view(-1, BLOCK).abs().amax(1)
        y = torch.where(top[:, None] > 0, t.view(-1, BLOCK) / top[:, None] * E4M3_MAX, 0.0).view(-1)
        # e4m3: 3 bits behind the leading one, exponents from -6 on (below it steps of 2^-9)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        q = torch.round(y / step) * step
        if name == "v":
            q = torch.where((q == 0) & (y > 0), 2.0 ** -9, q)
        out[name], out[name + "_scale"] = q, top / E4M3_MAX
    return out

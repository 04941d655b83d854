"""Cases and plain forms of what a step of fine-tuning low-rank adapters takes beside the plain linear layer.

Three operators, run one after the other in such a step (the base weights are frozen throughout):

* ``gated``    the gated half of a feed-forward block whose two projections carry adapters:
               g = x Wg^T + bg + sg (x Ag^T) Bg^T,  u = x Wu^T + bu + su (x Au^T) Bu^T,  h = act(g) u
               Serving calls it forward only, from one token on; a training step runs it forward and then
               backward for a gradient dh: dx, dAg, dBg, dAu, dBu
* ``dropout``  a linear layer with dropout in front of its adapter, forward and backward:
               y = x W^T + b + s (D(x) A^T) B^T,  D(x) = x . keep / (1 - p)
               keep is a function of (seed, offset, element): it is formed anew wherever it is needed. Element
               (t, k) takes 16 of the 128 bits that Philox-4x32 with 7 rounds gives for the counter t K/8 + k/8
               and is kept where they are at least round(65536 p)
* ``loss``     softmax cross entropy over a vocabulary straight from the hidden states and the (frozen) output
               weight, l = h W^T: loss = logsumexp(l) - l[target], and dh for a weight per token. A token whose
               target lies outside the vocabulary has no loss

Layer sizes are this repository's own workloads' (1536 / 8960 and 4096 / 14336 wide layers) or generic.
"""
import math

import torch

own = False
DEV = "cuda:0"
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16


def listed():
    return [
        # one request, one new token through the smaller block: the smallest call, latency counts
        dict(name="gated one token", op="gated", T=1, K=1536, F=8960, rg=16, ru=16, act="silu", bias=False, step=False),
        # a decode batch of odd size through the larger block
        dict(name="gated decode 48", op="gated", T=48, K=4096, F=14336, rg=16, ru=16, act="silu", bias=False, step=False),
        # prompts through the smaller block, its adapters of rank 64, gelu and biases
        dict(name="gated prompts 4977", op="gated", T=4977, K=1536, F=8960, rg=64, ru=64, act="gelu_tanh", bias=True,
             step=False),
        # prompts through the larger block
        dict(name="gated prompts 12288", op="gated", T=12288, K=4096, F=14336, rg=32, ru=32, act="silu", bias=False,
             step=False),
        # training, a small ragged batch: forward, then backward
        dict(name="gated step 333", op="gated", T=333, K=1536, F=8960, rg=16, ru=8, act="gelu", bias=True, step=True),
        # training, a full batch on the larger block
        dict(name="gated step 4352", op="gated", T=4352, K=4096, F=14336, rg=32, ru=32, act="silu", bias=False, step=True),
        # training an attention projection with dropout, a small ragged batch
        dict(name="dropout step 333", op="dropout", T=333, K=1536, N=1536, R=16, p=0.05, bias=True),
        # training the widest input, all of a video's tokens
        dict(name="dropout step 18871", op="dropout", T=18871, K=8960, N=1536, R=64, p=0.1, bias=False),
        # a prompt's log-likelihood: the loss alone, an odd vocabulary
        dict(name="loss 777", op="loss", T=777, K=1536, V=32003, grad=False),
        # training, a small ragged batch
        dict(name="loss step 333", op="loss", T=333, K=1536, V=50261, grad=True),
        # training, a full batch over a large vocabulary
        dict(name="loss step 4096", op="loss", T=4096, K=4096, V=128017, grad=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated", "dropout", "dropout", "loss", "loss"])
    if op == "loss":
        K, V = 8 * _spread(rng, 16, 640), _spread(rng, 900, 150000)
        T = min(_spread(rng, 1, 9000), max(1, int(2.0e12 / (K * V))))
        return dict(op=op, T=T, K=K, V=V, grad=rng.random() < 0.7)
    if op == "dropout":
        K, N = 8 * _spread(rng, 16, 1120), 8 * _spread(rng, 16, 1120)
        T = min(_spread(rng, 1, 16000), max(1, int(2.4e11 / (K * N))))
        return dict(op=op, T=T, K=K, N=N, R=8 * rng.randint(1, 8), p=round(rng.uniform(0.01, 0.5), 3),
                    bias=rng.random() < 0.5)
    step = rng.random() < 0.5
    K, F = 8 * _spread(rng, 16, 640), 8 * _spread(rng, 16, 1800)
    T = min(_spread(rng, 1, 12000), max(1, int((2.5e11 if step else 7.0e11) / (K * F))))
    if not step and rng.random() < 0.3:
        T = rng.randint(1, 64)  # a decode batch
    return dict(op=op, T=T, K=K, F=F, rg=8 * rng.randint(1, 8), ru=8 * rng.randint(1, 8),
                act=rng.choice(["silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.4, step=step)


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(shape, std, dtype=BF16):
        return (torch.randn(shape, generator=g, device=DEV, dtype=F32) * std).to(dtype)

    T, K = c["T"], c["K"]
    st = dict(c, x=normal((T, K), 1.0), ws=None)
    if c["op"] == "gated":
        F = c["F"]
        for n, r in (("g", c["rg"]), ("u", c["ru"])):
            st["W" + n], st["A" + n], st["B" + n] = normal((F, K), K ** -0.5), normal((r, K), K ** -0.5), normal((F, r), 0.02 ** 0.5)
            st["b" + n] = normal((F,), 0.02 ** 0.5) if c["bias"] else None
            st["alpha" + n] = 1.0 * r
        if c["step"]:
            st["dh"] = normal((T, F), 1.0)
    elif c["op"] == "dropout":
        N, R = c["N"], c["R"]
        st.update(W=normal((N, K), K ** -0.5), A=normal((R, K), K ** -0.5), B=normal((N, R), 0.02 ** 0.5),
                  b=normal((N,), 0.02 ** 0.5) if c["bias"] else None, dy=normal((T, N), 1.0), alpha=2.0 * R,
                  seed=0x9E3779B97F4A7C15 ^ (int(seed) * 0x2545F4914F6CDD1D & (2 ** 64 - 1)), offset=int(seed) % 1000 + 1)
    else:
        V = c["V"]
        # logits of a few units; most tokens' targets stand out, from hardly to almost surely
        st["W"] = normal((V, K), 2.0 * K ** -0.5)
        target = torch.randint(0, V, (T,), generator=g, device=DEV)
        sure = torch.rand((T, 1), generator=g, device=DEV) * 5.0
        st["x"] = (st["x"].float() + sure * st["W"][target].float()).to(BF16)
        none = torch.rand((T,), generator=g, device=DEV) < (1 / 8 if T > 8 else 0.0)  # (the prompt's part has no loss)
        st["target"] = torch.where(none, -100, target)
        st["dloss"] = torch.full((T,), 1.0 / max(1, int((~none).sum())), device=DEV)
    if own:
        import rank_gemm_lora_amd as rg
        if c["op"] == "gated" and c["step"]:
            need = rg.lora_gated_bwd_workspace_size(T, K, c["F"], c["rg"], c["ru"])
        elif c["op"] == "gated":
            need = rg.lora_gated_workspace_size(T, K, c["F"], c["rg"], c["ru"])
        elif c["op"] == "dropout":
            need = rg.lora_linear_dropout_bwd_workspace_size(T, K, c["N"], c["R"])
        else:
            need = rg.lora_cross_entropy_workspace_size(T, K, c["V"], c["grad"])
        st["ws"] = torch.empty(max(1, need), dtype=torch.uint8, device=DEV)
    return st


# ----------------------------------------------------------------------------- the plain forms

def _erf(v):
    return torch.special.erf(v)


def _act(g, name):
    """act(g) and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        cdf = 0.5 * (1 + _erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _linear(x, W, b, A, B, s):
    """The layer of one adapter in 32 bits, and the scaled rank-wide product behind it."""
    t = (x @ A.float().T) * s
    y = x @ W.float().T + t @ B.float().T
    return (y if b is None else y + b.float()), t


def _plain_gated(st):
    x = st["x"].float()
    sg, su = st["alphag"] / st["rg"], st["alphau"] / st["ru"]
    g, tg = _linear(x, st["Wg"], st["bg"], st["Ag"], st["Bg"], sg)
    u, tu = _linear(x, st["Wu"], st["bu"], st["Au"], st["Bu"], su)
    a, da = _act(g, st["act"])
    out = {"h": (a * u).to(BF16)}
    if not st["step"]:
        return out
    dh = st["dh"].float()
    dg, du = dh * u * da, dh * a
    vg, vu = (dg @ st["Bg"].float()) * sg, (du @ st["Bu"].float()) * su
    out["dx"] = (dg @ st["Wg"].float() + du @ st["Wu"].float() + vg @ st["Ag"].float() + vu @ st["Au"].float()).to(BF16)
    out["dAg"], out["dBg"] = (vg.T @ x).to(BF16), (dg.T @ tg).to(BF16)
    out["dAu"], out["dBu"] = (vu.T @ x).to(BF16), (du.T @ tu).to(BF16)
    return out


def _words(count, seed, offset):
    """Philox-4x32, 7 rounds: the four 32-bit words for the counters (n, offset), n = 0 .. count - 1, as int64."""
    low = 0xFFFFFFFF
    n = torch.arange(count, device=DEV, dtype=torch.int64)
    a, b = n & low, n >> 32
    c, d = torch.full_like(n, offset & low), torch.full_like(n, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(7):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57  # (the low 64 bits of the product; the shift's sign bits are cut off)
        a, b, c, d = ((q >> 32) & low) ^ b ^ k0, q & low, ((p >> 32) & low) ^ d ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return a, b, c, d


def _keep(st):
    """[T, K]: kept or not."""
    T, K = st["x"].shape
    thr = round(st["p"] * 65536)
    w = torch.stack(_words(T * K // 8, st["seed"], st["offset"]), 1)
    return torch.stack((w & 0xFFFF, w >> 16), 2).reshape(T, K) >= thr


def _scale(st):
    return st["alpha"] / st["R"] / (1 - round(st["p"] * 65536) / 65536)


def _plain_dropout(st):
    x, dy, s = st["x"].float(), st["dy"].float(), _scale(st)
    keep = _keep(st)
    xd = torch.where(keep, x, 0.0)
    t = (xd @ st["A"].float().T) * s
    y = x @ st["W"].float().T + t @ st["B"].float().T
    if st["b"] is not None:
        y = y + st["b"].float()
    u = (dy @ st["B"].float()) * s
    dx = dy @ st["W"].float() + torch.where(keep, u @ st["A"].float(), 0.0)
    return {"y": y.to(BF16), "dx": dx.to(BF16), "dA": (u.T @ xd).to(BF16), "dB": (dy.T @ t).to(BF16)}


def _plain_loss(st):
    logits = st["x"].float() @ st["W"].float().T
    V = logits.shape[1]
    some = (st["target"] >= 0) & (st["target"] < V)
    at = torch.where(some, st["target"], 0)[:, None]
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    out = {"loss": torch.where(some, lse - logits.gather(1, at)[:, 0], 0.0), "lse": lse}
    if st["grad"]:
        # 1 - p[target] is the sum of the other tokens' shares: the difference would lose what a sure token has left
        others = e.scatter(1, at, 0.0)
        share = others / total
        d = share.scatter(1, at, -share.sum(1, keepdim=True)) * torch.where(some, st["dloss"], 0.0)[:, None]
        out["dh"] = (d @ st["W"].float()).to(BF16)
    return out


def run(state):
    st = state
    if not own:
        return {"gated": _plain_gated, "dropout": _plain_dropout, "loss": _plain_loss}[st["op"]](st)
    import rank_gemm_lora_amd as rg
    if st["op"] == "loss":
        loss, lse, dh = rg.lora_cross_entropy(st["x"], st["W"], st["target"], dloss=st["dloss"] if st["grad"] else None,
                                              want=("loss", "lse", "dh") if st["grad"] else ("loss", "lse"),
                                              workspace=st["ws"])
        return {"loss": loss, "lse": lse, "dh": dh} if st["grad"] else {"loss": loss, "lse": lse}
    if st["op"] == "dropout":
        how = dict(alpha=st["alpha"], p=st["p"], seed=st["seed"], offset=st["offset"], workspace=st["ws"])
        y = rg.lora_linear_dropout(st["x"], st["W"], st["b"], st["A"], st["B"], **how)
        dx, dA, dB = rg.lora_linear_dropout_backward(st["x"], st["W"], st["A"], st["B"], st["dy"], grad_dtype=BF16, **how)
        return {"y": y, "dx": dx, "dA": dA, "dB": dB}
    gate = dict(A=st["Ag"], B=st["Bg"], alpha=st["alphag"])
    up = dict(A=st["Au"], B=st["Bu"], alpha=st["alphau"])
    how = dict(b_gate=st["bg"], b_up=st["bu"], act=st["act"], workspace=st["ws"])
    if not st["step"]:
        return {"h": rg.lora_gated(st["x"], st["Wg"], st["Wu"], gate, up, **how)}
    # the forward keeps what its backward reads in place of a second pass over the weights
    h, saved = rg.lora_gated(st["x"], st["Wg"], st["Wu"], gate, up, save=True, **how)
    dx, dAg, dBg, dAu, dBu = rg.lora_gated_backward(st["x"], st["Wg"], st["Wu"], gate, up, st["dh"], saved=saved,
                                                    grad_dtype=BF16, **how)
    return {"h": h, "dx": dx, "dAg": dAg, "dBg": dBg, "dAu": dAu, "dBu": dBu}


def work(case):
    c = case
    T, K = c["T"], c["K"]
    if c["op"] == "loss":
        V = c["V"]
        return {"bytes": 2 * (T * K + V * K) + 16 * T + (2 * T * K + 4 * T if c["grad"] else 0),
                "flops": (4 if c["grad"] else 2) * T * V * K}
    if c["op"] == "dropout":
        N, R = c["N"], c["R"]
        return {"bytes": 2 * (2 * T * K + 2 * T * N + N * K) + 4 * R * (K + N) + (2 * N if c["bias"] else 0),
                "flops": 4 * T * K * N + 2 * T * R * (3 * K + 3 * N)}
    F, r = c["F"], c["rg"] + c["ru"]
    side = 2 * r * (K + F) + (4 * F if c["bias"] else 0)
    fwd = {"bytes": 2 * (T * K + 2 * F * K + T * F) + side, "flops": 2 * T * (2 * F * K + r * (K + F))}
    if not c["step"]:
        return fwd
    return {"bytes": fwd["bytes"] + 2 * (T * F + T * K) + 2 * r * (K + F), "flops": 2 * fwd["flops"] + 2 * T * r * (K + F)}


# ----------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"gated": _exact_gated, "dropout": _exact_dropout, "loss": _exact_loss}[st["op"]](st)


def _exact_gated(st):
    v = {n: None if st[n] is None else st[n].to(F64) for n in ("x", "Wg", "Wu", "bg", "bu", "Ag", "Bg", "Au", "Bu")}
    if st["step"]:
        for n in ("x", "Ag", "Bg", "Au", "Bu"):
            v[n].requires_grad_(True)
    pre = {}
    for n in "gu":
        weight = v["W" + n] + (st["alpha" + n] / st["r" + n]) * (v["B" + n] @ v["A" + n])
        pre[n] = v["x"] @ weight.T if v["b" + n] is None else v["x"] @ weight.T + v["b" + n]
    z = pre["g"]
    if st["act"] == "silu":
        a = z * torch.sigmoid(z)
    elif st["act"] == "gelu":
        a = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    else:
        a = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    h = a * pre["u"]
    out = {"h": h.detach()}
    if st["step"]:
        names = ("x", "Ag", "Bg", "Au", "Bu")
        grads = torch.autograd.grad(h, [v[n] for n in names], st["dh"].to(F64))
        out.update({"d" + n: t for n, t in zip(names, grads)})
    return out


def _exact_dropout(st):
    T, K = st["x"].shape
    half = 0xFFFF

    def product(m, w):  # the high and the low word of a 32 x 32 bit product, from 16-bit halves
        ml, mh, wl, wh = m & half, m >> 16, w & half, w >> 16
        mid = mh * wl + ((ml * wl) >> 16)
        low = ml * wh + (mid & half)
        return mh * wh + (mid >> 16) + (low >> 16), ((low & half) << 16) | ((ml * wl) & half)

    n = torch.arange(T * K // 8, device=DEV)
    ctr = [n % 2 ** 32, n // 2 ** 32, torch.full_like(n, st["offset"] % 2 ** 32), torch.full_like(n, st["offset"] // 2 ** 32)]
    key = [st["seed"] % 2 ** 32, st["seed"] // 2 ** 32]
    for _ in range(7):
        h0, l0 = product(0xD2511F53, ctr[0])
        h1, l1 = product(0xCD9E8D57, ctr[2])
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = torch.empty((T * K // 8, 8), dtype=torch.int64, device=DEV)
    for i in range(4):
        bits[:, 2 * i], bits[:, 2 * i + 1] = ctr[i] % 65536, ctr[i] // 65536
    cut = round(st["p"] * 65536)
    keep = (bits.view(T, K) >= cut).to(F64) * (65536 / (65536 - cut))
    del bits, ctr, n
    s = st["alpha"] / st["R"]
    x, W, A, B, dy = (st[k].to(F64) for k in ("x", "W", "A", "B", "dy"))
    t = s * ((x * keep) @ A.T)
    y = x @ W.T + t @ B.T
    u = s * (dy @ B)
    return {"y": y if st["b"] is None else y + st["b"].to(F64), "dx": dy @ W + (u @ A) * keep, "dA": u.T @ (x * keep),
            "dB": dy.T @ t}


def _exact_loss(st):
    W = st["W"].to(F64)
    V = W.shape[0]
    parts = {"loss": [], "lse": [], "dh": []}
    for t0 in range(0, st["x"].shape[0], 1024):
        logits = st["x"][t0:t0 + 1024].to(F64) @ W.T
        target = st["target"][t0:t0 + 1024]
        some = (target >= 0) & (target < V)
        at = target.clamp(0, V - 1)[:, None]
        lse = torch.logsumexp(logits, 1)
        parts["lse"].append(lse)
        parts["loss"].append(torch.where(some, lse - logits.gather(1, at)[:, 0], 0.0))
        if st["grad"]:
            p = torch.exp(logits - lse[:, None])
            rest = p.scatter(1, at, 0.0).sum(1, keepdim=True)  # (1 - p[target])
            p.scatter_(1, at, -rest)
            parts["dh"].append((p @ W) * (some * st["dloss"][t0:t0 + 1024].to(F64))[:, None])
    return {k: torch.cat(v) for k, v in parts.items() if v}

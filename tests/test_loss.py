"""The vocabulary loss: refusals on the CPU, parity with the formula in 64 bits on the GPU, and the operators of a
fine-tuning step run together against autograd in 64 bits."""
import math

import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import step_ref as sr

OK, NULL, SHAPE, DTYPE, NONFIN, ALIGN, OVERLAP, WS, UNSUP, HIP = range(10)
DEV = "cuda:0"
BF, F64 = torch.bfloat16, torch.float64
BASE = 0x10_0000_0000


def say(*a):
    print(*a, flush=True)


ARGS = dict(h=BASE, T=100, K=256, ldh=256, W=BASE * 2, V=1000, target=BASE * 3, dloss=BASE * 4, loss=BASE * 5, lse=BASE * 6,
            dh=BASE * 7, lddh=256, ws=BASE * 8, wb=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), NULL), (dict(W=None), NULL), (dict(target=None), NULL),
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(V=0), SHAPE), (dict(ldh=255), SHAPE), (dict(lddh=255), SHAPE),
    (dict(T=1 << 21), UNSUP), (dict(V=(1 << 24) + 1), UNSUP), (dict(T=1 << 20, V=1 << 17), UNSUP),
    (dict(T=1 << 20, K=1 << 14, ldh=1 << 14, lddh=1 << 14), UNSUP), (dict(K=1 << 21, ldh=1 << 21, lddh=1 << 21), UNSUP),
    (dict(h=BASE + 8), ALIGN), (dict(W=BASE * 2 + 8), ALIGN), (dict(target=BASE * 3 + 4), ALIGN), (dict(dloss=BASE * 4 + 2), ALIGN),
    (dict(loss=BASE * 5 + 1), ALIGN), (dict(lse=BASE * 6 + 2), ALIGN), (dict(dh=BASE * 7 + 1), ALIGN),
    (dict(ws=BASE * 8 + 8), ALIGN), (dict(K=252, ldh=256), ALIGN), (dict(ldh=260), ALIGN),
    (dict(ws=None), WS), (dict(wb=100), WS),
    (dict(loss=BASE), OVERLAP), (dict(lse=BASE * 5 + 16), OVERLAP), (dict(dh=BASE + 1024), OVERLAP), (dict(dh=BASE * 8), OVERLAP),
    (dict(ws=BASE * 2), OVERLAP), (dict(loss=BASE * 4), OVERLAP),
])
def test_refusals(kw, code):
    a = dict(ARGS, **kw)
    assert rg._lib.lora_cross_entropy(a["h"], a["T"], a["K"], a["ldh"], a["W"], a["V"], a["target"], a["dloss"], a["loss"],
                                      a["lse"], a["dh"], a["lddh"], a["ws"], a["wb"], None) == code


def test_nothing_to_do_and_sizes():
    call = rg._lib.lora_cross_entropy
    assert call(None, 0, 64, 64, BASE, 10, None, None, None, None, None, 0, None, 0, None) == OK
    assert call(BASE, 4, 64, 64, BASE * 2, 10, BASE * 3, None, None, None, None, 0, BASE * 8, 1 << 20, None) == OK
    size = rg.lora_cross_entropy_workspace_size
    assert size(0, 64, 10) == 0 and size(4, 64, 0) == 0 and size(1 << 21, 64, 10) == 0
    for T, V in ((1, 10), (333, 50000), (9000, 200000)):
        assert 0 < size(T, 64, V, False) < size(T, 64, V, True)
    with pytest.raises(TypeError):
        rg.lora_cross_entropy(torch.zeros(2, 64, dtype=BF), torch.zeros(5, 64, dtype=BF), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        rg.lora_cross_entropy(torch.zeros(2, 64, dtype=BF), torch.zeros(5, 64, dtype=BF), torch.zeros(3, dtype=torch.int64))


def case(T, K, V, seed=0, sure=4.0, none=0.1, std=2.0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, K, generator=g) * std * K ** -0.5).to(BF)
    target = torch.randint(0, V, (T,), generator=g)
    h = torch.randn(T, K, generator=g) + torch.rand(T, 1, generator=g) * sure * W[target].float()
    gone = torch.rand(T, generator=g) < none
    target = torch.where(gone, torch.where(torch.rand(T, generator=g) < 0.5, -100, V), target)
    return dict(h=h.to(BF), W=W, target=target, dloss=torch.rand(T, generator=g) + 0.1)


def reference(c, rows=None):
    """{name: (value, bound before the output's rounding)}."""
    rows = slice(None) if rows is None else rows
    h, W, t, w = sr.d(c["h"][rows]), sr.d(c["W"]), c["target"][rows], sr.d(c["dloss"][rows])[:, None]
    V, K = W.shape
    l = h @ W.T
    # logits: an fp32 sum of K products; 2^-22 for the exponential and its argument's rounding
    le = (K + 4) * sr.U * (h.abs() @ W.abs().T)
    some = (t >= 0) & (t < V)
    at = t.clamp(0, V - 1)[:, None]
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    # relative error of an exponential: its argument's, and sums of V positive terms in fp32 in blocks of 128 and more
    far = (l.amax(1, keepdim=True) - l).abs() + l.abs().amax(1, keepdim=True)
    rel = le + 4 * sr.U * (1 + far)
    lsee = (p * rel).sum(1) + (300 + V // 64) * sr.U + 4 * sr.U * lse.abs()
    others = p.scatter(1, at, 0.0)
    rest = torch.where(some[:, None], others.sum(1, keepdim=True), 0.0)
    # (as a difference only where it is not small: its last digits are lost in 64 bits too)
    lt = l.gather(1, at)
    near = torch.log1p(torch.exp((l - lt).clamp_max(700.0)).scatter(1, at, 0.0).sum(1))
    loss = torch.where(some, torch.where(near < 1, near, lse - lt[:, 0]), 0.0)
    # a sure token's loss is log(1 + the others): an error relative to it beside that of the difference
    losse = torch.where(some, lsee + le.gather(1, at)[:, 0] + 4 * sr.U * l.abs().amax(1), 0.0)
    losse = torch.minimum(losse, 8 * rel.amax(1) * rest[:, 0] + losse * (loss > 0.5) + (300 + V // 64) * sr.U * rest[:, 0] + losse * (rest[:, 0] > 0.3))
    # Proof of the absolute part: an exponential below 2^-126, the smallest normal number, is flushed to zero, and so is its
    # product with a block's sum: each of the V terms of `others` loses at most 2^-126, whatever the order of the sums.
    losse = losse + V * 2.0 ** -126
    pe = others * (2.0 ** -8 + rel + lsee[:, None])
    d = others.scatter(1, at, -rest) * some[:, None] * w
    Wt = W[at[:, 0]].abs()
    dhe = (pe @ W.abs() + V * 2.0 ** -126 * (W.abs().amax(0) + Wt) + (V + 64) * sr.U * (others @ W.abs()) + rest * (rel.amax(1) + 2 * lsee + (300 + V // 64) * sr.U)[:, None] * Wt) * some[:, None] * w
    return {"loss": (loss, losse), "lse": (lse, lsee), "dh": (d @ W, dhe + 4 * sr.U * (d @ W).abs())}


def run(c, **kw):
    v = {k: t.to(DEV) for k, t in c.items()}
    return dict(zip(("loss", "lse", "dh"), rg.lora_cross_entropy(v["h"], v["W"], v["target"], dloss=v["dloss"], **kw)))


def check(got, want, what=""):
    for k, v in got.items():
        if v is not None:
            sr.check(v, want[k], BF if k == "dh" else torch.float32, f"{what} {k}")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,V", [
    (1, 64, 1), (1, 1536, 50000), (2, 8, 7), (3, 264, 63), (5, 64, 64), (17, 72, 65), (33, 512, 127), (64, 64, 129), (65, 1032, 1000),
    (128, 136, 4097), (129, 512, 32003), (300, 1536, 5000), (257, 64, 100001), (1000, 256, 256), (2049, 128, 257),
])
def test_against_the_formula(T, K, V):
    say("loss", T, K, V)
    c = case(T, K, V)
    check(run(c), reference(c))


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,V", [(9000, 64, 70001), (5000, 520, 33000)])
def test_pieces_and_large_tiles(T, K, V):
    """More columns than one piece holds, and the larger tiles."""
    say("loss pieces", T, K, V)
    c = case(T, K, V, 1)
    got = run(c)
    rows = torch.cat((torch.arange(0, 60), torch.arange(T - 60, T)))
    check({k: v[rows] for k, v in got.items()}, reference(c, rows))


@pytest.mark.gpu
def test_sure_tokens_and_far_logits():
    """Targets that are all but certain: the gradient's small values keep their leading digits. And logits far beyond
    where their exponentials exist."""
    say("loss sure")
    c = case(200, 128, 3000, 2, sure=0.0, none=0.0)
    W = c["W"].float()
    c["h"] = (torch.linspace(0.5, 60, 200)[:, None] * W[c["target"]]).to(BF)
    got = run(c)
    check(got, reference(c))
    for scale in (30.0, -30.0):
        c = case(100, 64, 5000, 3, sure=0.0, std=1.0)
        c["h"] = (c["h"].float() * scale).to(BF)
        check(run(c), reference(c))
    # logits that rise along the vocabulary, by far more than one exponential's range
    c = case(70, 8, 2000, 4, sure=0.0, none=0.0)
    c["W"][:, 1:] = 0
    c["W"][:, 0] = torch.linspace(-300, 300, 2000).to(BF)
    c["h"][:, 0] = torch.linspace(-2, 2, 70).to(BF)
    check(run(c), reference(c))


@pytest.mark.gpu
def test_wants_strides_and_ignored_tokens():
    say("loss wants")
    c = case(70, 200, 700, 5)
    full = run(c)
    for want in (("loss",), ("lse",), ("dh",), ("loss", "dh")):
        got = run(c, want=want)
        for k, v in got.items():
            assert (v is None) == (k not in want) and (v is None or torch.equal(v, full[k])), (want, k)
    gone = (c["target"] < 0) | (c["target"] >= 700)
    assert bool(gone.any()) and not bool(full["loss"][gone].any()) and not bool(full["dh"][gone].any())
    v = {k: t.to(DEV) for k, t in c.items()}
    h = torch.full((70, 224), float("nan"), dtype=BF, device=DEV)
    h[:, :200] = v["h"]
    wide = torch.full((71, 205), 3.0, dtype=BF, device=DEV)
    loss, lse, dh = rg.lora_cross_entropy(h[:, :200], v["W"], v["target"], dloss=v["dloss"], dh=wide[:70, 3:203])
    assert torch.equal(dh, full["dh"]) and torch.equal(loss, full["loss"])
    assert bool((wide[:, :3] == 3).all()) and bool((wide[:, 203:] == 3).all()) and bool((wide[70] == 3).all())
    ones = rg.lora_cross_entropy(v["h"], v["W"], v["target"])[2]
    check({"dh": ones}, reference(dict(c, dloss=torch.ones(70))))
    none = rg.lora_cross_entropy(v["h"], v["W"], torch.full_like(v["target"], -1))
    assert not bool(none[0].any()) and not bool(none[2].any())
    check({"lse": none[1]}, reference(c))  # (the same sum; a target is added to it last, so its bits may differ)


@pytest.mark.gpu
def test_a_broken_token_stays_alone():
    say("loss broken")
    c = case(100, 64, 1000, 6)
    full = run(c)
    for bad in (math.nan, math.inf):
        h = c["h"].clone()
        h[13] = bad
        got = run(dict(c, h=h, target=torch.where(torch.arange(100) == 13, 5, c["target"])))
        rest = torch.arange(100) != 13
        for k in got:
            assert torch.equal(got[k][rest], full[k][rest]), k
        assert bool(torch.isnan(got["loss"][13])) and bool(torch.isnan(got["lse"][13])) and bool(torch.isnan(got["dh"][13]).all())


@pytest.mark.gpu
def test_gradient_against_differences():
    say("loss differences")
    c = case(20, 32, 300, 7, none=0.0)
    got, want = run(c), reference(c)
    g = torch.Generator().manual_seed(8)
    way = torch.randn(20, 32, generator=g, dtype=F64)
    value = lambda h: float((reference(dict(c, h=h))["loss"][0] * sr.d(c["dloss"])).sum())  # noqa: E731
    h, eps = sr.d(c["h"]), 1e-5
    diff = (value(h + eps * way) - value(h - eps * way)) / (2 * eps)
    v, e = want["dh"]
    assert abs(float((sr.d(got["dh"]) * way).sum()) - diff) <= float((sr.rounded(v, e, BF) * way.abs()).sum()) + 1e-6 * abs(diff)


@pytest.mark.gpu
def test_streams_and_replays():
    say("loss graph")
    c = case(150, 128, 5000, 9)
    v = {k: t.to(DEV) for k, t in c.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = rg.lora_cross_entropy(v["h"], v["W"], v["target"], stream=s)
    s.synchronize()
    here = rg.lora_cross_entropy(v["h"], v["W"], v["target"])
    assert all(torch.equal(a, b) for a, b in zip(side, here))
    ws = torch.empty(rg.lora_cross_entropy_workspace_size(150, 128, 5000), dtype=torch.uint8, device=DEV)
    call = lambda: rg.lora_cross_entropy(v["h"], v["W"], v["target"], dloss=v["dloss"], workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for i in range(4):
        n = case(150, 128, 5000, 20 + i)
        v["h"].copy_(n["h"])
        v["target"].copy_(n["target"])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, call()))
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_step_of_all_of_them_together():
    """Projection with dropout, gated block, down projection, loss, and back: gradients of every adapter against autograd
    in 64 bits, then one AdamW step that reads them. Every bf16 tensor on a path changes what follows by at most 2^-8 of
    it; a gradient passes at most 12 of them (x' and y, h, z, logits' shares, dz, dh, dg or du, dx, its own), and sums
    of independent errors stay below their sum."""
    say("a whole step")
    T, D, F, V, R = 160, 128, 328, 1003, 16
    g = torch.Generator().manual_seed(1)
    mk = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    x, W0, Wg, Wu, W1, Wv = mk(T, D), mk(D, D, std=D ** -0.5), mk(F, D, std=D ** -0.5), mk(F, D, std=D ** -0.5), mk(D, F, std=F ** -0.5), mk(V, D, std=3 * D ** -0.5)
    ad = [(mk(R, i, std=i ** -0.5), mk(o, R, std=0.15)) for i, o in ((D, D), (D, F), (D, F), (F, D))]
    target = torch.randint(0, V, (T,), generator=g)
    alpha, p, seed = float(R), 0.2, 77
    # in 64 bits
    leaves = [t.to(F64).requires_grad_(True) for ab in ad for t in ab]
    q = [t.to(F64) for t in (x, W0, Wg, Wu, W1, Wv)]
    keep = sr.keep_mask(T, D, p, seed, 1) / sr.kept_share(p)
    y = q[0] @ q[1].T + ((q[0] * keep) @ leaves[0].T) @ leaves[1].T
    lin = lambda v, W, k: v @ W.T + (v @ leaves[k].T) @ leaves[k + 1].T  # noqa: E731
    z = lin(torch.nn.functional.silu(lin(y, q[2], 2)) * lin(y, q[3], 4), q[4], 6)
    loss = torch.nn.functional.cross_entropy(z @ q[5].T, target)
    want = torch.autograd.grad(loss, leaves)
    # on the card
    x, W0, Wg, Wu, W1, Wv, target = (t.to(DEV) for t in (x, W0, Wg, Wu, W1, Wv, target))
    ad = [(a.to(DEV), b.to(DEV)) for a, b in ad]
    params = [t for ab in ad for t in ab]
    grads = [torch.zeros(t.shape, dtype=torch.float32, device=DEV) for t in params]
    opt = rg.LoraAdamW(params, grads, lr=1e-2, weight_decay=0.0)
    gate, up = (dict(A=ad[i][0], B=ad[i][1], alpha=alpha) for i in (1, 2))
    y = rg.lora_linear_dropout(x, W0, None, *ad[0], alpha, p, seed, offset=1)
    h, saved = rg.lora_gated(y, Wg, Wu, gate, up, save=True)
    z = rg.lora_linear(h, W1, None, *ad[3], alpha)
    per, _, dz = rg.lora_cross_entropy(z, Wv, target, dloss=torch.full((T,), 1 / T, device=DEV), want=("loss", "dh"))
    dh, dA, dB, _ = rg.lora_linear_backward(h, W1, *ad[3], dz, alpha, want=("dx", "dA", "dB"))
    grads[6].copy_(dA)
    grads[7].copy_(dB)
    dy = rg.lora_gated_backward(y, Wg, Wu, gate, up, dh, saved=saved, dA_gate=grads[2], dB_gate=grads[3], dA_up=grads[4],
                                dB_up=grads[5])[0]
    rg.lora_linear_dropout_backward(x, W0, *ad[0], dy, alpha, p, seed, offset=1, want=("dA", "dB"), dA=grads[0], dB=grads[1])
    loss = float(loss.detach())
    assert abs(float(per.mean()) - loss) <= 6 * 2.0 ** -8 * loss
    for i, (a, b) in enumerate(zip(grads, want)):
        rel = float((sr.d(a) - b).norm() / b.norm())
        say(f"gradient {i}: {rel:.4f}")
        assert rel <= 12 * 2.0 ** -8, i
    before = [t.clone() for t in params]
    opt.step()
    for t, b, gr in zip(params, before, grads):
        # (the first step moves every element by lr against its gradient's sign, as far as bf16 shows it)
        moved = t.float() - b.float()
        assert bool(((moved * gr <= 0) | (gr == 0)).all()) and bool((moved != 0).any())

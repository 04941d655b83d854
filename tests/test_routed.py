"""The routed linear layer (tokens take their adapters from a pool) and its gradients: refusals on the
CPU, parity with the plain 64-bit form on the GPU."""
import numpy as np
import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import routed_ref as rr

OK, NULL, SHAPE, DTYPE, NONFIN, ALIGN, OVERLAP, WS, UNSUP, HIP = range(10)
DEV = "cuda:0"
X, W, Y, A, B, BIAS, WSP, IDS, TS, SC, RK, DY, DA, DB = (0x10_0000_0000 + i * 0x10_0000_0000 for i in range(14))


def say(*a):
    print(*a, flush=True)


# ----------------------------------------------------------------------------- refusals (no GPU)

def fwd(**kw):
    a = dict(x=X, T=0, K=128, ldx=128, W=W, N=96, bias=BIAS, A=A, B=B, sc=SC, rk=None, n=4, R=16, res=0, ids=IDS,
             ts=None, y=Y, ldy=96, ws=WSP, wsb=1 << 30)
    a.update(kw)
    pool = rg.LoraPool(a["A"], a["B"], a["sc"], a["rk"], a["n"], a["R"], a["res"])
    return rg._lib.lora_linear_routed_fwd(a["x"], a["T"], a["K"], a["ldx"], a["W"], a["N"], a["bias"],
                                          None if a.get("nopool") else pool, a["ids"], a["ts"], a["y"], a["ldy"],
                                          a["ws"], a["wsb"], None)


def bwd(**kw):
    a = dict(x=X, T=64, K=128, ldx=128, W=W, N=96, A=A, B=B, sc=SC, rk=None, n=4, R=16, res=0, ids=IDS, ts=None,
             dy=DY, lddy=96, dx=Y, lddx=128, dA=DA, dB=DB, ws=WSP, wsb=1 << 30)
    a.update(kw)
    pool = rg.LoraPool(a["A"], a["B"], a["sc"], a["rk"], a["n"], a["R"], a["res"])
    return rg._lib.lora_linear_routed_bwd(a["x"], a["T"], a["K"], a["ldx"], a["W"], a["N"],
                                          None if a.get("nopool") else pool, a["ids"], a["ts"], a["dy"], a["lddy"],
                                          a["dx"], a["lddx"], a["dA"], a["dB"], a["ws"], a["wsb"], None)


COMMON = [
    (dict(nopool=True), NULL), (dict(A=None), NULL), (dict(B=None), NULL), (dict(sc=None), NULL),
    (dict(x=None), NULL), (dict(W=None), NULL), (dict(ids=None), NULL),
    (dict(T=-1), SHAPE), (dict(K=0, ldx=0), SHAPE), (dict(N=0), SHAPE), (dict(ldx=120), SHAPE),
    (dict(n=-1), SHAPE), (dict(R=0), SHAPE), (dict(res=1), SHAPE),
    (dict(n=20000), UNSUP), (dict(R=1032), UNSUP), (dict(T=1 << 31), UNSUP),
    (dict(K=1 << 21, ldx=1 << 21, lddx=1 << 21), UNSUP), (dict(ldx=1 << 22), UNSUP),
    (dict(x=X + 2), ALIGN), (dict(W=W + 8), ALIGN), (dict(A=A + 8), ALIGN), (dict(B=B + 2), ALIGN),
    (dict(sc=SC + 2), ALIGN), (dict(rk=RK + 1), ALIGN), (dict(ids=IDS + 2), ALIGN), (dict(ts=TS + 1), ALIGN),
    (dict(R=12), ALIGN), (dict(K=124), ALIGN), (dict(ldx=132), ALIGN), (dict(ws=WSP + 8), ALIGN),
    (dict(ws=None), WS), (dict(wsb=255), WS),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(y=None), NULL), (dict(ldy=95), SHAPE), (dict(y=Y + 1), ALIGN), (dict(bias=BIAS + 1), ALIGN),
    (dict(ldy=1 << 22), UNSUP),
    (dict(y=X + 64), OVERLAP), (dict(y=A + 64), OVERLAP), (dict(y=IDS), OVERLAP), (dict(ws=B), OVERLAP),
    (dict(ws=Y), OVERLAP), (dict(ws=W), OVERLAP), (dict(y=SC), OVERLAP), (dict(ws=TS, ts=TS), OVERLAP),
])
def test_forward_refusals(kw, code):
    assert fwd(**{"T": 64, **kw}) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dy=None), NULL), (dict(lddy=88), SHAPE), (dict(lddx=120), SHAPE), (dict(dy=DY + 2), ALIGN),
    (dict(N=92, lddy=96), ALIGN), (dict(lddy=100), ALIGN), (dict(dA=DA + 2), ALIGN), (dict(dB=DB + 1), ALIGN),
    (dict(dx=Y + 1), ALIGN),
    (dict(dx=X), OVERLAP), (dict(dA=A), OVERLAP), (dict(dB=DA), OVERLAP), (dict(dA=WSP + 64), OVERLAP),
    (dict(ws=DY), OVERLAP), (dict(dB=IDS), OVERLAP),
])
def test_backward_refusals(kw, code):
    assert bwd(**kw) == code


def test_empty_calls_and_workspace_queries():
    assert fwd() == OK and fwd(x=None, y=None, ids=None, ws=None, wsb=0) == OK
    assert bwd(dx=None, dA=None, dB=None) == OK                       # nothing asked for
    q = rg.lora_linear_routed_workspace_size
    assert q(0, 128, 96, 4, 16) == 0 and q(64, 0, 96, 4, 16) == 0 and q(64, 128, 96, -1, 16) == 0
    assert q(64, 128, 96, 4, 16) >= 64 * 64 * 2
    need = q(64, 128, 96, 4, 16)
    assert fwd(T=64, wsb=need - 1) == WS
    qb = rg.lora_linear_routed_bwd_workspace_size
    assert qb(0, 128, 96, 4, 16) == 0
    assert qb(64, 128, 96, 4, 16, True) > qb(64, 128, 96, 4, 16, False) > 0
    assert bwd(wsb=qb(64, 128, 96, 4, 16) - 1) == WS
    assert bwd(W=None, dx=None, wsb=qb(64, 128, 96, 4, 16, False) - 1) == WS


@pytest.mark.parametrize("kw,code", [
    (dict(n=8193), UNSUP), (dict(T=1 << 26), UNSUP), (dict(K=1 << 62, ldx=1 << 62, lddx=1 << 62), UNSUP),
    (dict(ldx=(1 << 63) - 8), UNSUP), (dict(N=1 << 62, ldy=1 << 62, lddy=1 << 62), UNSUP),
])
def test_sizes_beyond_the_limits(kw, code):
    """Sizes whose bytes would pass 63 bits among them; the workspace queries know no size for them."""
    f = {k: v for k, v in kw.items() if k not in ("lddx", "lddy")}
    b = {k: v for k, v in kw.items() if k != "ldy"}
    assert fwd(**{"T": 64, **f}) == code and bwd(**b) == code
    if "n" in kw or "T" in kw or "K" in kw or "N" in kw:
        args = (kw.get("T", 64), kw.get("K", 128), kw.get("N", 96), kw.get("n", 4), 16)
        assert rg.lora_linear_routed_workspace_size(*args) == 0
        assert rg.lora_linear_routed_bwd_workspace_size(*args) == 0


def test_tensor_helpers_refuse():
    d = rr.case(8, 32, 24, 2, 8, 0)
    args = lambda **k: {**dict(x=d["x"], W=d["W"], b=d["b"], A=d["A"], B=d["B"], scales=d["scales"],  # noqa: E731
                               token_adapter=d["ids"]), **k}
    for bad, err in ((dict(token_adapter=d["ids"].long()), TypeError), (dict(scales=d["scales"].double()), TypeError),
                     (dict(A=d["A"].float()), TypeError), (dict(A=d["A"][:, :, ::2]), ValueError),
                     (dict(B=d["B"][:1]), ValueError), (dict(token_adapter=d["ids"][:4]), ValueError),
                     (dict(token_scale=torch.ones(3)), ValueError), (dict(ranks=torch.ones(2)), TypeError),
                     (dict(x=d["x"][0]), ValueError), (dict(W=d["W"].t()), ValueError)):
        with pytest.raises(err):
            rg.lora_linear_routed(**args(**bad))


# ----------------------------------------------------------------------------- parity (GPU)

def gpu(d):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def run_fwd(g, **kw):
    return rg.lora_linear_routed(g["x"], g["W"], g["b"], g["A"], g["B"], g["scales"], g["ids"],
                                 token_scale=g["token_scale"], ranks=g["ranks"], **kw)


def run_bwd(g, **kw):
    return rg.lora_linear_routed_backward(g["x"], g["W"], g["A"], g["B"], g["dy"], g["scales"], g["ids"],
                                          token_scale=g["token_scale"], ranks=g["ranks"], **kw)


# from one token to several tiles; ranks below, at and above a 64-rank stage; K below one MFMA step and off
# the 64-k stages; N of one column, odd, and over several tiles; more adapters than tokens and none at all
FWD = [
    (1, 8, 1, 1, 8, "mixed"), (1, 1536, 96, 3, 16, "mixed"), (2, 40, 7, 2, 8, "mixed"), (15, 200, 130, 4, 24, "mixed"),
    (16, 128, 96, 16, 16, "mixed"), (17, 264, 257, 40, 8, "mixed"), (64, 512, 300, 64, 32, "mixed"),
    (65, 520, 300, 7, 72, "mixed"), (129, 1544, 64, 3, 64, "packed"), (200, 72, 520, 5, 136, "mixed"),
    (300, 256, 513, 2, 64, "packed"), (257, 64, 256, 1, 16, "packed"), (1000, 136, 264, 6, 40, "packed"),
    (700, 328, 1100, 9, 128, "packed"), (33, 64, 48, 0, 8, "mixed"), (1030, 96, 2304, 300, 8, "mixed"),
    (1025, 2056, 72, 2, 64, "long"), (3001, 584, 260, 4, 136, "long"), (5000, 1032, 1100, 3, 24, "long"),
    (16500, 72, 40, 3, 72, "long"), (16500, 200, 24, 1, 64, "long"), (2100, 1160, 72, 30, 40, "packed"),
    (9000, 64, 24, 7, 72, "mixed"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout", FWD)
@pytest.mark.parametrize("variant", [0, 1])
def test_forward(T, K, N, n, R, layout, variant):
    say("routed fwd", T, K, N, n, R, layout, variant)
    d = rr.case(T, K, N, n, R, 7 * T + R, layout, bias=variant == 0, ranks=variant == 1 and n > 0, tscale=variant == 0)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    run_fwd(gpu(d), out=y)
    rr.check(y, *rr.forward(d), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 70, 300])
def test_forward_strides_and_rows_behind(T):
    """x and y as column views of wider buffers; what lies beside and behind the views stays as it was."""
    say("routed strides", T)
    K, N = 104, 75
    d = rr.case(T, K, N, 3, 16, T, "mixed")
    g = gpu(d)
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + K] = g["x"]
    out = torch.full((T + 3, N + 9), 7.0, dtype=torch.bfloat16, device=DEV)
    g["x"] = wide[:, 8:8 + K]
    run_fwd(g, out=out[:T, 5:5 + N])
    rr.check(out[:T, 5:5 + N], *rr.forward(d), "y")
    out[:T, 5:5 + N] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 90, 400])
def test_routing_values(T):
    """Indices outside the pool, zero scales and zero ranks give the base output; a rank is cut at the slot."""
    say("routed values", T)
    d = rr.case(T, 128, 160, 5, 24, T, "mixed", ranks=True)
    d["ids"][::3] = torch.tensor([5, -1, -7, 2 ** 31 - 1, -2 ** 31] * T)[: d["ids"][::3].numel()].to(torch.int32)
    d["token_scale"][1::5] = 0.0
    d["scales"][1] = 0.0
    d["ranks"][2] = 0
    d["ranks"][3] = 24
    ref = rr.forward(d)
    g = gpu(d)
    g["ranks"][3] = 1000
    rr.check(run_fwd(g), *ref, "y")
    (dx, dA, dB), bounds = rr.backward(d)
    for got, want, bound, what in zip(run_bwd(g), (dx, dA, dB), bounds, ("dx", "dA", "dB")):
        rr.check(got, want, bound, what)


@pytest.mark.gpu
@pytest.mark.parametrize("T,layout", [(40, "mixed"), (150, "mixed"), (600, "packed")])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_broken_adapter_stays_with_its_tokens(T, layout, value):
    """Infinite or NaN weights of one adapter reach its own tokens' outputs and gradients and no others;
    slots that no token takes and what lies behind an adapter's rank are not read."""
    say("routed broken", T, layout, value)
    d = rr.case(T, 96, 200, 4, 32, 3, layout, ranks=True)
    d["ids"][:4] = torch.tensor([0, 1, 2, 1])
    d["ids"][d["ids"] == 3] = 0
    clean = gpu(d)
    y0, g0 = run_fwd(clean), run_bwd(clean)
    bad = gpu(d)
    r = int(d["ranks"][0])
    bad["B"][1, 17, 0] = value
    bad["B"][1, 150, 3] = -value
    bad["A"][3], bad["B"][3] = value, value
    bad["A"][0, r:], bad["B"][0, :, r:] = value, value
    y1, g1 = run_fwd(bad), run_bwd(bad)
    mine = bad["ids"] == 1
    cols = torch.ones(200, dtype=torch.bool, device=DEV)
    cols[[17, 150]] = False
    assert torch.equal(y0[~mine], y1[~mine])
    rr.check(y1[mine][:, cols], rr.forward(d)[0][mine.cpu()][:, cols.cpu()],
             rr.forward(d)[1][mine.cpu()][:, cols.cpu()], "y, other columns")
    assert not bool(torch.isfinite(y1[mine][:, ~cols]).any())
    assert torch.equal(g0[0][~mine], g1[0][~mine])
    for a in (0, 2, 3):
        assert torch.equal(g0[1][a], g1[1][a]) and torch.equal(g0[2][a], g1[2][a])
    bad["A"][1, 2, 5] = value  # and in A: every output of its tokens
    y2 = run_fwd(bad)
    assert torch.equal(y0[~mine], y2[~mine]) and not bool(torch.isfinite(y2[mine][:, 17]).any())


@pytest.mark.gpu
def test_one_adapter_for_all_matches_the_plain_layer():
    """A pool of one: the accuracy of lora_linear on the same layer."""
    say("routed one adapter")
    d = rr.case(600, 256, 512, 1, 64, 5, "mixed", none=0.0, tscale=False)
    g = gpu(d)
    y = run_fwd(g)
    y1 = rg.lora_linear(g["x"], g["W"], g["b"], g["A"][0], g["B"][0], float(d["scales"][0]) * 64)
    want, bound = rr.forward(d)
    rr.check(y, want, bound, "routed")
    rr.check(y1, want, bound, "lora_linear")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 80])
def test_a_pool_beyond_32_bit_offsets(T):
    say("routed large pool", T)
    n, R, K, N = 1100, 256, 8192, 8200
    d = rr.case(T, K, N, 1, R, 1, "mixed", none=0.0)
    g = gpu(d)
    Ap = torch.zeros((n, R, K), dtype=torch.bfloat16, device=DEV)
    Bp = torch.zeros((n, N, R), dtype=torch.bfloat16, device=DEV)
    Ap[-1], Bp[-1] = g["A"][0], g["B"][0]
    sc = torch.ones(n, device=DEV)
    sc[-1] = g["scales"][0]
    y = rg.lora_linear_routed(g["x"], g["W"], g["b"], Ap, Bp, sc, g["ids"] + (n - 1), token_scale=g["token_scale"])
    rr.check(y, *rr.forward(d), "y")


BWD = [
    (1, 8, 8, 1, 8, "mixed"), (5, 128, 96, 3, 16, "mixed"), (17, 264, 200, 40, 8, "mixed"),
    (64, 512, 304, 9, 32, "mixed"), (129, 136, 64, 3, 64, "packed"), (300, 256, 520, 2, 72, "packed"),
    (1000, 136, 264, 6, 40, "packed"), (2500, 64, 48, 3, 16, "packed"), (5000, 40, 24, 2, 8, "packed"),
    (33, 64, 48, 0, 8, "mixed"), (700, 72, 528, 5, 136, "mixed"), (1100, 520, 1032, 3, 64, "long"),
    (3001, 264, 136, 4, 136, "long"), (16500, 40, 72, 2, 24, "long"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout", BWD)
@pytest.mark.parametrize("variant", [0, 1])
def test_backward(T, K, N, n, R, layout, variant):
    say("routed bwd", T, K, N, n, R, layout, variant)
    d = rr.case(T, K, N, n, R, 3 * T + R, layout, ranks=variant == 1 and n > 0, tscale=variant == 0)
    outs = dict(dx=torch.full((T, K), float("nan"), dtype=torch.bfloat16, device=DEV),
                dA=torch.full((n, R, K), float("nan"), device=DEV), dB=torch.full((n, N, R), float("nan"), device=DEV))
    got = run_bwd(gpu(d), **outs)
    want, bounds = rr.backward(d)
    for g, w, b, what in zip(got, want, bounds, ("dx", "dA", "dB")):
        rr.check(g, w, b, what)


@pytest.mark.gpu
def test_backward_against_differences():
    """L = sum(dy y) is linear in A and in B apart: its central difference along a direction D is <grad, D>
    exactly, here with the 64-bit forward."""
    say("routed differences")
    d = rr.case(90, 64, 72, 3, 16, 9, "packed")
    _, dA, dB = run_bwd(gpu(d))
    rng = np.random.default_rng(0)
    (_, wA, wB), (_, bA, bB) = rr.backward(d)
    for key, grad, bound in (("A", dA, bA), ("B", dB, bB)):
        D = torch.from_numpy(rng.choice([-1.0, 1.0], d[key].shape))
        loss = []
        for sign in (1, -1):
            e = dict(d)
            e[key] = d[key].double() + sign * 0.5 * D
            loss.append(float((rr.forward(e)[0] * d["dy"].double()).sum()))
        diff = loss[0] - loss[1]
        assert abs(diff - float((grad.cpu().double() * D).sum())) <= float(bound.sum()) + 1e-9 * sum(map(abs, loss))


@pytest.mark.gpu
def test_backward_partial_wants_and_empty_batch():
    say("routed wants")
    d = rr.case(50, 64, 48, 2, 8, 4)
    g = gpu(d)
    dx, dA, dB = run_bwd(g)
    for want in (("dx",), ("dA",), ("dB",), ("dA", "dB")):
        for name, got, full in zip(("dx", "dA", "dB"), run_bwd(g, want=want), (dx, dA, dB)):
            assert (got is None) == (name not in want) and (got is None or torch.equal(got, full))
    no_w = rg.lora_linear_routed_backward(g["x"], None, g["A"], g["B"], g["dy"], g["scales"], g["ids"],
                                          token_scale=g["token_scale"], want=("dA", "dB"))
    assert torch.equal(no_w[1], dA) and torch.equal(no_w[2], dB)
    e = {**g, "x": g["x"][:0], "dy": g["dy"][:0], "ids": g["ids"][:0], "token_scale": g["token_scale"][:0]}
    assert run_fwd(e).shape == (0, 48)
    _, eA, eB = run_bwd(e, dA=torch.full_like(dA, 3.0), dB=torch.full_like(dB, 3.0))
    assert not bool(eA.any()) and not bool(eB.any())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [12, 100, 500])
def test_captured_calls_take_the_routing_of_each_replay(T):
    """A captured forward and backward replayed with other routing, scales and inputs in the same buffers,
    eager calls of the same layer in between: the bits of the eager calls."""
    say("routed graph", T)
    d = rr.case(T, 128, 200, 4, 16, T, "packed")
    g = gpu(d)
    ws = torch.empty(rg.lora_linear_routed_workspace_size(T, 128, 200, 4, 16), dtype=torch.uint8, device=DEV)
    wb = torch.empty(rg.lora_linear_routed_bwd_workspace_size(T, 128, 200, 4, 16), dtype=torch.uint8, device=DEV)
    y, dx = torch.empty((T, 200), dtype=torch.bfloat16, device=DEV), torch.empty_like(g["x"])
    dA, dB = torch.empty(g["A"].shape, device=DEV), torch.empty(g["B"].shape, device=DEV)

    def both():
        run_fwd(g, out=y, workspace=ws)
        run_bwd(g, dx=dx, dA=dA, dB=dB, workspace=wb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        e = gpu(rr.case(T, 128, 200, 4, 16, 50 + k, "mixed" if k % 2 else "packed"))
        for name in ("x", "dy", "ids", "token_scale", "scales", "A", "B"):
            g[name].copy_(e[name])
        ref = (run_fwd(g), *run_bwd(g))
        for o in (y, dx, dA, dB):
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip((y, dx, dA, dB), ref):
            assert torch.equal(o, w)


@pytest.mark.gpu
def test_two_streams_and_repeats_give_the_same_bits():
    say("routed streams")
    cases = [gpu(rr.case(300, 128, 264, 5, 24, s, "mixed")) for s in (1, 2)]
    refs = [(run_fwd(g), *run_bwd(g)) for g in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(3):
        for k, (g, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[k].append((run_fwd(g), *run_bwd(g)))
    torch.cuda.synchronize()
    for ref, outs in zip(refs, got):
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, ref))


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout", [
    (200, 8968, 136, 5, 72, "mixed"), (20, 9000, 72, 6, 16, "mixed"), (16, 9000, 64, 16, 16, "mixed"),
    (700, 8200, 200, 9, 40, "packed"), (150, 72, 8200, 5, 72, "mixed"), (256, 1544, 2056, 40, 24, "mixed"),
    (1, 9000, 8, 1, 136, "mixed"), (300, 4104, 3000, 7, 16, "packed"),
])
def test_long_sums_beside_the_base_product(T, K, N, n, R, layout):
    """Rank-wide products in several parts, in one product of the backward or in both."""
    say("routed long sums", T, K, N, n, R, layout)
    d = rr.case(T, K, N, n, R, T + K, layout, ranks=True)
    g = gpu(d)
    rr.check(run_fwd(g), *rr.forward(d), "y")
    want, bounds = rr.backward(d)
    for got, w, b, what in zip(run_bwd(g), want, bounds, ("dx", "dA", "dB")):
        rr.check(got, w, b, what)


@pytest.mark.gpu
def test_rows_of_x_far_apart():
    """Rows of 4 MB: x spans more than 32 bits of bytes, tokens as they come and sorted."""
    say("routed wide rows")
    ld = 1 << 21
    wide = torch.empty((1024, ld), dtype=torch.bfloat16, device=DEV)
    for T in (1023, 200, 12):
        d = rr.case(T, 64, 72, 5, 16, T, "mixed")
        g = gpu(d)
        wide[:T, :64] = g["x"]
        g["x"] = wide[:T, :64]
        rr.check(run_fwd(g), *rr.forward(d), f"y, {T}")
    d = rr.case(1023, 72, 64, 5, 16, 4, "mixed")  # and of dy
    g = gpu(d)
    wide[:1023, :64] = g["dy"]
    g["dy"] = wide[:1023, :64]
    want, bounds = rr.backward(d)
    for got, w, b, what in zip(run_bwd(g), want, bounds, ("dx", "dA", "dB")):
        rr.check(got, w, b, what)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [30, 1500])
def test_the_largest_pool(T):
    say("routed largest pool", T)
    d = rr.case(T, 24, 16, 8192, 8, T, "mixed")
    d["ids"][0], d["ids"][1] = 8191, 0
    g = gpu(d)
    rr.check(run_fwd(g), *rr.forward(d), "y")
    want, bounds = rr.backward(d)
    for got, w, b, what in zip(run_bwd(g), want, bounds, ("dx", "dA", "dB")):
        rr.check(got, w, b, what)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 1200])
def test_broken_tokens_leave_the_rest_of_a_slot_at_zero(T):
    """Infinite and NaN tokens: other tokens' outputs and other adapters' gradients keep their bits, and what lies
    behind the adapter's rank stays zero."""
    say("routed broken tokens", T)
    d = rr.case(T, 96, 72, 3, 32, T, "mixed")
    d["ids"][:3] = torch.tensor([0, 1, 2])
    d["ranks"] = torch.tensor([16, 32, 8], dtype=torch.int32)
    live = torch.arange(32)[None, :] < d["ranks"][:, None]
    d["A"], d["B"] = d["A"] * live[:, :, None], d["B"] * live[:, None, :]
    g = gpu(d)
    y0, (dx0, dA0, dB0) = run_fwd(g), run_bwd(g)
    g["x"][0, 5], g["x"][0, 6] = float("inf"), float("nan")
    g["dy"][0, 7] = float("inf")
    y1, (dx1, dA1, dB1) = run_fwd(g), run_bwd(g)
    assert torch.equal(y0[1:], y1[1:]) and torch.equal(dx0[1:], dx1[1:])
    assert torch.equal(dA0[1:], dA1[1:]) and torch.equal(dB0[1:], dB1[1:])
    assert not bool(dA1[0, 16:].any()) and not bool(dB1[0, :, 16:].any())
    assert not bool(torch.isfinite(y1[0]).any()) and not bool(torch.isfinite(dA1[0, :16, 5]).any())


@pytest.mark.gpu
def test_calls_on_a_named_stream():
    """stream=: the call's own tensors belong to that stream; a stream of no device of the tensors is refused."""
    say("routed named stream")
    d = rr.case(300, 128, 264, 5, 24, 1, "mixed")
    g = gpu(d)
    ref = (run_fwd(g), *run_bwd(g))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(run_fwd(g, stream=side), *run_bwd(g, stream=side)) for _ in range(3)]
    side.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    with pytest.raises(ValueError):
        rg.lora_linear_routed(*(d[k] for k in ("x", "W", "b", "A", "B", "scales", "ids")), stream=side)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout", [
    (2100001, 16, 24, 3, 8, "long"), (3, 8, 1 << 20, 2, 8, "mixed"), (3, 1 << 20, 8, 2, 8, "mixed"),
    (1030, 1 << 16, 8, 2, 8, "long"), (1030, 8, 1 << 16, 6, 8, "mixed"),
])
def test_the_largest_extents(T, K, N, n, R, layout):
    """Millions of tokens, and the widest inputs and outputs."""
    say("routed extents", T, K, N, n, R, layout)
    d = rr.case(T, K, N, n, R, 11, layout)
    g = gpu(d)
    rr.check(run_fwd(g), *rr.forward(d), "y")
    want, bounds = rr.backward(d)
    for got, w, b, what in zip(run_bwd(g), want, bounds, ("dx", "dA", "dB")):
        rr.check(got, w, b, what)

"""Dropout before an adapter and the gated feed-forward: refusals on the CPU, parity with the formulas in 64 bits on
the GPU (tests/step_ref.py says what is allowed), gradients against differences, strides, streams and graphs."""
import ctypes
import math

import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import step_ref as sr

OK, NULL, SHAPE, DTYPE, NONFIN, ALIGN, OVERLAP, WS, UNSUP, HIP = range(10)
DEV = "cuda:0"
BF = torch.bfloat16
BASE = 0x10_0000_0000
NAN, INF = math.nan, math.inf


def say(*a):
    print(*a, flush=True)


# ----------------------------------------------------------------------------- refusals (no GPU)

DROP = dict(x=BASE, T=100, K=256, ldx=256, W=BASE * 2, N=128, bias=None, A=BASE * 3, B=BASE * 4, rank=16, alpha=16.0,
            strength=1.0, request=1.0, p=0.1, seed=1, offset=2, rng=None, dy=BASE * 5, lddy=128, y=BASE * 6, ldy=128,
            dx=BASE * 6, lddx=256, dA=BASE * 7, dB=BASE * 8, dtype=rg.LORA_F32, ws=BASE * 9, wb=1 << 30)


def drop_fwd(**kw):
    a = dict(DROP, **kw)
    return rg._lib.lora_linear_dropout_fwd(a["x"], a["T"], a["K"], a["ldx"], a["W"], a["N"], a["bias"], a["A"], a["B"],
                                           a["rank"], a["alpha"], a["strength"], a["request"], a["p"], a["seed"],
                                           a["offset"], a["rng"], a["y"], a["ldy"], a["ws"], a["wb"], None)


def drop_bwd(**kw):
    a = dict(DROP, **kw)
    return rg._lib.lora_linear_dropout_bwd(a["x"], a["T"], a["K"], a["ldx"], a["W"], a["N"], a["A"], a["B"], a["rank"],
                                           a["alpha"], a["strength"], a["request"], a["p"], a["seed"], a["offset"],
                                           a["rng"], a["dy"], a["lddy"], a["dx"], a["lddx"], a["dA"], a["dB"],
                                           a["dtype"], a["ws"], a["wb"], None)


BOTH = [
    (dict(x=None), NULL), (dict(A=None, B=None), NULL), (dict(A=None), NULL), (dict(B=None), NULL), (dict(W=None), NULL),
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(ldx=255), SHAPE), (dict(rank=0), SHAPE),
    (dict(rank=1032), UNSUP), (dict(T=1 << 21), UNSUP), (dict(K=1 << 21, ldx=1 << 21, lddx=1 << 21), UNSUP),
    (dict(p=-0.1), UNSUP), (dict(p=1.0), UNSUP), (dict(p=0.999999), UNSUP),
    (dict(p=NAN), NONFIN), (dict(alpha=INF), NONFIN), (dict(strength=NAN), NONFIN), (dict(request=INF), NONFIN),
    (dict(alpha=1e300), NONFIN),
    (dict(x=BASE + 8), ALIGN), (dict(W=BASE * 2 + 2), ALIGN), (dict(A=BASE * 3 + 8), ALIGN), (dict(B=BASE * 4 + 4), ALIGN),
    (dict(rank=12), ALIGN), (dict(K=260, ldx=264, lddx=264), ALIGN), (dict(ldx=260), ALIGN), (dict(ws=BASE * 9 + 8), ALIGN),
    (dict(rng=BASE + 4), ALIGN), (dict(ws=None), WS), (dict(wb=64), WS),
    (dict(ws=BASE), OVERLAP), (dict(ws=BASE * 3), OVERLAP),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(y=None), NULL), (dict(ldy=127), SHAPE), (dict(y=BASE * 6 + 1), ALIGN), (dict(y=BASE + 1024), OVERLAP),
    (dict(y=BASE * 2), OVERLAP), (dict(y=BASE * 9 + 4096), OVERLAP), (dict(bias=BASE * 6 + 20), OVERLAP),
    (dict(bias=BASE + 1), ALIGN),
])
def test_dropout_forward_refusals(kw, code):
    assert drop_fwd(**kw) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(dy=None), NULL), (dict(lddy=127), SHAPE), (dict(lddx=255), SHAPE), (dict(dtype=2), DTYPE),
    (dict(N=132, lddy=136), ALIGN), (dict(lddy=132), ALIGN), (dict(dy=BASE * 5 + 2), ALIGN), (dict(dA=BASE * 7 + 2), ALIGN),
    (dict(dx=BASE * 5), OVERLAP), (dict(dA=BASE * 6 + 8), OVERLAP), (dict(dB=BASE * 7 + 64), OVERLAP),
    (dict(lddx=1 << 22), UNSUP),
])
def test_dropout_backward_refusals(kw, code):
    assert drop_bwd(**kw) == code


GATED = dict(x=BASE, T=100, K=256, ldx=256, F=128, act=0, strength=1.0, request=1.0, h=BASE * 2, ldh=128, saved=None,
             dh=BASE * 3, lddh=128, dx=BASE * 4, lddx=256, grads=(BASE * 5, BASE * 6, BASE * 7, BASE * 8), dtype=rg.LORA_F32,
             ws=BASE * 9, wb=1 << 32, Wg=BASE * 10, Wu=BASE * 11, bg=None, bu=None, Ag=BASE * 12, Bg=BASE * 13, Au=BASE * 14,
             Bu=BASE * 15, rg=16, ru=8, alg=16.0, alu=8.0, layer=True)


def gated(backward, **kw):
    a = dict(GATED, **kw)
    layer = rg.LoraGatedLayer(a["Wg"], a["Wu"], a["bg"], a["bu"], a["Ag"], a["Bg"], a["Au"], a["Bu"], a["rg"], a["ru"],
                              a["alg"], a["alu"])
    ref = ctypes.byref(layer) if a["layer"] else None
    if not backward:
        return rg._lib.lora_gated_fwd(a["x"], a["T"], a["K"], a["ldx"], ref, a["F"], a["act"], a["strength"], a["request"],
                                      a["h"], a["ldh"], a["saved"], a["ws"], a["wb"], None)
    return rg._lib.lora_gated_bwd(a["x"], a["T"], a["K"], a["ldx"], ref, a["F"], a["act"], a["strength"], a["request"],
                                  a["dh"], a["lddh"], a["saved"], a["dx"], a["lddx"], *a["grads"], a["dtype"], a["ws"],
                                  a["wb"], None)


GATED_BOTH = [
    (dict(layer=False), NULL), (dict(x=None), NULL), (dict(Wg=None), NULL), (dict(Wu=None), NULL), (dict(Ag=None), NULL),
    (dict(Bu=None), NULL),
    (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(F=0), SHAPE), (dict(ldx=100), SHAPE), (dict(rg=0), SHAPE),
    (dict(ru=-8), SHAPE), (dict(ru=1032), UNSUP), (dict(act=3), UNSUP), (dict(act=-1), UNSUP), (dict(T=1 << 21), UNSUP),
    (dict(strength=NAN), NONFIN), (dict(alu=INF), NONFIN), (dict(alg=1e300), NONFIN), (dict(request=-INF), NONFIN),
    (dict(rg=12), ALIGN), (dict(K=252, ldx=256), ALIGN), (dict(ldx=260), ALIGN), (dict(Wu=BASE * 11 + 8), ALIGN),
    (dict(x=BASE + 2), ALIGN), (dict(bg=BASE + 1), ALIGN), (dict(saved=BASE * 20 + 8), ALIGN), (dict(ws=BASE * 9 + 8), ALIGN),
    (dict(ws=None), WS), (dict(wb=128), WS), (dict(ws=BASE * 12), OVERLAP),
]


@pytest.mark.parametrize("kw,code", GATED_BOTH + [
    (dict(h=None), NULL), (dict(ldh=127), SHAPE), (dict(h=BASE * 2 + 1), ALIGN), (dict(h=BASE * 10), OVERLAP),
    (dict(h=BASE * 9), OVERLAP), (dict(saved=BASE * 2), OVERLAP), (dict(saved=BASE * 9), OVERLAP),
    (dict(bu=BASE * 2 + 32), OVERLAP),
])
def test_gated_forward_refusals(kw, code):
    assert gated(False, **kw) == code


@pytest.mark.parametrize("kw,code", GATED_BOTH + [
    (dict(dh=None), NULL), (dict(lddh=127), SHAPE), (dict(lddx=255), SHAPE), (dict(dtype=7), DTYPE),
    (dict(F=132, lddh=136), ALIGN), (dict(lddh=132), ALIGN), (dict(grads=(BASE * 5 + 2, None, None, None)), ALIGN),
    (dict(Ag=None, Bg=None), NULL), (dict(dx=BASE), OVERLAP), (dict(grads=(BASE * 5, BASE * 5, None, None)), OVERLAP),
    (dict(saved=BASE * 4), OVERLAP), (dict(grads=(BASE * 3, None, None, None)), OVERLAP),
])
def test_gated_backward_refusals(kw, code):
    assert gated(True, **kw) == code


def test_workspace_sizes():
    d, db = rg.lora_linear_dropout_workspace_size, rg.lora_linear_dropout_bwd_workspace_size
    g, gb, gs = rg.lora_gated_workspace_size, rg.lora_gated_bwd_workspace_size, rg.lora_gated_saved_size
    assert d(0, 64, 64, 8) == 0 and db(5, 0, 64, 8) == 0 and g(0, 64, 64, 8, 8) == 0 and gs(0, 64, 8, 8) == 0
    assert d(1 << 21, 64, 64, 8) == 0 and gb(1 << 21, 64, 64, 8, 8) == 0
    for T in (1, 65, 5000):
        assert 0 < d(T, 512, 256, 16) <= db(T, 512, 256, 16)
        assert 0 < g(T, 512, 256, 16, 8) <= gb(T, 512, 256, 16, 8)
        assert gs(T, 256, 16, 8) >= T * 256 * 8


def test_python_refusals():
    x, W, A, B = torch.zeros(4, 64, dtype=BF), torch.zeros(32, 64, dtype=BF), torch.zeros(8, 64, dtype=BF), torch.zeros(32, 8, dtype=BF)
    with pytest.raises(TypeError):
        rg.lora_linear_dropout(x.float(), W, None, A, B, 8.0, 0.1, 1)
    with pytest.raises(ValueError):
        rg.lora_linear_dropout(x, W, None, A, B.T, 8.0, 0.1, 1)
    with pytest.raises(ValueError):
        rg.lora_linear_dropout(x, W, None, A, B, 8.0, 0.1, 1, rng=torch.zeros(3, dtype=torch.int64))
    ad = dict(A=A, B=B, alpha=8.0)
    with pytest.raises(ValueError):
        rg.lora_gated(x, W, W[:16], ad, ad)
    with pytest.raises(TypeError):
        rg.lora_gated(x, W, W.float(), ad, ad)
    with pytest.raises(KeyError):
        rg.lora_gated(x, W, W, ad, ad, act="relu")
    with pytest.raises(ValueError):
        rg.lora_gated(x, W, W, ad, ad, saved=torch.zeros(8, dtype=torch.uint8))


def test_the_generator_keeps_the_share_it_is_asked_for():
    """The oracle's masks: their share (within 6 deviations), and none alike for another seed, offset or row."""
    for p in (0.0, 0.05, 0.5, 0.9):
        m = sr.keep_mask(64, 4096, p, 123456789012345, 7)
        n, q = m.numel(), sr.kept_share(p)
        assert abs(float(m.sum()) - n * q) <= 6 * math.sqrt(n * q * (1 - q)) + 1e-9
    a = sr.keep_mask(2, 2048, 0.5, 1, 0)
    for b in (sr.keep_mask(2, 2048, 0.5, 2, 0), sr.keep_mask(2, 2048, 0.5, 1, 1), sr.keep_mask(2, 2048, 0.5, 1 << 32, 0), a.flip(0)):
        assert 0.4 < float((a != b).double().mean()) < 0.6


# ----------------------------------------------------------------------------- parity (GPU)

def rand(g, shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(BF)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def up_to(t):
    return None if t is None else t.to(DEV)


def drop_case(T, K, N, R, seed=0, bias=True):
    g = gen(seed)
    return dict(x=rand(g, (T, K)), W=rand(g, (N, K), K ** -0.5), b=rand(g, (N,), 0.1) if bias else None,
                A=rand(g, (R, K), K ** -0.5), B=rand(g, (N, R), 0.15), dy=rand(g, (T, N)))


def run_drop(c, dtype=torch.float32, **how):
    v = {k: up_to(t) for k, t in c.items()}
    y = rg.lora_linear_dropout(v["x"], v["W"], v["b"], v["A"], v["B"], **how)
    dx, dA, dB = rg.lora_linear_dropout_backward(v["x"], v["W"], v["A"], v["B"], v["dy"], grad_dtype=dtype, **how)
    return dict(y=y, dx=dx, dA=dA, dB=dB)


def check_drop(got, want, dtype, what):
    for k, v in got.items():
        sr.check(v, want[k], BF if k in ("y", "dx") else dtype, f"{what} {k}")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,R,p", [
    (1, 64, 64, 8, 0.1), (1, 1536, 8, 16, 0.5), (3, 8, 1536, 8, 0.3), (17, 72, 200, 24, 0.0), (64, 128, 136, 64, 0.05),
    (65, 520, 264, 40, 0.25), (129, 1032, 128, 72, 0.1), (257, 256, 640, 128, 0.9), (300, 2048, 1000, 136, 0.2),
    (700, 1536, 1536, 16, 0.05), (4100, 512, 256, 32, 0.1), (2500, 264, 4104, 200, 0.15),
])
def test_dropout_against_the_formulas(T, K, N, R, p):
    say("dropout", T, K, N, R, p)
    c = drop_case(T, K, N, R)
    how = dict(alpha=1.5 * R, p=p, seed=0xDEADBEEF12345678, offset=3 + (1 << 40), strength=0.8, request_scale=1.25)
    want = sr.dropout(c["x"], c["W"], c["b"], c["A"], c["B"], how["alpha"], p, how["seed"], how["offset"], 0.8, 1.25, c["dy"])
    for dtype in (torch.float32, BF):
        check_drop(run_drop(c, dtype, **how), want, dtype, f"{dtype}")


@pytest.mark.gpu
@pytest.mark.parametrize("tiles", ["256", "128"])
def test_dropout_large_tiles(tiles):
    """Both output tiles of the base product and of its gradient."""
    T, K, N, R = (8200, 1032, 2056, 16) if tiles == "256" else (1100, 2056, 1544, 72)
    say("dropout tiles", T, K, N, R)
    c = drop_case(T, K, N, R, 5, bias=False)
    how = dict(alpha=2.0 * R, p=0.1, seed=11, offset=0)
    got = run_drop(c, BF, **how)
    rows = torch.cat((torch.arange(0, 40), torch.arange(T - 300, T)))
    # (the outputs of a row need its own tokens alone; the masks of the whole tensor)
    keep = sr.keep_mask(T, K, 0.1, 11, 0)[rows]
    x, W, A, B, dy = (sr.d(v) for v in (c["x"][rows], c["W"], c["A"], c["B"], c["dy"][rows]))
    s = 2.0 / sr.kept_share(0.1)
    t, te = sr.rank_pair(x * keep, A, s)
    sr.check(got["y"][rows], sr.linear(x, W, None, [(t, te, B)]), BF, "y")
    u, ue = sr.rank_pair(dy, B.T, s)
    base, be = sr.linear(dy, W.T, None, [])
    ext, ee = sr.linear(dy, torch.zeros_like(W.T), None, [(u, ue, A.T)])
    sr.check(got["dx"][rows], (base + keep * ext, be + keep * ee + 2 * R * sr.U * base.abs()), BF, "dx")


@pytest.mark.gpu
def test_dropout_zero_scale_zero_tokens_and_partial_wants():
    say("dropout edges")
    c = drop_case(70, 128, 64, 16)
    v = {k: up_to(t) for k, t in c.items()}
    how = dict(alpha=0.0, p=0.3, seed=1)
    v["A"][0, 0], v["B"][0, 0] = INF, NAN  # an inactive adapter is not read
    y = rg.lora_linear_dropout(v["x"], v["W"], v["b"], v["A"], v["B"], **how)
    dx, dA, dB = rg.lora_linear_dropout_backward(v["x"], v["W"], v["A"], v["B"], v["dy"], **how)
    sr.check(y, sr.linear(sr.d(c["x"]), sr.d(c["W"]), sr.d(c["b"]), []), BF, "y")
    sr.check(dx, sr.linear(sr.d(c["dy"]), sr.d(c["W"]).T, None, []), BF, "dx")
    assert not bool(dA.any()) and not bool(dB.any())
    v = {k: up_to(t) for k, t in c.items()}
    how["alpha"] = 16.0
    e = v["x"][:0]
    assert rg.lora_linear_dropout(e, v["W"], v["b"], v["A"], v["B"], **how).shape == (0, 64)
    dA = torch.full((16, 128), 7.0, device=DEV)
    _, dA, dB = rg.lora_linear_dropout_backward(e, v["W"], v["A"], v["B"], v["dy"][:0], dA=dA, grad_dtype=torch.float32, **how)
    assert not bool(dA.any()) and not bool(dB.any())
    whole = run_drop(c, **how)
    for want in (("dx",), ("dA",), ("dB",), ("dA", "dB")):
        got = dict(zip(("dx", "dA", "dB"), rg.lora_linear_dropout_backward(v["x"], v["W"], v["A"], v["B"], v["dy"], want=want, **how)))
        for k, t in got.items():
            assert (t is None) == (k not in want)
            assert t is None or torch.equal(t, whole[k]), k


def rows_of(t, ld, fill=float("nan")):
    """The same values in a buffer with a wider row stride, what lies between them not finite."""
    buf = torch.full((t.shape[0], ld), fill, dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.gpu
def test_dropout_strides_and_outputs_beside():
    """Row strides wider than the rows (NaN between them), outputs as column views: nothing beside them is written."""
    say("dropout strides")
    T, K, N, R = 130, 200, 72, 16
    c = drop_case(T, K, N, R, 3)
    how = dict(alpha=8.0, p=0.2, seed=9, offset=1)
    plain = run_drop(c, BF, **how)
    v = {k: up_to(t) for k, t in c.items()}
    x, dy = rows_of(v["x"], K + 24), rows_of(v["dy"], N + 8)
    wide = torch.full((T + 1, N + 5), 3.0, dtype=BF, device=DEV)
    y = rg.lora_linear_dropout(x, v["W"], v["b"], v["A"], v["B"], out=wide[:T, 3:3 + N], **how)
    assert torch.equal(y, plain["y"])
    assert bool((wide[:, :3] == 3).all()) and bool((wide[:, 3 + N:] == 3).all()) and bool((wide[T] == 3).all())
    wide = torch.full((T + 1, K + 7), 3.0, dtype=BF, device=DEV)
    dx, dA, dB = rg.lora_linear_dropout_backward(x, v["W"], v["A"], v["B"], dy, dx=wide[:T, 5:5 + K], grad_dtype=BF, **how)
    assert torch.equal(dx, plain["dx"]) and torch.equal(dA, plain["dA"]) and torch.equal(dB, plain["dB"])
    assert bool((wide[:, :5] == 3).all()) and bool((wide[:, 5 + K:] == 3).all()) and bool((wide[T] == 3).all())


@pytest.mark.gpu
def test_dropout_no_mask_is_the_plain_layer_and_offsets_differ():
    say("dropout p = 0")
    c = drop_case(200, 512, 256, 32, 1)
    v = {k: up_to(t) for k, t in c.items()}
    a = rg.lora_linear_dropout(v["x"], v["W"], v["b"], v["A"], v["B"], 32.0, 0.0, 5)
    b = rg.lora_linear_dropout(v["x"], v["W"], v["b"], v["A"], v["B"], 32.0, 0.0, 6, offset=9)
    assert torch.equal(a, b)
    one = run_drop(c, alpha=32.0, p=0.5, seed=5, offset=0)
    two = run_drop(c, alpha=32.0, p=0.5, seed=5, offset=1)
    assert not torch.equal(one["y"], two["y"]) and not torch.equal(one["dA"], two["dA"])
    rng = torch.tensor([5, 1], dtype=torch.int64, device=DEV)
    dev = run_drop(c, alpha=32.0, p=0.5, seed=77, offset=77, rng=rng)
    assert all(torch.equal(dev[k], two[k]) for k in two)


def gated_case(T, K, F, rg_, ru, seed=0, bias=True):
    g = gen(seed)
    side = lambda r: None if r == 0 else dict(A=rand(g, (r, K), K ** -0.5), B=rand(g, (F, r), 0.15), alpha=1.25 * r)  # noqa: E731
    return dict(x=rand(g, (T, K)), Wg=rand(g, (F, K), K ** -0.5), Wu=rand(g, (F, K), K ** -0.5), gate=side(rg_), up=side(ru),
                bg=rand(g, (F,), 0.2) if bias else None, bu=rand(g, (F,), 0.2) if bias else None, dh=rand(g, (T, F)))


def on_gpu(c):
    return {k: {n: up_to(t) if torch.is_tensor(t) else t for n, t in v.items()} if isinstance(v, dict) else up_to(v)
            for k, v in c.items()}


NAMES = ("dx", "dA_gate", "dB_gate", "dA_up", "dB_up")


def run_gated(c, act, dtype=torch.float32, save=True, backward=True, **how):
    v = on_gpu(c)
    kw = dict(b_gate=v["bg"], b_up=v["bu"], act=act, **how)
    h = rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], save=save, **kw)
    h, saved = h if save else (h, None)
    out = {"h": h}
    if backward:
        got = rg.lora_gated_backward(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], v["dh"], saved=saved, grad_dtype=dtype, **kw)
        out.update({n: t for n, t in zip(NAMES, got) if t is not None})
    return out


def want_gated(c, act, strength=1.0, request=1.0, backward=True):
    return sr.gated(c["x"], c["Wg"], c["Wu"], c["gate"], c["up"], c["bg"], c["bu"], act, strength, request,
                    c["dh"] if backward else None)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,F,rg_,ru", [
    (1, 64, 64, 8, 8), (2, 1536, 40, 16, 0), (5, 8, 1000, 0, 24), (16, 136, 16, 0, 0), (48, 512, 272, 16, 16), (64, 264, 520, 64, 8),
    (65, 72, 136, 40, 72), (129, 1032, 64, 8, 200), (300, 512, 1544, 64, 64), (1030, 264, 2056, 32, 16),
])
def test_gated_against_the_formulas(T, K, F, rg_, ru, act):
    say("gated", T, K, F, rg_, ru, act)
    c = gated_case(T, K, F, rg_, ru)
    want = want_gated(c, act, 0.7, 1.1)
    for dtype, save in ((torch.float32, True), (BF, False)):
        got = run_gated(c, act, dtype, save, strength=0.7, request_scale=1.1)
        assert set(got) == set(want)
        for k, t in got.items():
            sr.check(t, want[k], BF if k in ("h", "dx") else dtype, f"{dtype} {k}")


@pytest.mark.gpu
@pytest.mark.parametrize("T,F", [(1, 37), (7, 129), (64, 1001), (100, 63), (70, 1)])
def test_gated_forward_odd_widths(T, F):
    """F need not be a multiple of anything in the forward call."""
    say("gated odd", T, F)
    c = gated_case(T, 128, F, 16, 8, 2)
    sr.check(run_gated(c, "silu", backward=False, save=False)["h"], want_gated(c, "silu", backward=False)["h"], BF, "h")


@pytest.mark.gpu
def test_gated_large_tiles():
    T, K, F = 8200, 520, 1608
    say("gated large", T, K, F)
    c = gated_case(T, K, F, 16, 8, 4)
    got = run_gated(c, "silu", BF)
    rows = torch.cat((torch.arange(0, 20), torch.arange(T - 300, T)))
    part = dict(c, x=c["x"][rows], dh=c["dh"][rows])
    want = want_gated(part, "silu")
    sr.check(got["h"][rows], want["h"], BF, "h")
    sr.check(got["dx"][rows], want["dx"], BF, "dx")


@pytest.mark.gpu
def test_gated_extreme_activations():
    """Gate values far out on both sides: no NaN where the function has a value."""
    say("gated extremes")
    for act in ("silu", "gelu", "gelu_tanh"):
        c = gated_case(40, 64, 64, 0, 0, 6, bias=False)
        c["x"] = (c["x"].float() * 60).to(BF)
        want = want_gated(c, act)
        got = run_gated(c, act, BF)
        for k, t in got.items():
            assert bool(torch.isfinite(t).all()), (act, k)
            sr.check(t, want[k], BF, f"{act} {k}")


@pytest.mark.gpu
def test_gated_strides_inactive_and_empty():
    say("gated strides")
    T, K, F = 70, 136, 200
    c = gated_case(T, K, F, 16, 8, 7)
    plain = run_gated(c, "silu", BF)
    v = on_gpu(c)
    x, dh = rows_of(v["x"], K + 8), rows_of(v["dh"], F + 16)
    wide = torch.full((T + 1, F + 3), 3.0, dtype=BF, device=DEV)
    kw = dict(b_gate=v["bg"], b_up=v["bu"])
    h, saved = rg.lora_gated(x, v["Wg"], v["Wu"], v["gate"], v["up"], out=wide[:T, 1:1 + F], save=True, **kw)
    assert torch.equal(h, plain["h"]) and bool((wide[:, 0] == 3).all()) and bool((wide[:, 1 + F:] == 3).all()) and bool((wide[T] == 3).all())
    wide = torch.full((T + 1, K + 3), 3.0, dtype=BF, device=DEV)
    got = rg.lora_gated_backward(x, v["Wg"], v["Wu"], v["gate"], v["up"], dh, saved=saved, dx=wide[:T, 2:2 + K], grad_dtype=BF, **kw)
    assert all(torch.equal(a, plain[n]) for n, a in zip(NAMES, got))
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 2 + K:] == 3).all()) and bool((wide[T] == 3).all())
    # one adapter inactive, its values broken: not read, zero gradients
    off = dict(v["up"], alpha=0.0, A=v["up"]["A"] * INF)
    h = rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], off, **kw)
    sr.check(h, want_gated(dict(c, up=None), "silu", backward=False)["h"], BF, "inactive h")
    got = rg.lora_gated_backward(v["x"], v["Wg"], v["Wu"], v["gate"], off, v["dh"], **kw)
    want = want_gated(dict(c, up=None), "silu")
    for n in ("dx", "dA_gate", "dB_gate"):
        sr.check(got[NAMES.index(n)], want[n], BF if n == "dx" else torch.float32, f"inactive {n}")
    assert not bool(got[3].any()) and not bool(got[4].any())
    e = rg.lora_gated_backward(v["x"][:0], v["Wg"], v["Wu"], v["gate"], v["up"], v["dh"][:0], **kw)
    assert e[0].shape == (0, K) and not any(bool(t.any()) for t in e[1:])
    assert rg.lora_gated(v["x"][:0], v["Wg"], v["Wu"], v["gate"], v["up"], **kw).shape == (0, F)


@pytest.mark.gpu
def test_a_broken_token_stays_alone():
    """A token that is not finite reaches its own outputs and no other token's."""
    say("broken token")
    c = gated_case(100, 128, 136, 16, 16, 8)
    plain = run_gated(c, "silu", BF)
    drop = drop_case(100, 128, 136, 16, 8)
    dplain = run_drop(drop, BF, alpha=16.0, p=0.1, seed=3)
    for bad in (NAN, INF):
        x = c["x"].clone()
        x[41] = bad
        got = run_gated(dict(c, x=x), "silu", BF)
        rest = torch.arange(100) != 41
        for k in ("h", "dx"):
            assert torch.equal(got[k][rest], plain[k][rest]), k
        y = run_drop(dict(drop, x=torch.where(rest[:, None], drop["x"], torch.tensor(bad, dtype=BF))), BF, alpha=16.0, p=0.1, seed=3)
        for k in ("y", "dx"):
            assert torch.equal(y[k][rest], dplain[k][rest]), k


@pytest.mark.gpu
def test_gradients_against_differences():
    """Directional derivatives of the formulas' own sums by central differences in 64 bits: the kernels' gradients agree
    to the sum of their bounds along the direction."""
    say("differences")
    c = gated_case(24, 64, 48, 8, 16, 9)
    want = want_gated(c, "gelu")
    got = run_gated(c, "gelu", torch.float32)
    dh = sr.d(c["dh"])
    eps = 1e-5

    def value(**kw):
        v = {k: sr.d(t) if torch.is_tensor(t) else t for k, t in c.items()}
        v = dict(v, gate={k: sr.d(t) if torch.is_tensor(t) else t for k, t in c["gate"].items()},
                 up={k: sr.d(t) if torch.is_tensor(t) else t for k, t in c["up"].items()})
        for name, t in kw.items():
            if name == "x":
                v["x"] = t
            else:
                part, key = name.split("_")
                v[part][key] = t
        return float((sr.gated(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], v["bg"], v["bu"], "gelu")["h"][0] * dh).sum())

    g = gen(10)
    for name, grad in (("x", "dx"), ("gate_A", "dA_gate"), ("gate_B", "dB_gate"), ("up_A", "dA_up"), ("up_B", "dB_up")):
        base = sr.d(c["x"]) if name == "x" else sr.d(c[name.split("_")[0]][name.split("_")[1]])
        way = torch.randn(base.shape, generator=g, dtype=torch.float64)
        diff = (value(**{name: base + eps * way}) - value(**{name: base - eps * way})) / (2 * eps)
        v, e = want[grad]
        bound = (sr.rounded(v, e, BF if grad == "dx" else torch.float32) * way.abs()).sum() + 1e-6 * abs(diff)
        assert abs(float((sr.d(got[grad]) * way).sum()) - diff) <= float(bound), grad


@pytest.mark.gpu
def test_streams_workspaces_and_replays():
    """A named stream, a caller's workspace, and captured calls that are replayed with new inputs and a new offset."""
    say("streams and graphs")
    c, d = gated_case(200, 256, 136, 16, 16, 11), drop_case(200, 256, 136, 16, 11)
    v, w = on_gpu(c), {k: up_to(t) for k, t in d.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], stream=s)
    s.synchronize()
    assert torch.equal(h, rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"]))
    rng = torch.tensor([3, 0], dtype=torch.int64, device=DEV)
    ws = torch.empty(rg.lora_gated_bwd_workspace_size(200, 256, 136, 16, 16), dtype=torch.uint8, device=DEV)
    wd = torch.empty(rg.lora_linear_dropout_bwd_workspace_size(200, 256, 136, 16), dtype=torch.uint8, device=DEV)

    def step():
        h, saved = rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], save=True, workspace=ws)
        a = rg.lora_gated_backward(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], v["dh"], saved=saved, workspace=ws)
        y = rg.lora_linear_dropout(w["x"], w["W"], w["b"], w["A"], w["B"], 16.0, 0.3, 0, rng=rng, workspace=wd)
        b = rg.lora_linear_dropout_backward(w["x"], w["W"], w["A"], w["B"], w["dy"], 16.0, 0.3, 0, rng=rng, workspace=wd)
        return [h, *a, y, *b]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        v["x"].copy_(rand(gen(100 + i), (200, 256)))
        w["dy"].copy_(rand(gen(200 + i), (200, 136)))
        rng[1] += 1
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_same_call_same_bits():
    say("same bits")
    c = gated_case(1500, 512, 1000, 64, 64, 12)
    a, b = run_gated(c, "gelu_tanh"), run_gated(c, "gelu_tanh")
    assert all(torch.equal(a[k], b[k]) for k in a)
    d = drop_case(1500, 512, 1000, 64, 12)
    a, b = run_drop(d, alpha=64.0, p=0.1, seed=4), run_drop(d, alpha=64.0, p=0.1, seed=4)
    assert all(torch.equal(a[k], b[k]) for k in a)

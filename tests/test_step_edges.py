"""The operators of a fine-tuning step where they change their way or reach the ends of their ranges: sizes on both sides
of every choice of a kernel, tails of the activations, rows far apart, several calls at once."""
import math

import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import step_ref as sr
from tests import test_loss as tl
from tests import test_step as ts

BF, DEV = torch.bfloat16, "cuda:0"
say = ts.say


# ----------------------------------------------------------------------------- no GPU

@pytest.mark.parametrize("big", [1 << 40, 1 << 61, 1 << 62])
def test_sizes_beyond_64_bit_products(big):
    """Sizes whose bytes do not fit 64 bits are refused, not taken for small ones."""
    assert ts.drop_fwd(K=big, ldx=big) == ts.UNSUP and ts.drop_fwd(N=big, ldy=big) == ts.UNSUP
    assert ts.drop_fwd(ldx=big) == ts.UNSUP and ts.drop_bwd(lddx=big) == ts.UNSUP and ts.drop_bwd(lddy=big) == ts.UNSUP
    assert rg._lib.lora_cross_entropy(1 << 36, 4, big, big, 2 << 36, 10, 3 << 36, None, 4 << 36, None, None, 0, 5 << 36,
                                      1 << 30, None) == ts.UNSUP
    assert rg.lora_linear_dropout_workspace_size(100, big, 64, 16) == 0
    assert rg.lora_linear_dropout_bwd_workspace_size(100, 64, big, 16) == 0
    assert rg.lora_gated_workspace_size(100, big, 64, 16, 16) == 0 and rg.lora_gated_saved_size(100, big, 16, 16) == 0
    assert rg.lora_gated_bwd_workspace_size(big, 64, 64, 16, 16) == 0
    assert rg.lora_cross_entropy_workspace_size(100, 64, big) == 0 and rg.lora_cross_entropy_workspace_size(100, big, 64) == 0


def test_size_queries_take_what_the_calls_take():
    assert rg.lora_gated_saved_size(100, 64, 1024, 1024) > 0
    for bad in (1032, -1, 1 << 30):
        assert rg.lora_gated_saved_size(100, 64, bad, 16) == 0 and rg.lora_gated_workspace_size(100, 64, 64, 16, bad) == 0
        assert rg.lora_gated_bwd_workspace_size(100, 64, 64, bad, bad) == 0
        assert rg.lora_linear_dropout_workspace_size(100, 64, 64, bad) == 0
    assert rg.lora_linear_dropout_workspace_size(100, 64, 64, 0) == 0


# ----------------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 80])
def test_gelu_tails_keep_their_digits(T):
    """gelu far below zero, where it is a small part of its argument: right to the output's half step.

    Bound, relative: 2^-8 the output's rounding; the exponential's argument z^2 <= 72 carries 7 roundings of
    2^-24 (1 / sqrt 2 and z count twice in its square, the square, log2 e and the product), 72 * 7 * 2^-24 < 2^-15; the polynomial and the rest below 2^-20."""
    say("gelu tails", T)
    g = -torch.linspace(0.25, 12, 64)
    x = torch.zeros(T, 8)
    x[:, 0] = 1
    Wg, Wu = torch.zeros(64, 8), torch.zeros(64, 8)
    Wg[:, 0], Wu[:, 0] = g, 1
    got = rg.lora_gated(*(t.to(BF).to(DEV) for t in (x, Wg, Wu)), act="gelu")
    want = sr.act(sr.d(Wg.to(BF))[:, 0], "gelu")[0]
    assert bool(((sr.d(got) - want).abs() <= (2.0 ** -8 + 2.0 ** -15 + 2.0 ** -20) * want.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_far_out_have_their_limits(act):
    """Gates beyond where their squares are finite: act is g or 0 and act' 1 or 0, exactly."""
    say("far out", act)
    vals = torch.tensor([3e20, 1e30, 2e37, -3e20, -1e30, -2e37, 100.0, -120.0])  # (dh act(g) stays finite)
    T = 72
    x = torch.zeros(T, 8)
    x[torch.arange(T), torch.arange(T) % 8] = vals[torch.arange(T) % 8]
    eye = torch.eye(8)
    v = [t.to(BF).to(DEV) for t in (x, eye, torch.zeros(8, 8))]
    kw = dict(act=act, b_up=torch.ones(8, dtype=BF, device=DEV))
    dh = ts.rand(ts.gen(1), (T, 8)).to(DEV)
    for save in (True, False):
        h = rg.lora_gated(*v, save=save, **kw)
        h, saved = h if save else (h, None)
        assert torch.equal(h.float(), v[0].float().clamp_min(0))
        dx = rg.lora_gated_backward(*v, None, None, dh, saved=saved, want=("dx",), **kw)[0]
        on = v[0].float()
        # (a gate of 0 has act' = 1/2 in all three)
        want = torch.where(on > 0, dh.float(), torch.where(on < 0, 0.0, 0.5 * dh.float()))
        assert bool(((dx.float() - want).abs() <= 2.0 ** -7 * want.abs()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,R", [
    (1024, 520, 264, 64), (1025, 520, 264, 64), (40, 8192, 8192, 16), (40, 8200, 64, 16), (40, 64, 8200, 16),
    (40, 520, 136, 72), (30, 264, 136, 1024), (130, 136, 264, 512), (4096, 264, 136, 16), (4097, 264, 136, 16), (2730, 136, 264, 24),
    (2731, 136, 264, 24),
])
def test_dropout_on_both_sides_of_the_choices(T, K, N, R):
    say("dropout choices", T, K, N, R)
    c = ts.drop_case(T, K, N, R, 31)
    how = dict(alpha=1.0 * R, p=0.15, seed=5, offset=9)
    want = sr.dropout(c["x"], c["W"], c["b"], c["A"], c["B"], 1.0 * R, 0.15, 5, 9, dy=c["dy"])
    ts.check_drop(ts.run_drop(c, **how), want, torch.float32, "choice")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,F,rg_,ru", [
    (64, 136, 200, 32, 32), (65, 136, 200, 32, 32), (65, 136, 200, 0, 64), (70, 136, 200, 40, 32), (33, 72, 136, 1024, 1024),
    (1024, 72, 136, 16, 16), (1025, 72, 136, 64, 64), (20, 8200, 40, 16, 16), (20, 40, 8200, 16, 16), (1, 8, 8, 8, 8),
])
def test_gated_on_both_sides_of_the_choices(T, K, F, rg_, ru):
    say("gated choices", T, K, F, rg_, ru)
    c = ts.gated_case(T, K, F, rg_, ru, 32)
    want = ts.want_gated(c, "silu")
    for save in (True, False):
        for k, t in ts.run_gated(c, "silu", torch.float32, save).items():
            sr.check(t, want[k], BF if k in ("h", "dx") else torch.float32, f"{save} {k}")


@pytest.mark.gpu
@pytest.mark.parametrize("T,F", [(64, 8192), (65, 8192), (128, 8192), (129, 8192), (100, 8185), (128, 8200)])
def test_gated_forward_with_long_weights(T, F):
    """65 to 128 tokens where the weights are long (from 2^25 elements on), and beside it."""
    say("gated long", T, F)
    c = ts.gated_case(T, 4096, F, 16, 8, 39)
    sr.check(ts.run_gated(c, "silu", backward=False, save=False)["h"], ts.want_gated(c, "silu", backward=False)["h"], BF, "h")


@pytest.mark.gpu
def test_partial_wants_of_both_projections():
    """Each gradient alone, and one projection's alone."""
    say("gated wants")
    c = ts.gated_case(100, 136, 200, 16, 24, 33)
    v = ts.on_gpu(c)
    args = (v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], v["dh"])
    kw = dict(b_gate=v["bg"], b_up=v["bu"])
    want = ts.want_gated(c, "silu")
    for names in (("dx",), ("dA",), ("dB",), ("dx", "dB")):
        for n, a in zip(ts.NAMES, rg.lora_gated_backward(*args, want=names, **kw)):
            assert (a is None) != (n[:2] in names)
            if a is not None:
                sr.check(a, want[n], BF if n == "dx" else torch.float32, n)
    ws = torch.empty(rg.lora_gated_bwd_workspace_size(100, 136, 200, 16, 24), dtype=torch.uint8, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    layer = rg._gated_args(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], v["bg"], v["bu"])[3]
    one = torch.empty(200, 24, device=DEV)  # dB_up and nothing else
    rg.lora_gated_bwd(v["x"].data_ptr(), 100, 136, 136, layer, 200, 0, 1.0, 1.0, v["dh"].data_ptr(), 200, None, None, 0, None,
                      None, None, one.data_ptr(), rg.LORA_F32, ws.data_ptr(), ws.numel(), s)
    sr.check(one, want["dB_up"], torch.float32, "dB_up alone")


@pytest.mark.gpu
def test_rows_far_apart():
    """Row strides that put the last rows beyond 32-bit offsets."""
    say("far rows")
    T, K, N, R = 2100, 264, 136, 16
    c = ts.drop_case(T, K, N, R, 34)
    how = dict(alpha=16.0, p=0.1, seed=5, offset=0)
    near = ts.run_drop(c, BF, **how)
    v = {k: ts.up_to(t) for k, t in c.items()}
    ld = 1 << 20
    wide = [torch.empty(T, ld, dtype=BF, device=DEV) for _ in range(4)]  # 4.4 GB each
    x, dy, y, dx = wide[0][:, 8:8 + K], wide[1][:, :N], wide[2][:, 3:3 + N], wide[3][:, 1:1 + K]
    x.copy_(v["x"])
    dy.copy_(v["dy"])
    rg.lora_linear_dropout(x, v["W"], v["b"], v["A"], v["B"], out=y, **how)
    _, dA, dB = rg.lora_linear_dropout_backward(x, v["W"], v["A"], v["B"], dy, dx=dx, grad_dtype=BF, **how)
    for a, b in ((y, near["y"]), (dx, near["dx"]), (dA, near["dA"]), (dB, near["dB"])):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_more_than_two_to_the_31_outputs():
    say("large output")
    T, K, F = 33000, 64, 65544
    c = dict(ts.gated_case(8, K, F, 8, 0, 35), x=ts.rand(ts.gen(36), (T, K)))
    v = ts.on_gpu({k: c[k] for k in ("x", "Wg", "Wu", "gate", "bg", "bu")})
    h = rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], None, v["bg"], v["bu"])
    rows = torch.tensor([0, 1, 16383, 32767, 32768, 32775, T - 2, T - 1])
    sr.check(h[rows], ts.want_gated(dict(c, x=c["x"][rows]), "silu", backward=False)["h"], BF, "h")


@pytest.mark.gpu
@pytest.mark.parametrize("way", [1, -1])
def test_loss_pieces_with_logits_that_rise_or_fall(way):
    """Each piece of the vocabulary far above or far below those before it."""
    say("loss pieces", way)
    T, K, V = 9000, 8, 130003
    g = torch.Generator().manual_seed(36)
    W = torch.zeros(V, K)
    W[:, 0] = way * torch.linspace(-300, 300, V)
    W[:, 1:] = torch.randn(V, K - 1, generator=g)
    h = torch.randn(T, K, generator=g)
    h[:, 0] = torch.linspace(0.01, 2, T)
    target = torch.randint(0, V, (T,), generator=g)
    target[::7] = V - 1
    target[1::7] = 0
    c = dict(h=h.to(BF), W=W.to(BF), target=target, dloss=torch.ones(T))
    got = tl.run(c)
    rows = torch.cat((torch.arange(0, 40), torch.arange(4000, 4020), torch.arange(T - 40, T)))
    tl.check({k: v[rows] for k, v in got.items()}, tl.reference(c, rows))


@pytest.mark.gpu
def test_calls_at_once_on_two_streams():
    """Two streams, each with its own workspaces, the same leaves: the bits of one after the other."""
    say("two streams")
    c, d, e = ts.gated_case(300, 264, 520, 16, 16, 37), ts.drop_case(300, 264, 520, 16, 37), tl.case(300, 264, 5000, 37)
    v, w, l = ts.on_gpu(c), {k: ts.up_to(t) for k, t in d.items()}, {k: t.to(DEV) for k, t in e.items()}

    def calls(stream):
        h, saved = rg.lora_gated(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], save=True, stream=stream)
        return [h, *rg.lora_gated_backward(v["x"], v["Wg"], v["Wu"], v["gate"], v["up"], v["dh"], saved=saved, stream=stream),
                rg.lora_linear_dropout(w["x"], w["W"], w["b"], w["A"], w["B"], 16.0, 0.3, 1, stream=stream),
                *rg.lora_linear_dropout_backward(w["x"], w["W"], w["A"], w["B"], w["dy"], 16.0, 0.3, 1, stream=stream),
                *rg.lora_cross_entropy(l["h"], l["W"], l["target"], dloss=l["dloss"], stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(calls(s))
    torch.cuda.synchronize()
    for each in outs:
        for got in each:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_two_graphs_of_the_same_workspaces():
    """Two captured calls of different sizes that share their workspaces, replayed in turn on one stream."""
    say("two graphs")
    sizes = [(1, 5), (90, 6)]
    v = [ts.on_gpu(ts.gated_case(T, 136, 264, 16, 8, s)) for T, s in sizes]
    l = [{k: t.to(DEV) for k, t in tl.case(T, 136, 3001, s).items()} for T, s in sizes]
    size = max(rg.lora_gated_bwd_workspace_size(90, 136, 264, 16, 8), rg.lora_cross_entropy_workspace_size(90, 136, 3001))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def calls(i):
        a = v[i]
        h = rg.lora_gated(a["x"], a["Wg"], a["Wu"], a["gate"], a["up"], workspace=ws)
        g = rg.lora_gated_backward(a["x"], a["Wg"], a["Wu"], a["gate"], a["up"], a["dh"], workspace=ws)
        e = rg.lora_cross_entropy(l[i]["h"], l[i]["W"], l[i]["target"], dloss=l[i]["dloss"], workspace=ws)
        return [h, *g, *e]

    want = [[t.clone() for t in calls(i)] for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(calls(i))
    for i in (0, 1, 1, 0, 1, 0):
        for t in outs[i]:
            t.fill_(math.nan)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
        ws.fill_(0xFF)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,F,rg_,ru", [(1, 136, 264, 8, 16), (5, 64, 1000, 16, 8), (64, 264, 520, 64, 72), (300, 136, 1544, 16, 24),
                                          (200, 72, 520, 200, 136)])
def test_adapter_gradients_keep_more_than_bf16(T, K, F, rg_, ru):
    """dA at any length, and up to 64 tokens dB and dx, come from two bf16 terms of dg and du, not from one.

    Norms: two terms leave 2^-17 of each element and as much of each rank-wide row; were all errors of one sign, a sum of n
    products of random signs would have sqrt(n) times that, relative, which is below 2^-12 for n = 1544. One term leaves
    2^-9.2 in a norm (a uniform error of up to 2^-9 to 2^-8), eight times as much."""
    say("gated terms", T, K, F, rg_, ru)
    c = ts.gated_case(T, K, F, rg_, ru, 38)
    want = ts.want_gated(c, "gelu")
    got = ts.run_gated(c, "gelu", torch.float32)
    off = {n: float((sr.d(got[n]) - want[n][0]).norm() / want[n][0].norm()) for n in ts.NAMES}
    print(off, flush=True)
    for n in ("dA_gate", "dA_up") + (("dB_gate", "dB_up") if T <= 64 else ()):
        assert off[n] <= 2.0 ** -12, (n, off[n])
    if T <= 64:  # (its own rounding to bf16 alone, and 2^-12)
        own = float((sr.d(want["dx"][0].to(BF)) - want["dx"][0]).norm() / want["dx"][0].norm())
        assert off["dx"] <= 1.1 * own + 2.0 ** -12, (off["dx"], own)

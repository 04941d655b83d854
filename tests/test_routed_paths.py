"""The routed linear layer on each of the ways its sizes choose: the few-token kernels, and the hot GEMM behind the
rank-wide producer with its 128 x 128 and its 256 x 256 tile. Every GPU case names the way it is there for, and a
copy of the rules here (held to the sources by a CPU test) has to agree, so that a rule that moves shows which
cases it has emptied.

Bounds: a value rounded to bf16 is off by at most 2^-8 of it, to two bf16 terms by 2^-16, to fp32 by 2^-24, and a
sum of n fp32 products by at most (n + 1) 2^-24 of the sum of their magnitudes."""
import os
import shutil
import subprocess

import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import routed_ref as rr
from tests.test_routed import DEV, gpu, run_bwd, run_fwd, say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
U16, U32 = rr.U16, rr.U32


# ----------------------------------------------------------------------------- the rules

def up(a, b):
    return -(-a // b)


def way(T, N):
    """few: the few-token kernels; 128 or 256: the hot GEMM's tile on 256 compute units."""
    if T <= 256 or (T < 1025 and up(T, 128) * up(N, 128) <= 128):
        return "few"
    whole, small = 4.0 * up(up(T, 256) * up(N, 256), 256), 2.0 / 0.85 * up(up(T, 128) * up(N, 128), 512)
    return "128" if small < whole else "256"


def ring_splits(T, K):
    """Parts of K of the LDS ring that forms the rank-wide product; 0: no ring."""
    if T < 1025:
        return 0
    best, got, nk, mt = None, 0, up(2 * K, 128), up(T, 128)
    for s in range(1, 9):
        if s > 1 and nk // s < 4:
            break
        cost = up(mt * s, 256) / s * (1 + 0.04 * (s - 1))
        if best is None or cost < best:
            best, got = cost, up(nk, up(nk, s))
    return got


def taken(d):
    """The adapter of each token as the kernels see it: -1 without one."""
    s = torch.full((len(d["ids"]),), -1)
    for a, rows, _ in rr._per_adapter(d):
        s[rows] = a
    return s


def tiles(d, tokens):
    """(tiles of one adapter, tiles of several) of so many tokens."""
    kinds = [set(t.tolist()) for t in taken(d).split(tokens)]
    return sum(len(k) == 1 and k != {-1} for k in kinds), sum(len(k) > 1 for k in kinds)


def left_over(d):
    """Blocks of 128 tokens with more adapters than the ring takes (8)."""
    return sum(len(set(t.tolist()) - {-1}) > 8 for t in taken(d).split(128))


SHAPES = [(T, N) for T in (1, 16, 17, 256, 257, 300, 512, 1000, 1024, 1025, 1500, 3001, 4000, 9000, 32760)
          for N in (1, 40, 200, 513, 1100, 2049, 2900, 6000, 8960)]


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the ROCm headers")
def test_rules_are_the_sources(tmp_path):
    src = tmp_path / "rules.cpp"
    src.write_text("""
#include <cstdio>
#include "routed.hpp"
int main() {
  long T, N;
  while (std::scanf("%ld %ld", &T, &N) == 2) {
    int splits, ks;
    lora::ring_plan(T, N, &splits, &ks);
    std::printf("%s %d\\n", lora::few_path(T, N) ? "few" : (lora::small_tile(T, N, 256) ? "128" : "256"), splits);
  }
}
""")
    exe = str(tmp_path / "rules")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "rank_gemm_lora_amd", "csrc"), str(src),
                    "-o", exe], check=True)
    out = subprocess.run([exe], input="\n".join(f"{T} {N}" for T, N in SHAPES), text=True, capture_output=True, check=True)
    assert out.stdout.split("\n")[:-1] == [f"{way(T, N)} {ring_splits(T, N)}" for T, N in SHAPES]


# ----------------------------------------------------------------------------- the layer in 64 bits

def layer(d, x, W, b, A, B):
    """x W^T + b + s (x A^T) B^T in 64 bits, and how far a correct bf16 result may be off: the rank-wide product is
    kept as two bf16 terms (2^-16 of it), everything else in fp32, and the sum is rounded once."""
    K, R = x.shape[1], A.shape[1]
    y, mag = x @ W.T, x.abs() @ W.abs().T
    tb = torch.zeros_like(y)
    for a, rows, s in rr._per_adapter(d):
        r = R if d["ranks"] is None else min(int(d["ranks"][a]), R)
        Aa, Ba = A[a, :r], B[a, :, :r]
        t, tmag = (x[rows] @ Aa.T) * s, (x[rows].abs() @ Aa.abs().T) * s.abs()
        y[rows] += t @ Ba.T
        mag[rows] += (t.abs() * (1 + 2 * U16)) @ Ba.abs().T
        # (K products, up to 8 parts of K, the scale)
        tb[rows] += (t.abs() * U16 ** 2 + tmag * (K + 11) * U32) @ Ba.abs().T
    if b is not None:
        y += b
        mag += b.abs()
    # K + 2 R products, up to 16 parts of K, the adapter and the bias
    off = tb + (K + 2 * R + 20) * U32 * (mag + tb)
    return y, off + U16 * (y.abs() + off)


def forward(d):
    return layer(d, d["x"].double(), d["W"].double(), None if d["b"] is None else d["b"].double(), d["A"].double(),
                 d["B"].double())


def gradient(d):
    """dx and its bound: the layer of dy with W, A and B transposed."""
    return layer(d, d["dy"].double(), d["W"].double().T, None, d["B"].double().transpose(1, 2),
                 d["A"].double().transpose(1, 2))


# ----------------------------------------------------------------------------- the rank-wide product's bits

# (T, K, N, n, R, layout, way): tokens of one adapter per tile ("long") and of several
BITS = [
    (9, 72, 200, 3, 24, "mixed", "few"), (100, 264, 304, 5, 64, "mixed", "few"), (600, 72, 200, 3, 64, "packed", "few"),
    (300, 72, 5600, 3, 40, "mixed", "128"), (1100, 136, 304, 2, 64, "long", "128"), (1100, 136, 304, 20, 72, "mixed", "128"),
    (3001, 136, 2904, 2, 64, "long", "256"), (3001, 72, 2904, 5, 136, "mixed", "256"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout,route", BITS)
def test_the_adapters_term_alone(T, K, N, n, R, layout, route):
    """A base weight of zeros leaves the adapter's term: a rank-wide product of fewer bits than two bf16 terms shows
    wherever its sum over the ranks cancels."""
    say("routed adapter term", T, K, N, n, R, layout, route)
    d = rr.case(T, K, N, n, R, T + R, layout, bias=False)
    d["W"].zero_()
    assert way(T, N) == route
    rr.check(run_fwd(gpu(d)), *forward(d), "y")
    e = rr.case(T, N, K, n, R, T + R + 1, layout)  # dx: the layer of dy, with K inputs and N outputs
    e["W"].zero_()
    rr.check(run_bwd(gpu(e), want=("dx",))[0], *gradient(e), "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("small,large,N", [(200, 257, 5600), (256, 1030, 300), (1024, 1025, 200), (1000, 3001, 2904)])
def test_a_token_in_batches_of_two_sizes(small, large, N):
    """The first tokens of a batch alone and within it, on two ways: each within its bound of the definition, and so
    of one another."""
    say("routed batch sizes", small, large, N)
    assert way(small, N) != way(large, N) or ring_splits(small, 72) != ring_splits(large, 72)
    d = rr.case(large, 72, N, 7, 32, large, "mixed")
    d["W"] *= 0.05  # (the adapter's term is most of an output)
    d["W"] = d["W"].to(torch.bfloat16)
    g = gpu(d)
    first = {**g, **{k: g[k][:small] for k in ("x", "dy", "ids", "token_scale")}}
    y, bound = forward(d)
    a, b = run_fwd(first).double().cpu(), run_fwd(g)[:small].double().cpu()
    rr.check(b, y[:small], bound[:small], "in the batch")
    rr.check(a, y[:small], bound[:small], "alone")
    assert bool(((a - b).abs() <= 2 * bound[:small]).all())


# ----------------------------------------------------------------------------- infinite tokens

INFINITE = [
    (3, 72, 40, 2, 24, "mixed", "few"), (100, 72, 200, 3, 40, "mixed", "few"), (200, 9000, 72, 3, 24, "mixed", "few"),
    (300, 72, 5600, 3, 40, "mixed", "128"), (1100, 72, 304, 1, 8, "long", "128"), (1100, 1160, 304, 2, 72, "long", "128"),
    (1100, 72, 304, 20, 24, "mixed", "128"), (3001, 72, 2904, 2, 24, "long", "256"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout,route", INFINITE)
@pytest.mark.parametrize("ranks", [False, True])
def test_an_infinite_token_meets_no_padding(T, K, N, n, R, layout, route, ranks):
    """Positive weights and one infinite input: the outputs are infinite, and a NaN among them would come from the
    zeros that pad a rank (to the slot, to 8 or to 64). Ranks that are no multiples of 8 among them."""
    say("routed infinite token", T, K, N, n, R, layout, route, ranks)
    d = rr.case(T, K, N, n, R, T, layout, none=0.0)
    d["ids"] %= n
    if ranks:
        d["ranks"] = torch.tensor([R - 3 - 2 * (i % 2) for i in range(n)], dtype=torch.int32)
    live = torch.arange(R)[None, :] < (torch.full((n,), R) if d["ranks"] is None else d["ranks"])[:, None]
    for k in ("W", "A", "B"):
        d[k] = d[k].abs().clamp_min(0.01)
    d["A"], d["B"] = d["A"] * live[:, :, None], d["B"] * live[:, None, :]
    assert way(T, N) == route
    g = gpu(d)
    rows = [0, T // 2, T - 1]
    y0, dx0 = run_fwd(g), run_bwd(g, want=("dx",))[0]
    g["x"][rows, 5] = float("inf")
    g["dy"][rows, 7] = float("inf")
    y1, dx1 = run_fwd(g), run_bwd(g, want=("dx",))[0]
    rest = torch.ones(T, dtype=torch.bool)
    rest[rows] = False
    for a, b in ((y0, y1), (dx0, dx1)):
        assert torch.equal(a[rest], b[rest])
        assert bool((b[rows] == float("inf")).all()), b[rows]


# ----------------------------------------------------------------------------- parity behind the few-token kernels

# (T, K, N, n, R, layout, way of y, way of dx): ranks over a 64-rank stage, K of several stages and off them, odd
# outputs of y only where no gradient is asked for
LARGE = [
    (3001, 584, 2904, 3, 72, "long", "256", "128"), (3001, 520, 2904, 12, 136, "mixed", "256", "128"),
    (3001, 2904, 328, 3, 136, "long", "128", "256"), (3300, 2904, 200, 20, 40, "packed", "128", "256"),
    (1000, 136, 2600, 6, 40, "mixed", "128", "few"), (300, 1160, 6000, 4, 72, "packed", "128", "few"),
    (500, 5200, 264, 30, 24, "mixed", "few", "128"), (1024, 72, 2056, 1, 136, "mixed", "128", "few"),
    (1500, 1160, 72, 30, 40, "mixed", "128", "128"), (1500, 1160, 1096, 30, 136, "mixed", "128", "128"),
    (9000, 1160, 24, 12, 40, "mixed", "128", "256"), (9000, 72, 520, 40, 72, "mixed", "128", "128"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout,route,back", LARGE)
@pytest.mark.parametrize("ranks", [False, True])
def test_large_batches(T, K, N, n, R, layout, route, back, ranks):
    say("routed large", T, K, N, n, R, layout, ranks)
    assert (way(T, N), way(T, K)) == (route, back)
    d = rr.case(T, K, N, n, R, T + N + R, layout, ranks=ranks, tscale=not ranks)
    if layout == "long":
        for t in (128, 256):
            assert min(tiles(d, t)) > 0
    g = gpu(d)
    rr.check(run_fwd(g, out=torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)), *forward(d), "y")
    (_, dA, dB), (_, bA, bB) = rr.backward(d)
    got = run_bwd(g, dA=torch.full(dA.shape, float("nan"), device=DEV), dB=torch.full(dB.shape, float("nan"), device=DEV))
    for o, w, b, what in zip(got, (gradient(d)[0], dA, dB), (gradient(d)[1], bA, bB), ("dx", "dA", "dB")):
        rr.check(o, w, b, what)


@pytest.mark.parametrize("T,K,N,n,R,layout,route,back", [c for c in LARGE if c[0] > 1024 and c[3] > 8])
def test_large_batches_leave_blocks_over(T, K, N, n, R, layout, route, back):
    """The ring leaves blocks of many adapters to the 16-token form, with sums in parts (K of several splits) and
    without, below and above the 8192 tokens from which on the joins have a launch of their own."""
    for ranks in (False, True):
        assert left_over(rr.case(T, K, N, n, R, T + N + R, layout, ranks=ranks, tscale=not ranks)) > 0 or layout == "packed"
    kinds = {(c[0] > 8192, max(ring_splits(c[0], c[1]), ring_splits(c[0], c[2])) > 1) for c in LARGE
             if c[0] > 1024 and c[3] > 8 and c[5] == "mixed"}
    assert {(False, True), (True, True)} <= kinds


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n,R,layout,route", [
    (1500, 1160, 71, 30, 40, "mixed", "128"), (9000, 1160, 25, 12, 136, "mixed", "128"),
    (3001, 136, 2901, 5, 72, "mixed", "256"), (257, 72, 5501, 9, 16, "mixed", "128"),
])
def test_strides_and_odd_outputs(T, K, N, n, R, layout, route):
    """x and y as column views of wider buffers, rows of y at any 2-byte place; what lies beside and behind the
    views stays as it was."""
    say("routed large strides", T, K, N, n, R)
    assert way(T, N) == route
    d = rr.case(T, K, N, n, R, T, layout)
    g = gpu(d)
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + K] = g["x"]
    g["x"] = wide[:, 8:8 + K]
    for left, more in ((5, 9), (0, 0)):
        out = torch.full((T + 3, left + N + more), 7.0, dtype=torch.bfloat16, device=DEV)
        run_fwd(g, out=out[:T, left:left + N])
        rr.check(out[:T, left:left + N], *forward(d), "y")
        out[:T, left:left + N] = 7.0
        assert bool((out == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,route", [(400, 5600, "128"), (1200, 160, "128"), (3001, 2904, "256")])
@pytest.mark.parametrize("layout", ["mixed", "long"])
def test_routing_values_of_large_batches(T, N, route, layout):
    """Indices outside the pool, zero scales and zero ranks give the base output; a rank is cut at the slot."""
    say("routed large values", T, N, layout)
    assert way(T, N) == route
    d = rr.case(T, 128, N, 5, 24, T, layout, ranks=True)
    d["ids"][::37] = torch.tensor([5, -1, -7, 2 ** 31 - 1, -2 ** 31] * T)[: d["ids"][::37].numel()].to(torch.int32)
    d["token_scale"][1::45] = 0.0
    d["scales"][1] = 0.0
    d["ranks"][2] = 0
    d["ranks"][3] = 24
    ref = forward(d)
    g = gpu(d)
    g["ranks"][3] = 1000
    rr.check(run_fwd(g), *ref, "y")
    (_, dA, dB), (_, bA, bB) = rr.backward(d)
    for got, want, bound, what in zip(run_bwd(g), (gradient(d)[0], dA, dB), (gradient(d)[1], bA, bB), ("dx", "dA", "dB")):
        rr.check(got, want, bound, what)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,layout,route,back", [
    (300, 72, 5600, "mixed", "128", "few"), (1100, 96, 304, "mixed", "128", "128"), (1100, 96, 301, "long", "128", "128"),
    (3001, 72, 2904, "mixed", "256", "128"), (3001, 72, 2901, "long", "256", "128"),
    (3001, 2904, 72, "mixed", "128", "256"),
])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_broken_adapter_stays_with_its_tokens(T, K, N, layout, route, back, value):
    """Infinite or NaN weights of one adapter, in tiles of its own tokens and in tiles of several adapters: its own
    outputs of the columns that they reach are not finite, its other columns and all other tokens are as without."""
    say("routed large broken", T, K, N, layout, value)
    assert (way(T, N), way(T, K)) == (route, back)
    back = N % 8 == 0
    d = rr.case(T, K, N, 4, 32, 3, layout, ranks=True)
    d["ids"][:4] = torch.tensor([0, 1, 2, 1])
    d["ids"][d["ids"] == 3] = 0
    d["ranks"] = torch.tensor([8, 24, 32, 16], dtype=torch.int32)
    live = torch.arange(32)[None, :] < d["ranks"][:, None]
    d["A"], d["B"] = d["A"] * live[:, :, None], d["B"] * live[:, None, :]
    if layout == "long":
        assert min(tiles(d, 128)) > 0
    clean = gpu(d)
    y0, g0 = run_fwd(clean), run_bwd(clean) if back else None
    bad = gpu(d)
    rows = [17, N - 1]
    bad["B"][1, 17, 0] = value
    bad["B"][1, N - 1, 20] = -value
    bad["A"][3], bad["B"][3] = value, value          # (no token's)
    bad["A"][0, 8:], bad["B"][0, :, 8:] = value, value  # (behind the adapter's rank)
    y1 = run_fwd(bad)
    mine = bad["ids"] == 1
    cols = torch.ones(N, dtype=torch.bool, device=DEV)
    cols[rows] = False
    assert torch.equal(y0[~mine], y1[~mine])
    want, bound = forward(d)
    rr.check(y1[mine][:, cols], want[mine.cpu()][:, cols.cpu()], bound[mine.cpu()][:, cols.cpu()], "y, other columns")
    assert not bool(torch.isfinite(y1[mine][:, ~cols]).any())
    if back:
        g1 = run_bwd(bad)
        assert torch.equal(g0[0][~mine], g1[0][~mine])
        for a in (0, 2, 3):
            assert torch.equal(g0[1][a], g1[1][a]) and torch.equal(g0[2][a], g1[2][a])
    bad["B"][1] = clean["B"][1]
    bad["A"][1, 2, 5] = value  # and in A: every output of its tokens, and of dx the one column
    y2 = run_fwd(bad)
    assert torch.equal(y0[~mine], y2[~mine]) and not bool(torch.isfinite(y2[mine]).any())
    if back:
        dx2 = run_bwd(bad, want=("dx",))[0]
        other = torch.arange(K, device=DEV) != 5
        assert torch.equal(g0[0][~mine], dx2[~mine]) and not bool(torch.isfinite(dx2[mine][:, 5]).any())
        wx, bx = gradient(d)
        rr.check(dx2[mine][:, other], wx[mine.cpu()][:, other.cpu()], bx[mine.cpu()][:, other.cpu()], "dx, other columns")


@pytest.mark.gpu
@pytest.mark.parametrize("T,N", [(400, 5600), (1200, 200), (3001, 2904)])
def test_one_adapter_for_all_of_a_large_batch(T, N):
    """A pool of one, every tile uniform; lora_linear on the same layer, with its one bf16 term."""
    say("routed large one adapter", T, N)
    assert way(T, N) != "few"
    d = rr.case(T, 256, N, 1, 64, 5, "mixed", none=0.0, tscale=False)
    g = gpu(d)
    y1 = rg.lora_linear(g["x"], g["W"], g["b"], g["A"][0], g["B"][0], float(d["scales"][0]) * 64)
    rr.check(run_fwd(g), *forward(d), "routed")
    rr.check(y1, *rr.forward(d), "lora_linear")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,n", [(400, 128, 5600, 4), (1300, 520, 200, 20), (3001, 128, 2904, 4)])
def test_captured_large_calls_take_the_routing_of_each_replay(T, K, N, n):
    """A captured forward and backward replayed with other routing, scales and inputs in the same buffers,
    eager calls of the same layer in between: the bits of the eager calls."""
    say("routed large graph", T, K, N, n)
    assert way(T, N) != "few"
    g = gpu(rr.case(T, K, N, n, 16, T, "packed"))
    ws = torch.empty(rg.lora_linear_routed_workspace_size(T, K, N, n, 16), dtype=torch.uint8, device=DEV)
    wb = torch.empty(rg.lora_linear_routed_bwd_workspace_size(T, K, N, n, 16), dtype=torch.uint8, device=DEV)
    y, dx = torch.empty((T, N), dtype=torch.bfloat16, device=DEV), torch.empty_like(g["x"])
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
        e = gpu(rr.case(T, K, N, n, 16, 50 + k, ("packed", "mixed", "long")[k]))
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
@pytest.mark.parametrize("T,K,N", [(1300, 520, 264), (3001, 72, 2904)])
def test_two_streams_and_named_streams_of_large_calls(T, K, N):
    say("routed large streams", T, K, N)
    assert way(T, N) != "few"
    cases = [gpu(rr.case(T, K, N, 12, 24, s, "mixed")) for s in (1, 2)]
    refs = [(run_fwd(g), *run_bwd(g)) for g in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for named in (False, True, False):
        for k, (g, s) in enumerate(zip(cases, streams)):
            if named:
                got[k].append((run_fwd(g, stream=s), *run_bwd(g, stream=s)))
            else:
                with torch.cuda.stream(s):
                    got[k].append((run_fwd(g), *run_bwd(g)))
    torch.cuda.synchronize()
    for ref, outs in zip(refs, got):
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, ref))


@pytest.mark.gpu
def test_a_large_batch_on_a_pool_beyond_32_bit_offsets():
    """The last slots of pools of 4.4 GB, in tiles of one adapter and of two."""
    say("routed large batch, large pool")
    T, n, R, K, N = 1100, 8192, 256, 1040, 1048
    d = rr.case(T, K, N, 2, R, 1, "long", none=0.0)
    assert way(T, N) == "128" and min(tiles(d, 128)) > 0 and n * R * K * 2 > 1 << 32
    g = gpu(d)
    Ap = torch.zeros((n, R, K), dtype=torch.bfloat16, device=DEV)
    Bp = torch.zeros((n, N, R), dtype=torch.bfloat16, device=DEV)
    Ap[-2:], Bp[-2:] = g["A"], g["B"]
    sc = torch.ones(n, device=DEV)
    sc[-2:] = g["scales"]
    ids = torch.where(g["ids"] < 0, -1, g["ids"] + (n - 2)).to(torch.int32)
    y = rg.lora_linear_routed(g["x"], g["W"], g["b"], Ap, Bp, sc, ids, token_scale=g["token_scale"])
    rr.check(y, *forward(d), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("want", [("dx",), ("dx", "dA")])
def test_transposed_copies_of_several_launches(want):
    """A pool of 17 GB whose copies take more than 2^24 tiles of 64 x 64, the threads of one launch; with dA the
    plan goes before them."""
    say("routed copies of several launches", want)
    T, n, R, K, N = 40, 8192, 8, 1 << 17, 8
    slots = torch.tensor([0, 5000, n - 1], dtype=torch.int32)
    d = rr.case(T, K, N, 3, R, 2, "mixed")
    g = gpu(d)
    Ap = torch.zeros((n, R, K), dtype=torch.bfloat16, device=DEV)
    Bp = torch.zeros((n, N, R), dtype=torch.bfloat16, device=DEV)
    sc = torch.ones(n, device=DEV)
    at = slots.to(DEV).long()
    Ap[at], Bp[at], sc[at] = g["A"], g["B"], g["scales"]
    ids = torch.where(d["ids"] < 0, -1, slots[d["ids"].clamp_min(0).long()]).to(torch.int32).to(DEV)
    dx, dA, _ = rg.lora_linear_routed_backward(g["x"], g["W"], Ap, Bp, g["dy"], sc, ids, token_scale=g["token_scale"],
                                               want=want)
    rr.check(dx, *gradient(d), "dx")
    if dA is not None:
        rr.check(dA[at], rr.backward(d)[0][1], rr.backward(d)[1][1], "dA")
        dA[at] = 0
        assert all(not bool(part.any()) for part in dA.split(512))

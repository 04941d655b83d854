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

"""The operators of a fine-tuning step at the sizes of a full batch: what lies behind the largest adapters, the larger
output tiles, tiles cut along the contraction, several pieces of a vocabulary."""
import math
import os
import shutil
import subprocess

import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import step_ref as sr
from tests import test_loss as tl
from tests import test_step as ts

BF, DEV = torch.bfloat16, "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
say = ts.say


# ----------------------------------------------------------------------------- plans (no GPU)

def plans(tmp_path, lines):
    """What the sources' own rules say to "ring T N stages" (tile, tiles, whole ones, parts of the others, their stages)
    and "loss T K V" (columns of a piece, of the last one, logits' tile, then dh's as above)."""
    if shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")):
        pytest.skip("needs g++ and the ROCm headers")
    src, exe = tmp_path / "plans.cpp", str(tmp_path / "plans")
    src.write_text("""
#include <cstdio>
#include "loss.hpp"
int main() {
  char what[8];
  long a, b, c;
  while (std::scanf("%7s %ld %ld %ld", what, &a, &b, &c) == 4) {
    lora::RingPlan p;
    if (what[0] == 'l') {
      const long piece = lora::loss_piece(a, c);
      p = lora::loss_plan(a, b, c);
      std::printf("%ld %ld %d ", piece, c - (c - 1) / piece * piece,
                  lora::ring_plan(a, piece < c ? piece : c, (b + 63) / 64).big ? 256 : 128);
    } else {
      p = lora::ring_plan(a, b, c);
    }
    std::printf("%d %ld %ld %d %d\\n", p.big ? 256 : 128, (long)p.tiles, (long)p.full, p.S, p.ks);
  }
}
""")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"), "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "rank_gemm_lora_amd", "csrc"), str(src), "-o", exe],
                   check=True)
    out = subprocess.run([exe], input="\n".join(lines), text=True, capture_output=True, check=True).stdout
    return [tuple(int(v) for v in line.split()) for line in out.splitlines()]


@pytest.mark.parametrize("T,V", [(4096, 128017), (4194, 128017), (4352, 128017), (9000, 60000), (33000, 50257), (140000, 9000),
                                 (2000000, 4097), (1, 1 << 24)])
def test_pieces_of_a_vocabulary_are_alike(tmp_path, T, V):
    """As few pieces as 2^29 shares each (or 4096 columns) make, and none narrower than the others but for its last 256."""
    piece, last = plans(tmp_path, [f"loss {T} 512 {V}"])[0][:2]
    most = min(max((1 << 29) // T // 256 * 256, 4096), 1 << 19)
    n = -(-V // piece)
    assert piece % 256 == 0 and piece <= most and n == -(-V // most)
    assert last > piece - 256 * n


@pytest.mark.parametrize("T", [4096, 4194, 4352, 8192, 8448, 9000, 32768, 33000, 131072, 200000])
def test_workspace_of_the_loss_does_not_jump_between_rounds_of_tiles(T):
    """On both sides of a full round of tiles: the shares (1 GiB, or 4096 columns), a power of two, a sum and a shift per
    token and 64 columns, the sums of dh once, and beside them those of cut tiles, at most seven rounds of 256."""
    for K, V in ((4096, 128017), (1536, 128017), (5120, 50257)):
        sums = -(-T // 256) * -(-K // 256) * 256 * 256 * 4 + 7 * 256 * 256 * 256 * 4
        blocks = (-(-V // 128) * 2) * (T * 8 + T + 256)
        assert rg.lora_cross_entropy_workspace_size(T, K, V) <= max(1 << 30, 8192 * T) + blocks + T * 24 + 4096 + sums


# ----------------------------------------------------------------------------- zeros


@pytest.mark.gpu
def test_zeros_behind_the_second_term_of_an_adapter_of_two_gigabytes():
    """dx where A has more than 2^30 bytes: the columns behind the second term of u (2032 used of 2048) meet zeros, not a
    row of A from 2^30 bytes further on, so an infinity in one column of A reaches that column of dx alone.

    2^30 bytes are 512 rows of 2^20 - 8 inputs and 4096 columns: the infinities at rows 512 to 519 of a column would meet
    the zeros of u 4096 columns before it."""
    K, R, N, T, col = (1 << 20) - 8, 1016, 8, 3, 4196
    say("wide adapter")
    g = ts.gen(41)
    x, dy = torch.zeros(T, K, dtype=BF, device=DEV), ts.rand(g, (T, N)).to(DEV)
    W = torch.randn(N, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(41)).to(BF)
    A, B = torch.zeros(R, K, dtype=BF, device=DEV), ts.rand(g, (N, R), 0.15).to(DEV)
    dx = lambda: rg.lora_linear_dropout_backward(x, W, A, B, dy, 16.0, 0.1, 1, want=("dx",))[0]  # noqa: E731
    clean = dx()
    A[512:520, col] = math.inf
    got = dx()
    rest = torch.arange(K, device=DEV) != col
    assert bool(torch.isfinite(clean).all())
    assert torch.equal(got[:, rest], clean[:, rest])


# ----------------------------------------------------------------------------- the loss

# ((T, K, V), its plan)
LOSS = [
    # the larger tile of dh, whole behind both tiles of the logits, and cut
    ((8200, 904, 200), (256, 200, 128, 256, 132, 132, 1, 4)),
    ((8200, 904, 904), (1024, 904, 256, 256, 132, 132, 1, 15)),
    ((7300, 2200, 832), (1024, 832, 128, 256, 261, 256, 4, 4)),
    ((4352, 4096, 2600), (2816, 2600, 256, 256, 272, 256, 6, 7)),
    # several pieces: whole tiles with sums in memory, alone and beside cut ones; all cut
    ((16384, 1024, 33000), (16640, 16360, 256, 256, 256, 256, 1, 260)),
    ((16500, 1032, 33000), (16640, 16360, 256, 256, 325, 256, 3, 87)),
    ((2500, 512, 215000), (107520, 107480, 256, 256, 20, 0, 12, 140)),
    # the smaller tile, and a last piece of so few columns that some parts have none
    ((8300, 520, 65000), (32512, 32488, 256, 128, 325, 0, 3, 170)),
    ((131100, 64, 128017), (4096, 1041, 256, 128, 1025, 1024, 16, 4)),
]
LOSS_ALONE = ((900, 128, 8200), 256)  # (the logits' tile over the whole vocabulary)


def test_plans_of_the_loss(tmp_path):
    assert plans(tmp_path, ["loss %d %d %d" % c for c, _ in LOSS]) == [p for _, p in LOSS]
    T, K, V = LOSS_ALONE[0]
    assert plans(tmp_path, [f"ring {T} {V} {stages(K, 0)}"])[0][0] == LOSS_ALONE[1]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,V", [c for c, _ in LOSS])
def test_loss_with_larger_tiles_and_several_pieces(T, K, V):
    say("loss tiles", T, K, V)
    c = tl.case(T, K, V, 42)
    got = tl.run(c)
    # (rows of the first tiles, of a middle one and of the last, which are the cut ones)
    rows = torch.cat((torch.arange(0, 20), torch.arange(T // 2, T // 2 + 20), torch.arange(T - 60, T)))
    say("reference")
    tl.check({k: v[rows] for k, v in got.items()}, tl.reference(c, rows))
    for k, v in got.items():
        assert bool(torch.isfinite(v).all()), k


# ----------------------------------------------------------------------------- larger tiles of the layers

def stages(K, R):
    """Stages of 64 of a contraction of K behind adapters of R columns in two terms."""
    return -(-K // 64) + -(-2 * R // 64)


# (T, K, F, ranks, activation), the forward's plan, dx's
WHOLE = (256, 132, 132, 1)
GATED = [((900, 64, 4100, 16, 0, act), WHOLE, None) for act in ("silu", "gelu", "gelu_tanh")]  # (F of no multiple of 8)
GATED += [((2200, 704, 3656, 24, 16, act), (256, 261, 256, 4), None) for act in ("silu", "gelu", "gelu_tanh")]
GATED += [((8200, 904, 72, 16, 8, "gelu"), None, WHOLE), ((7300, 2200, 328, 8, 24, "silu"), None, (256, 261, 256, 4)),
          ((7300, 2200, 264, 0, 72, "gelu_tanh"), None, (256, 261, 256, 4))]
# (T, K, N, rank, p), the forward's plan, dx's. At rank 136 the extension is five stages of dx: its first part (of four
# stages) ends before the base stages, and the second part has the mask between its first stage and the others.
DROP = [((8200, 200, 904, 16, 0.1), WHOLE, None), ((7300, 768, 2200, 16, 0.1), (256, 261, 256, 4), None)]
DROP += [((8200, 904, 200, 16, p), None, WHOLE) for p in (0.1, 0.0)]
DROP += [((7300, 2200, 512, 136, p), None, (256, 261, 256, 4)) for p in (0.1, 0.0)]
DROP += [((7300, 2200, 768, 16, 0.1), None, (256, 261, 256, 4))]


def test_plans_of_the_layers(tmp_path):
    lines, want = [], []
    for (T, K, F, rg_, ru, _), fwd, bwd in GATED:
        R = rg_ + ru
        for plan, line in ((fwd, (T, 2 * F, stages(K, R))), (bwd, (T, K, 2 * stages(F, 0) + stages(0, R)))):
            if plan is not None:
                lines.append("ring %d %d %d" % line)
                want.append(plan)
    for (T, K, N, R, _), fwd, bwd in DROP:
        for plan, line in ((fwd, (T, N, stages(K, R))), (bwd, (T, K, stages(N, R)))):
            if plan is not None:
                lines.append("ring %d %d %d" % line)
                want.append(plan)
    got = plans(tmp_path, lines)
    assert [p[:4] for p in got] == want
    assert all(p[4] == 4 for p in got if p[3] == 4)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,F,rg_,ru,act", [c for c, _, _ in GATED])
def test_gated_with_larger_tiles(T, K, F, rg_, ru, act):
    """Every output whole, from g and u that the larger tile kept."""
    say("gated tiles", T, K, F, rg_, ru, act)
    c = ts.gated_case(T, K, F, rg_, ru, 43)
    backward = F % 8 == 0
    got = ts.run_gated(c, act, torch.float32, backward=backward)
    say("reference")
    want = ts.want_gated(c, act, backward=backward)
    assert set(got) == set(want)
    for k, t in got.items():
        sr.check(t, want[k], BF if k in ("h", "dx") else torch.float32, k)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,R,p", [c for c, _, _ in DROP])
def test_dropout_with_larger_tiles(T, K, N, R, p):
    say("dropout tiles", T, K, N, R, p)
    c = ts.drop_case(T, K, N, R, 44)
    how = dict(alpha=1.0 * R, p=p, seed=21, offset=4)
    got = ts.run_drop(c, torch.float32, **how)
    say("reference")
    want = sr.dropout(c["x"], c["W"], c["b"], c["A"], c["B"], 1.0 * R, p, 21, 4, dy=c["dy"])
    ts.check_drop(got, want, torch.float32, "tiles")


@pytest.mark.gpu
def test_loss_alone_with_larger_tiles():
    """The loss without its gradient: 256 x 256 tiles of logits, ragged on both sides."""
    T, K, V = LOSS_ALONE[0]
    say("loss alone", T, K, V)
    c = tl.case(T, K, V, 45)
    got = tl.run(c, want=("loss", "lse"))
    assert got.pop("dh") is None
    tl.check(got, tl.reference(c))


# ----------------------------------------------------------------------------- the largest extents

MOST_T, MOST_K = (1 << 21) - 1, 1 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,R", [(MOST_T, 8, 8, 8), (2, 8, MOST_K, 16), (2, MOST_K, 8, 16)])
def test_dropout_at_the_largest_extents(T, K, N, R):
    say("dropout extents", T, K, N, R)
    c = ts.drop_case(T, K, N, R, 46)
    got = ts.run_drop(c, torch.float32, alpha=1.0 * R, p=0.1, seed=1 << 63, offset=(1 << 64) - 1)
    say("reference")
    want = sr.dropout(c["x"], c["W"], c["b"], c["A"], c["B"], 1.0 * R, 0.1, 1 << 63, (1 << 64) - 1, dy=c["dy"])
    ts.check_drop(got, want, torch.float32, "extents")


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,F", [(MOST_T, 8, 8), (3, 8, MOST_K), (3, MOST_K, 8)])
def test_gated_at_the_largest_extents(T, K, F):
    say("gated extents", T, K, F)
    c = ts.gated_case(T, K, F, 16, 8, 47)
    got = ts.run_gated(c, "silu", torch.float32, save=T > 3)
    say("reference")
    want = ts.want_gated(c, "silu")
    for k, t in got.items():
        sr.check(t, want[k], BF if k in ("h", "dx") else torch.float32, k)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,V", [(MOST_T, 8, 9), (1, 8, 1 << 24), (2, MOST_K, 9)])
def test_loss_at_the_largest_extents(T, K, V):
    say("loss extents", T, K, V)
    c = tl.case(T, K, V, 48)
    got = tl.run(c)
    say("reference")
    tl.check(got, tl.reference(c))

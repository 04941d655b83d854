"""The operators of a fine-tuning step at the sizes of a full batch: what lies behind the largest adapters, the larger
output tiles, tiles cut along the contraction, several pieces of a vocabulary."""
import math
import os
import shutil
import subprocess

import pytest
import torch

import rank_gemm_lora_amd as rg
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
    # several pieces: whole tiles with sums in memory, alone and beside cut ones; all cut
    ((16384, 1024, 33000), (16640, 16360, 256, 256, 256, 256, 1, 260)),
    ((16500, 1032, 33000), (16640, 16360, 256, 256, 325, 256, 3, 87)),
    ((2500, 512, 215000), (107520, 107480, 256, 256, 20, 0, 12, 140)),
    # the smaller tile, and a last piece of so few columns that some parts have none
    ((8300, 520, 65000), (32512, 32488, 256, 128, 325, 0, 3, 170)),
    ((131100, 64, 128017), (4096, 1041, 256, 128, 1025, 1024, 16, 4)),
]


def test_plans_of_the_loss(tmp_path):
    assert plans(tmp_path, ["loss %d %d %d" % c for c, _ in LOSS]) == [p for _, p in LOSS]


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

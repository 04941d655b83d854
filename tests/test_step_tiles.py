"""The operators of a fine-tuning step at the sizes of a full batch: what lies behind the largest adapters, the larger
output tiles, tiles cut along the contraction, several pieces of a vocabulary."""
import math

import pytest
import torch

import rank_gemm_lora_amd as rg
from tests import test_step as ts

BF, DEV = torch.bfloat16, "cuda:0"
say = ts.say


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

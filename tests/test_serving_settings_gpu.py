"""Sampling with settings at the ends of what a row may be given."""

import math

import pytest
import torch

from test_serving_gpu import BF16, F16, F32, run_sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("vocab", [100, 3000, 70000, 140000])
def test_temperatures_that_are_not_above_zero(dtype, vocab):
    """-1, -0, NaN and -inf count as 0: equal weights of the largest logits, by
    bins, in tiles and by digits (a row of ties, one with infinite logits)."""
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(6, vocab, generator=g) * 2.5).to(dtype)
    x[1, vocab // 3] = x[1, vocab // 2] = 20.0
    x[2] = 1.0
    x[3, 7] = x[3, 50] = math.inf
    x[4, ::2] = -math.inf
    x[5] = torch.randint(0, 3, (vocab,), generator=g).to(dtype)
    u = [0.3, 0.7, 0.9, 0.6, 0.1, 0.5]
    for t in (-1.0, -0.0, math.nan, -math.inf, -1e-30):
        bad = torch.full((6,), t)
        for settings in ({}, {"p": [0.5, 0.9, 0.3, 0.8, 0.01, 0.6]}, {"k": [1, 2, 50, 1, 7, 90]}, {"m": [0.1] * 6},
                         {"p": [0.9] * 6, "k": [5, 1, 40, 2, 3, vocab // 2], "m": [0.5] * 6}):
            run_sample_as(x, u, bad, [0.0] * 6, settings)


def run_sample_as(x, u, given, meant, settings):
    """run_sample with one temperature given and another one meant."""
    import nvfp4_quantized_matmul_amd as nv
    real = nv.sample
    try:
        nv.sample = lambda *a, temperature=None, **k: real(*a, temperature=given.to(temperature.device), **k)
        run_sample(x, u, meant, **settings)
    finally:
        nv.sample = real

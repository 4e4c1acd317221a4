"""Attention's weights at the ends of their range.  Tolerances are those of
test_serving_gpu.py unless a test says otherwise."""

import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded
from test_serving_gpu import BF16, E4M3, F16, F32, make_cache, paging, to_gpu

pytestmark = pytest.mark.gpu


def state(seed, dtype, n, count, dim=64, page=64, hq=2):
    """One sequence of n tokens, the last `count` of them new, of one kv head; value scales 1."""
    g = torch.Generator().manual_seed(seed)
    table, pages = paging(g, [n], page)
    return (torch.randn(count, hq, dim, generator=g) * 0.5).to(dtype), make_cache(g, pages, 1, page, dim, 0), table


def one_hot(q, cache):
    """A score is channel 0's code of the key, and these are 0 at first."""
    q.zero_()
    q[..., 0] = 1
    cache[0].zero_()


def attention(q, cache, table, n, scale):
    out, guard = guarded(q.shape, q.dtype)
    print("attention", q.dtype, tuple(q.shape), n, scale, flush=True)
    got = nv.paged_attention(q.to(DEV), to_gpu(cache), table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                             cu_q=torch.tensor([0, q.shape[0]], dtype=torch.int32, device=DEV), scale=scale, out=out)
    guard()
    return got.double().cpu()


# 1 and 40 new tokens: few rows and many
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("count", [1, 40])
@pytest.mark.parametrize("power", [8, 16, 18, 19, 20, 21, 24, 28, 32, 60])
def test_scores_of_any_size(dtype, count, power):
    """Two tokens share the largest score, far above the others': the mean of
    their values.  Their weights are equal, so each is off by its own rounding
    and the sums by a few of 32 bits."""
    n = 400
    for at in (0, 133):
        q, cache, table = state(6, dtype, n, count)
        one_hot(q, cache)
        k, v = cache[0], cache[1]
        for i in table[0]:
            k[int(i), 0, :, 0] = 0x7d                     # 416
        for t in (at, at + 64):
            k[int(table[0, t // 64]), 0, t % 64, 0] = 0x7e    # 448
        got = attention(q, cache, table, n, 2.0 ** power)
        a, b = (E4M3[v[int(table[0, t // 64]), 0, :, t % 64].long()] for t in (at, at + 64))
        h = torch.finfo(dtype).eps / 2
        weights = h if dtype != F32 else 0.0
        tol = h * (a + b).abs() / 2 + (weights * (1 + h) + 2.0 ** -20) * (a.abs() + b.abs()) / 2
        assert ((got - (a + b) / 2).abs() <= tol).all()
        assert attention(-q, cache, table, n, 2.0 ** power).isfinite().all()

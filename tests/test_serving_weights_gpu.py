"""Attention's weights at the ends of their range.

Tolerances are those of test_serving_gpu.py, and of f16 weights one more: in
units of the values' codes, weights below 2^-25 of the largest are off by at
most 2^-36 of that one."""

import math

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


def check(q, cache, table, n, scale):
    """Against 64 bits; returns the exact output."""
    got = attention(q, cache, table, n, scale)
    k, v, ks, vs = cache
    page, dim = k.shape[2:]
    ids, h = table[0].long(), torch.finfo(q.dtype).eps / 2
    at, t = torch.arange(n - q.shape[0], n), torch.arange(n)
    kk = (E4M3[k[ids, 0].long()] * torch.exp2(ks[ids, 0].double() - 127)[:, None, None]).reshape(-1, dim)[:n]
    codes = E4M3[v[ids, 0].long()].transpose(1, 2).reshape(-1, dim)[:n]
    scales = torch.exp2(vs[ids, 0].double() - 127).repeat_interleave(page)[:n]
    scale = float(np.float32(scale))
    for j in range(q.shape[1]):
        x = q[:, j].double()
        s = torch.where(t <= at[:, None], x @ kk.T * scale, -math.inf)
        size = (x.abs() @ kk.abs().T * scale).amax(1, keepdim=True)
        units = torch.softmax(s, 1) * scales
        ref, amount = units @ codes, units @ codes.abs()
        rel = 2.0 ** -24 * (2 * ((dim + 8) * size + 6 * size + 16) + n + 16)
        tol = h * ref.abs() + rel * amount + torch.finfo(q.dtype).smallest_normal * h
        if q.dtype != F32:
            tol = tol + h * (1 + h) * amount
        if q.dtype == F16:
            tol = tol + 2.0 ** -36 * units.amax(1, keepdim=True) * codes.abs().sum(0)
        assert got[:, j].isfinite().all()
        err = (got[:, j] - ref).abs() - tol
        assert err.max() <= 0, (j, float(err.max()), float((got[:, j] - ref).abs().max()), float(ref.abs().max()))
    return ref


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


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("count", [1, 40])
@pytest.mark.parametrize("code,nats", [(0x58, 14.0), (0x58, 17.5), (0x58, 20.0)])
def test_many_small_weights_beside_a_large_one(dtype, count, code, nats):
    """One token of zeros `nats` above 20000 others: the output is the others'."""
    n = 20000
    q, cache, table = state(2, dtype, n, count)
    one_hot(q, cache)
    first = int(table[0, 0])
    cache[0][first, 0, 0, 0] = code                       # 16
    cache[1][first, 0, :, 0] = 0
    assert check(q, cache, table, n, nats / 16).abs().max() > 1e-7


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("count", [1, 40])
@pytest.mark.parametrize("exponent", [8, 20, 26])
def test_a_page_with_a_value_scale_far_above_the_others(dtype, count, exponent):
    """Equal weights; the loud page is loud in one channel only, the others are not lost."""
    n = 1000
    q, cache, table = state(3, dtype, n, count)
    one_hot(q, cache)
    v, vs = cache[1], cache[3]
    loud = int(table[0, 1])
    vs[loud] = 127 + exponent
    v[loud] = 0
    v[loud, 0, 5] = 0x01                                  # 2^-9
    check(q, cache, table, n, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("count", [1, 40])
@pytest.mark.parametrize("exponent", [-110, -61, -60, 60, 61, 100])
def test_value_scales_at_the_ends(dtype, count, exponent):
    """All pages at the scale, and one of zeros whose byte is 0."""
    n = 300
    q, cache, table = state(4, dtype, n, count)
    cache[3].fill_(127 + exponent)
    zeros = int(table[0, 2])
    cache[1][zeros], cache[3][zeros] = 0, 0
    check(q, cache, table, n, 0.125)


@pytest.mark.parametrize("count", [1, 40])
@pytest.mark.parametrize("exponent", [16, 60, 61, 76, 100, 128])
def test_f16_zeros_at_a_scale_past_f16(count, exponent):
    """A float32 model's page may have such a scale; its zeros are no NaN."""
    q, cache, table = state(5, F16, 300, count)
    one_hot(q, cache)
    loud = int(table[0, 1])
    cache[1][loud], cache[3][loud] = 0, 127 + exponent
    check(q, cache, table, 300, 1.0)


@pytest.mark.parametrize("count", [1, 40])
def test_f16_scores_that_grow_along_the_row(count):
    """Each tile's largest score passes the one before, by less and by more
    than the reference waits for."""
    n = 640
    for step in (1.0, 4.0, 9.0, 12.0):
        q, cache, table = state(7, F16, n, count)
        one_hot(q, cache)
        for i, page in enumerate(table[0]):
            cache[0][int(page), 0, :, 0] = torch.tensor([0, 0x38, 0x40, 0x44, 0x48, 0x4a, 0x4c, 0x4e, 0x50, 0x51])[i]
        check(q, cache, table, n, step)

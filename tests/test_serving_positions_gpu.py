"""Positions, windows and bounds at their ends: lengths past the table and near
the end of int32, windows around the table's size, bounds below the new tokens.
Tolerances are those of test_serving_gpu.py."""

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded
from test_serving_gpu import BF16, E4M3, F16, F32, check_attention, make_cache, paging, to_gpu

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reference(q, cache, table, lens, cu, window, scale):
    """As test_serving_gpu.reference_attention, with lengths past the table."""
    k, v, ks, vs = cache
    pages, heads, page, dim = k.shape
    group, width = q.shape[1] // heads, table.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    amount, rel = torch.zeros_like(out), torch.zeros(q.shape[:2], dtype=torch.float64)
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        ids = table[b].long()
        there = ((ids >= 0) & (ids < pages)).repeat_interleave(page)
        ids = ids.clamp(0, pages - 1)
        pos, t = torch.arange(n - (hi - lo), n), torch.arange(width * page)
        see = (t <= pos[:, None]) & there
        if window > 0:
            see &= t > pos[:, None] - window
        for h in range(heads):
            kk = (E4M3[k[ids, h].long()] * torch.exp2(ks[ids, h].double() - 127)[:, None, None]).reshape(-1, dim)
            vv = E4M3[v[ids, h].long()] * torch.exp2(vs[ids, h].double() - 127)[:, None, None]
            vv = vv.transpose(1, 2).reshape(-1, dim)
            for j in range(h * group, (h + 1) * group):
                x = q[lo:hi, j].double()
                s = torch.where(see, x @ kk.T * scale, -torch.inf)
                size = torch.where(see, x.abs() @ kk.abs().T * scale, 0.0).amax(1)
                p = torch.where(see, torch.exp(s - s.amax(1, keepdim=True).clamp_min(-1e300)), 0.0)
                p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
                out[lo:hi, j], amount[lo:hi, j] = p @ vv, p @ vv.abs()
                rel[lo:hi, j] = 2.0 ** -24 * (2 * ((dim + 8) * size + 6 * size + 16) + width * page + 16)
    return out, amount, rel


def run(seed, dtype, hq, hkv, dim, page, width, lens, counts, window):
    g = torch.Generator().manual_seed(seed)
    table, pages = paging(g, [width * page] * len(lens), page)
    cache = make_cache(g, pages, hkv, page, dim)
    cu = [0] + [int(c) for c in np.cumsum(counts)]
    q = (torch.randn(cu[-1], hq, dim, generator=g) * 0.5).to(dtype)
    out, guard = guarded(q.shape, dtype)
    print("attention", dtype, hq, hkv, dim, page, width, lens, counts, window, flush=True)
    got = nv.paged_attention(q.to(DEV), to_gpu(cache), table.to(DEV), i32(lens), cu_q=i32(cu), max_q=max(counts),
                             window=window, out=out)
    guard()
    check_attention(got, *reference(q, cache, table, lens, cu, window, dim ** -0.5), dtype)
    return got


END = 2 ** 31 - 1


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("count", [1, 5, 40])
@pytest.mark.parametrize("window", [0, 1, 63, 100])
def test_lengths_at_the_end_of_int32(dtype, count, window):
    """Windows far behind the table see nothing; without one all of it is seen."""
    got = run(1, dtype, 4, 2, 64, 32, 4, [END, END - 63, END - 64, END - 200, 130], [count] * 5, window)
    assert window == 0 or (got[:4 * count] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths_at_the_end_of_int32_over_a_split_axis(dtype):
    got = run(2, dtype, 4, 1, 64, 64, 100, [END, END - 100], [1, 1], 5000)
    assert (got == 0).all()


@pytest.mark.parametrize("dtype,hq,count", [(BF16, 4, 1), (F16, 2, 40), (F32, 2, 5)])
@pytest.mark.parametrize("window", [1, 100, 127, 128, 129, 150, 200, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
def test_windows_around_the_table(dtype, hq, count, window):
    """A table of 128 tokens; lengths inside it, a little past it, and past it
    by as much as the windows and more."""
    run(3, dtype, hq, 1, 64, 32, 4, [100, 128, 129, 170, 228, 327, 400], [count] * 7, window)


@pytest.mark.parametrize("dtype,hq,count", [(BF16, 4, 1), (F16, 4, 40), (F32, 2, 3)])
@pytest.mark.parametrize("window", [3000, 6400, 6500])
def test_windows_around_a_split_table(dtype, hq, count, window):
    run(4, dtype, hq, 1, 64, 64, 100, [6300, 7000, 9500, 13000], [count] * 4, window)

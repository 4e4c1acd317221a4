"""Positions, windows and bounds at their ends: lengths past the table and near
the end of int32, windows around the table's size, bounds below the new tokens.
Tolerances are those of test_serving_gpu.py."""

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded
from test_serving_gpu import BF16, E4M3, F16, F32, check_attention, make_cache, paging, run_append, to_gpu

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


@pytest.mark.parametrize("dtype,hq,hkv,dim,page,firsts,counts,rot,interleaved", [
    (BF16, 4, 2, 64, 16, [5, 0, 9, 30, 15, 16, 7, 0, 1], [300, 1, 0, 17, 40, 0, 64, 3, 2], 64, False),
    (F32, 2, 1, 64, 16, [0] * 6 + [15], [1, 1, 1, 1, 1, 1, 200], 32, True),
    (F16, 3, 3, 128, 32, [31, 0, 0, 0, 100, 0, 0, 3], [0, 0, 500, 0, 1, 0, 0, 0], 128, False)])
@pytest.mark.parametrize("bound", [True, False])
def test_append_of_ragged_sequences(dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved, bound, monkeypatch):
    """One long sequence among short and empty ones, with and without a bound of their new tokens."""
    real = nv.kv_append
    if not bound:
        monkeypatch.setattr(nv, "kv_append", lambda *a, max_q=None, **k: real(*a, **k))
    run_append(21, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved)


def test_append_without_a_bound_of_many_tokens():
    """64 ragged prompts of 131072 tokens together, in pages of 16 and 16 heads:
    a block for each page that each of them might have would be 16.8 million."""
    g = torch.Generator().manual_seed(8)
    batch, tokens, heads, page, dim = 64, 131072, 16, 16, 64
    ends = torch.cat((torch.randint(0, tokens + 1, (batch - 1,), generator=g).sort().values, torch.tensor([tokens])))
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), ends))
    counts = cu[1:] - cu[:-1]
    firsts = torch.randint(0, 40, (batch,), generator=g)
    lens = firsts + counts
    need = -(-lens // page)
    table = torch.full((batch, int(need.max())), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    k = torch.randn(tokens, heads, dim, device=DEV).to(BF16)
    v = torch.randn(tokens, heads, dim, device=DEV).to(BF16)
    print("append", batch, tokens, heads, page, dim, flush=True)
    a, b = nv.KVCache.empty(at, heads, page, dim), nv.KVCache.empty(at, heads, page, dim)
    nv.kv_append(k, v, a, table.to(DEV), i32(lens.tolist()), cu_q=i32(cu.tolist()))
    nv.kv_append(k, v, b, table.to(DEV), i32(lens.tolist()), cu_q=i32(cu.tolist()), max_q=int(counts.max()))
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(x, y)
    # every new token is there: the values' codes against the definition
    seq = torch.searchsorted(cu[1:], torch.arange(tokens), right=True)
    pos = torch.arange(tokens) - cu[seq] + firsts[seq]
    pid = table[seq, pos // page].long().to(DEV)
    codes = a.v[pid, :, :, (pos % page).to(DEV)]
    scale = torch.exp2(a.v_scales[pid].double() - 127)[..., None]
    got = E4M3.to(DEV)[codes.int()] * scale
    assert ((got - v.double()).abs() <= torch.maximum(2.0 ** -4 * v.double().abs(), 2.0 ** -10 * scale)).all()


# few rows and many, one split, up to 16 (one wave joins) and more (four)
@pytest.mark.parametrize("dtype,hq,hkv,page,lens,counts,max_q", [
    (BF16, 4, 2, 32, [90, 40], [9, 3], 4), (F32, 4, 2, 32, [90, 40], [9, 3], 4), (F16, 2, 2, 64, [500, 300], [300, 50], 70),
    (BF16, 4, 1, 64, [6000, 5000], [9, 3], 4), (F32, 4, 1, 64, [6000, 5000], [9, 3], 4),
    (BF16, 4, 1, 64, [30000, 5000], [9, 3], 4), (F16, 2, 2, 64, [6000, 5000], [300, 50], 70),
    (F16, 1, 1, 64, [20000], [300], 70), (BF16, 4, 1, 64, [6000, 100], [64, 1], 1)])
def test_attention_leaves_out_rows_past_max_q(dtype, hq, hkv, page, lens, counts, max_q):
    g = torch.Generator().manual_seed(5)
    table, pages = paging(g, lens, page)
    cache = make_cache(g, pages, hkv, page, 64)
    cu = [0] + [int(c) for c in np.cumsum(counts)]
    q = (torch.randn(cu[-1], hq, 64, generator=g) * 0.5).to(dtype)
    out, guard = guarded(q.shape, dtype, fill=7.0)
    print("attention", dtype, hq, hkv, page, lens, counts, max_q, flush=True)
    # what a split axis leaves unwritten of its workspace is not to be found in the output: NaN
    junk = torch.full((1 << 24,), float("nan"), device=DEV)
    del junk
    nv.paged_attention(q.to(DEV), to_gpu(cache), table.to(DEV), i32(lens), cu_q=i32(cu), max_q=max_q, out=out)
    guard()
    ref = reference(q, cache, table, lens, cu, 0, 64 ** -0.5)
    taken = torch.cat([torch.arange(n) < max_q for n in counts])
    check_attention(out.cpu()[taken], *[r[taken] for r in ref], dtype)
    assert (out.cpu()[~taken] == 7.0).all()


@pytest.mark.parametrize("dtype,page,firsts,counts,max_q", [
    (BF16, 16, [5, 0, 30], [40, 3, 20], 10), (F32, 64, [60, 0], [10, 130], 4), (F16, 32, [0, 31], [600, 700], 65),
    (F32, 16, [0], [33], 16)])
def test_append_leaves_out_tokens_past_max_q(dtype, page, firsts, counts, max_q):
    """The same cache and queries as an append of the first max_q tokens alone."""
    g = torch.Generator().manual_seed(6)
    lens = [f + n for f, n in zip(firsts, counts)]
    table, pages = paging(g, lens, page)
    base = make_cache(g, pages, 2, page, 64, 2)
    cu = [0] + [int(c) for c in np.cumsum(counts)]
    q, k, v = ((torch.randn(cu[-1], h, 64, generator=g)).to(dtype).to(DEV) for h in (4, 2, 2))
    inv = (10000.0 ** (-torch.arange(0, 64, 2).float() / 64)).to(DEV)
    taken = torch.cat([torch.arange(n) < max_q for n in counts])
    print("append", dtype, page, firsts, counts, max_q, flush=True)
    out, guard = guarded(q.shape, dtype, fill=7.0)
    a, b = to_gpu([t.clone() for t in base]), to_gpu([t.clone() for t in base])
    nv.kv_append(k, v, a, table.to(DEV), i32(lens), q=q, cu_q=i32(cu), max_q=max_q, inv_freq=inv, out=out)
    guard()
    short = [min(n, max_q) for n in counts]
    rows = taken.nonzero()[:, 0].to(DEV)
    want = nv.kv_append(k[rows], v[rows], b, table.to(DEV), i32([f + n for f, n in zip(firsts, short)]), q=q[rows],
                        cu_q=i32([0] + [int(c) for c in np.cumsum(short)]), max_q=max(short), inv_freq=inv)
    assert torch.equal(out[rows], want)
    assert (out.cpu()[~taken] == 7.0).all()
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(x, y)

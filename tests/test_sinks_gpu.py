"""Attention through a window with first tokens that stay visible, against a
plain 64-bit implementation.  Tolerances are those of test_serving_gpu.py."""

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded
from test_serving_gpu import BF16, E4M3, F16, F32, check_attention, make_cache, paging, to_gpu

pytestmark = pytest.mark.gpu

END = 2 ** 31 - 1


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reference(q, cache, table, lens, cu, window, sinks, scale):
    """As test_serving_gpu.reference_attention, with sinks and lengths past the table."""
    k, v, ks, vs = cache
    pages, heads, page, dim = k.shape
    group, width = q.shape[1] // heads, table.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    amount, rel = torch.zeros_like(out), torch.zeros(q.shape[:2], dtype=torch.float64)
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        ids = table[b].long()
        there = ((ids >= 0) & (ids < pages)).repeat_interleave(page)
        ids = torch.where((ids >= 0) & (ids < pages), ids, 0)
        pos, t = torch.arange(n - (hi - lo), n), torch.arange(width * page)
        see = (t <= pos[:, None]) & there
        if window > 0:
            see &= (t > pos[:, None] - window) | (t < sinks)
        for h in range(heads):
            kk = (E4M3[k[ids, h].long()] * torch.exp2(ks[ids, h].double() - 127)[:, None, None]).reshape(-1, dim)
            vv = E4M3[v[ids, h].long()] * torch.exp2(vs[ids, h].double() - 127)[:, None, None]
            vv = vv.transpose(1, 2).reshape(-1, dim)
            for j in range(h * group, (h + 1) * group):
                x = q[lo:hi, j].double()
                s = torch.where(see, x @ kk.nan_to_num().T * scale, -torch.inf)
                bad = ((x @ kk.T).isnan() & see).any(1)
                size = torch.where(see, x.abs() @ kk.nan_to_num().abs().T * scale, 0.0).amax(1)
                p = torch.where(see, torch.exp(s - s.amax(1, keepdim=True).clamp_min(-1e300)), 0.0)
                p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
                nan = (see.double() @ vv.isnan().double()) > 0
                out[lo:hi, j] = torch.where(nan | bad[:, None], torch.nan, p @ vv.nan_to_num())
                amount[lo:hi, j] = p @ vv.nan_to_num().abs()
                rel[lo:hi, j] = 2.0 ** -24 * (2 * ((dim + 8) * size + 6 * size + 16) + width * page + 16)
    return out, amount, rel


def run(seed, dtype, hq, hkv, dim, page, lens, counts, window, sinks, width=None, edit=None, decode=False, drop=True):
    """Pages that no row of a sequence sees hold NaN codes, or are not there."""
    g = torch.Generator().manual_seed(seed)
    width = width or -(-max(lens) // page)
    table, pages = paging(g, [min(n, width * page) for n in lens], page, width)
    cache = make_cache(g, pages, hkv, page, dim)
    for b, (n, c) in enumerate(zip(lens, counts)):
        for i in range(min(-(-n // page), width)):
            first = max(0, n - c - window + 1)                 # what the first row's window starts with
            if window > 0 and c and i * page >= sinks and (i + 1) * page <= first:
                if drop and i % 2:
                    table[b, i] = -1
                else:
                    for x in cache[:2]:
                        x[table[b, i]] = 0x7f
    if edit:
        edit(cache, table)
    cu = [0] + [int(c) for c in np.cumsum(counts)]
    q = (torch.randn(cu[-1], hq, dim, generator=g) * 0.5).to(dtype)
    out, guard = guarded(q.shape, dtype)
    print("attention", seed, dtype, hq, hkv, dim, page, lens, counts, window, sinks, flush=True)
    got = nv.paged_attention(q.to(DEV), to_gpu(cache), table.to(DEV), i32(lens), cu_q=None if decode else i32(cu),
                             max_q=None if decode else max(counts), window=window, sinks=sinks, out=out)
    guard()
    check_attention(got, *reference(q, cache, table, lens, cu, window, sinks, dim ** -0.5), dtype)
    return got


# windows and sinks around tiles of 64 and around each other
PAIRS = [(1, 1), (1, 64), (2, 63), (64, 65), (63, 1), (65, 128), (100, 4), (100, 300), (128, 129), (700, 5), (5000, 7),
         (50, 5000), (END, 9), (2 ** 40, 70), (30, 2 ** 40), (0, 50), (-3, 50), (90, 0), (90, -4)]


@pytest.mark.parametrize("window,sinks", PAIRS)
@pytest.mark.parametrize("dtype,hq,hkv,dim,page", [(BF16, 4, 1, 64, 16), (F16, 8, 8, 128, 64), (F32, 6, 2, 128, 32)])
def test_single_tokens(dtype, hq, hkv, dim, page, window, sinks):
    lens = [1, 2, 63, 64, 65, 129, 200, 300, 777]
    run(1, dtype, hq, hkv, dim, page, lens, [1] * len(lens), window, sinks, decode=True)


@pytest.mark.parametrize("window,sinks", PAIRS)
@pytest.mark.parametrize("dtype,hq,hkv,dim,page,counts", [
    (BF16, 7, 1, 128, 64, [130, 40, 1, 65]), (F16, 2, 2, 64, 256, [300, 64, 33, 0]), (F32, 4, 2, 64, 16, [60, 2, 1, 9]),
    (BF16, 2, 1, 64, 32, [150, 100, 17, 3]), (F16, 12, 2, 64, 16, [5, 6, 2, 1]),
])
def test_several_tokens(dtype, hq, hkv, dim, page, counts, window, sinks):
    run(2, dtype, hq, hkv, dim, page, [333, 517, 150, 65], counts, window, sinks)


@pytest.mark.parametrize("dtype,hq,hkv,dim,page,counts", [
    (BF16, 2, 2, 192, 128, [1, 40]), (F16, 4, 2, 256, 64, [90, 7]), (F32, 5, 1, 192, 64, [6, 1]), (F32, 2, 1, 256, 256, [20, 3]),
    (BF16, 3, 1, 256, 16, [50, 1]), (F16, 32, 2, 192, 32, [1, 1]),
])
@pytest.mark.parametrize("window,sinks", [(70, 10), (200, 130)])
def test_wide_heads(dtype, hq, hkv, dim, page, counts, window, sinks):
    run(3, dtype, hq, hkv, dim, page, [700, 500], counts, window, sinks)


@pytest.mark.parametrize("dtype,hq,hkv,counts", [(BF16, 8, 2, [1, 1]), (F32, 4, 1, [3, 1]), (F16, 4, 4, [100, 64]), (BF16, 4, 1, [40, 9])])
@pytest.mark.parametrize("window,sinks", [(3000, 4), (2500, 700), (64, 3500)])
def test_split_axis(dtype, hq, hkv, counts, window, sinks):
    """Splits that lie among the sinks, across their end, and behind."""
    run(4, dtype, hq, hkv, 64, 64, [6000, 9100], counts, window, sinks)


def test_split_and_whole_agree():
    g = torch.Generator().manual_seed(8)
    lens, page, dim = [9000], 64, 128
    table, pages = paging(g, lens, page)
    cache = to_gpu(make_cache(g, pages, 2, page, dim))
    q = torch.randn(1, 8, dim, generator=g).to(DEV)
    t, n = table.to(DEV), i32(lens)
    lib = nv.load_library()
    assert lib.nvfp4_paged_attention_sinks_workspace_size(1, 8, 2, dim, page, 1, 1, t.shape[1], 6000, 300, 0) > 0
    a = nv.paged_attention(q, cache, t, n, window=6000, sinks=300)
    b, guard = guarded((1, 8, dim), F32)
    assert lib.nvfp4_paged_attention_sinks(cache._ref, q.data_ptr(), q.stride(0), q.stride(1), 8, 0, 1, None, 1, 1,
                                           t.data_ptr(), t.shape[1], n.data_ptr(), 6000, 300, dim ** -0.5, None, 0,
                                           b.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    guard()
    assert (a - b).abs().max() <= 1e-4 * a.abs().max()
    assert torch.equal(a, nv.paged_attention(q, cache, t, n, window=6000, sinks=300))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 60, 7], [6, 1, 2]])
def test_missing_pages_and_nan_codes(dtype, counts):
    """Sinks' pages that are not there; NaN codes among the sinks, right behind
    them in their tile, and among what only some rows see."""
    def edit(cache, table):
        k, v, ks, vs = cache
        table[0, 0] = -1
        table[1, 1], table[1, 0] = 1 << 30, -9
        a = int(table[2, 0])
        k[a, :, 21:], v[a, :, :, 21:] = 0x7f, 0xff           # behind 21 sinks
        v[a, 0, 5, 3] = 0x7f                                  # a sink's value: every row's channel 5
        last = int(table[2, 9])
        v[last, 1, 7, 31] = 0xff                              # token 319: the last row sees it alone
    run(5, dtype, 8, 2, 64, 32, [300, 301, 320], counts, 80, 21, edit=edit, drop=False)


@pytest.mark.parametrize("dtype,hq,count", [(BF16, 4, 1), (F16, 2, 40), (F32, 2, 5)])
@pytest.mark.parametrize("window,sinks", [(1, 3), (100, 65), (129, 500)])
def test_lengths_past_the_table(dtype, hq, count, window, sinks):
    """The sinks are all that far rows see."""
    run(6, dtype, hq, 1, 64, 32, [100, 128, 129, 228, 400, END, END - 64], [count] * 7, window, sinks, width=4)


@pytest.mark.parametrize("dtype,hq,counts", [(BF16, 4, [1] * 3), (F16, 4, [200, 30, 64]), (F32, 2, [4, 1, 2])])
def test_equal_to_the_window_alone(dtype, hq, counts):
    """Without sinks, or with a window that all is in, nothing changes, bit for bit."""
    g = torch.Generator().manual_seed(9)
    lens, page = [500, 130, 64], 64
    table, pages = paging(g, lens, page)
    cache, t, n = to_gpu(make_cache(g, pages, 2, page, 64)), table.to(DEV), i32(lens)
    q = torch.randn(sum(counts), hq, 64, generator=g).to(dtype).to(DEV)
    cu = i32([0] + list(np.cumsum(counts)))
    call = lambda **k: nv.paged_attention(q, cache, t, n, cu_q=cu, max_q=max(counts), **k)  # noqa: E731
    assert torch.equal(call(window=90), call(window=90, sinks=0))
    assert torch.equal(call(), call(sinks=40))
    check = call(window=1000, sinks=40)
    assert torch.equal(call(window=1000), check)


def test_rows_past_max_q_and_unaligned_queries():
    g = torch.Generator().manual_seed(10)
    lens, counts, page = [400, 300], [9, 4], 16
    table, pages = paging(g, lens, page)
    cache = make_cache(g, pages, 1, page, 64)
    base = torch.randn(13, 3 * 64 + 1, generator=g).to(BF16)
    q, dq = base[:, 1:].unflatten(1, (3, 64)), base.to(DEV)[:, 1:].unflatten(1, (3, 64))
    out, guard = guarded((13, 3, 64), BF16, fill=3.0)
    nv.paged_attention(dq, to_gpu(cache), table.to(DEV), i32(lens), cu_q=i32([0, 9, 13]), max_q=5, window=70, sinks=40, out=out)
    guard()
    ref = reference(q, cache, table, lens, [0, 9, 13], 70, 40, 0.125)
    rows = [0, 1, 2, 3, 4, 9, 10, 11, 12]
    check_attention(out[rows], *[x[rows] for x in ref], BF16)
    assert (out[5:9] == 3.0).all()


def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 4 GiB a side."""
    heads, page, dim = 8, 256, 256
    pages = (1 << 32) // (heads * page * dim) + 8
    g = torch.Generator().manual_seed(11)
    small = make_cache(g, 3, heads, page, dim)
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    big = nv.KVCache(z(pages, heads, page, dim), z(pages, heads, dim, page), z(pages, heads), z(pages, heads))
    where = [pages - 1, 1, pages - 5]
    for i, p in enumerate(where):
        for dst, src in zip((big.k, big.v, big.k_scales, big.v_scales), small):
            dst[p] = src[i].to(DEV)
    for count in (1, 50):
        q = torch.randn(count, heads, dim, generator=g).to(BF16)
        got = nv.paged_attention(q.to(DEV), big, i32([where]), i32([700]), cu_q=i32([0, count]), window=200, sinks=70)
        ref = reference(q, small, torch.tensor([[0, 1, 2]]), [700], [0, count], 200, 70, dim ** -0.5)
        check_attention(got, *ref, BF16)

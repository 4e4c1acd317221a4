"""The serving operators against plain 64-bit implementations on the CPU.

Tolerances come from the roundings.  Let h be half a step of the output type
(finfo.eps / 2).  Attention: the output's own rounding, h |out|; the weights'
rounding to the 2-byte type for their product, h * sum_t p_t |v_t| (float32
weights are exact); and the 32-bit arithmetic: a score is off by at most (dim +
8) 2^-24 sum |q k| scale plus roundings of its size in powers of two (below 4
|s| + 8 of them, two for the value scale's exponent), which goes into weights
and their sum, and the sums over n tokens by n 2^-24 of sum p |v|.  Appended
values: half a step of the code.  Sampling: tokens are equal; a probability is
off by its float rounding and the 1e-11 of each weight.
"""

import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def e4m3_table():
    t = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(1 + m / 8, e - 7) if e else math.ldexp(m, -9)
        t.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(t, dtype=torch.float64)


E4M3 = e4m3_table()


def make_cache(g, pages, heads, page, dim, spread=3, nan_codes=False):
    k = torch.randint(0, 256, (pages, heads, page, dim), generator=g, dtype=torch.int32).to(torch.uint8)
    v = torch.randint(0, 256, (pages, heads, dim, page), generator=g, dtype=torch.int32).to(torch.uint8)
    # codes of ordinary magnitude (exponent fields around 2^-2 .. 2^2), no NaN
    for c in (k, v):
        c &= 0x87
        c |= (torch.randint(4, 9, c.shape, generator=g, dtype=torch.int32) << 3).to(torch.uint8)
    ks = torch.randint(127 - spread, 127 + spread + 1, (pages, heads), generator=g, dtype=torch.int32).to(torch.uint8)
    vs = torch.randint(127 - spread, 127 + spread + 1, (pages, heads), generator=g, dtype=torch.int32).to(torch.uint8)
    return k, v, ks, vs


def to_gpu(c):
    return nv.KVCache(*[t.to(DEV) for t in c])


def paging(g, lens, page, width=None, extra=3):
    """A table of distinct random pages for each sequence; entries behind them -1."""
    need = [-(-max(n, 0) // page) for n in lens]
    width = width or max(need + [1])
    order = torch.randperm(sum(need) + extra, generator=g).int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, sum(need) + extra


def reference_attention(q, cache, table, lens, cu, window, scale):
    """out and, per element, the tolerance's sum p |v|, with the row's score sizes."""
    k, v, ks, vs = cache
    pages, heads, page, dim = k.shape
    group = q.shape[1] // heads
    out = torch.zeros(q.shape, dtype=torch.float64)
    amount, rel = torch.zeros_like(out), torch.zeros(q.shape[:2], dtype=torch.float64)
    for b, n in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if hi == lo or n <= 0:
            continue
        ids = table[b, :-(-n // page)].long()
        there = (ids >= 0) & (ids < pages)
        ids = torch.where(there, ids, 0)
        there = there.repeat_interleave(page)[:n]
        pos = torch.arange(n - (hi - lo), n)
        t = torch.arange(n)[:ids.numel() * page]
        see = (t <= pos[:, None]) & there[None, :]
        if window > 0:
            see &= t > pos[:, None] - window
        for h in range(heads):
            kk = (E4M3[k[ids, h].long()] * torch.exp2(ks[ids, h].double() - 127)[:, None, None]).reshape(-1, dim)[:n]
            vv = E4M3[v[ids, h].long()] * torch.exp2(vs[ids, h].double() - 127)[:, None, None]
            vv = vv.transpose(1, 2).reshape(-1, dim)[:n]
            for j in range(h * group, (h + 1) * group):
                x = q[lo:hi, j].double()
                s = torch.where(see, x @ kk.nan_to_num().T * scale, -math.inf)
                bad = torch.where(see, (x @ kk.T).isnan() & see, False).any(1)
                size = torch.where(see, x.abs() @ kk.nan_to_num().abs().T * scale, 0.0).amax(1)
                p = torch.exp(s - s.amax(1, keepdim=True).clamp_min(-1e300))
                p = torch.where(see, p, 0.0)
                total = p.sum(1, keepdim=True)
                p = p / torch.where(total > 0, total, 1.0)
                o = p @ vv.nan_to_num()
                nan = (see.double() @ vv.isnan().double()) > 0
                out[lo:hi, j] = torch.where(nan | bad[:, None], math.nan, o)
                amount[lo:hi, j] = p @ vv.nan_to_num().abs()
                rel[lo:hi, j] = 2.0 ** -24 * (2 * ((dim + 8) * size + 6 * size + 16) + n + 16)
    return out, amount, rel


def check_attention(got, ref, amount, rel, dtype):
    h = torch.finfo(dtype).eps / 2
    weights = h if dtype != F32 else 0.0
    tiny = torch.finfo(dtype).smallest_normal * h    # the step below the normal numbers
    tol = h * ref.abs() + weights * (1 + h) * amount + rel[..., None] * amount + tiny
    got = got.double().cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    err = torch.where(ref.isnan(), 0.0, (got - ref).abs() - tol)
    assert err.max() <= 0, (float(err.max()), float((got - ref).abs().nan_to_num().max()))


def run_attention(seed, dtype, hq, hkv, dim, page, lens, counts, window=0, spread=3, width=None, edit=None, q=None,
                  scale=None, decode=False):
    g = torch.Generator().manual_seed(seed)
    table, pages = paging(g, lens, page, width)
    cache = make_cache(g, pages, hkv, page, dim, spread)
    if edit:
        edit(cache, table)
    cu = [0] + list(np.cumsum(counts))
    tokens = cu[-1]
    if q is None:
        q = (torch.randn(tokens, hq, dim, generator=g) * 0.5).to(dtype)
    out, guard = guarded((tokens, hq, dim), dtype)
    print("attention", seed, dtype, hq, hkv, dim, page, lens, counts, window, flush=True)
    got = nv.paged_attention(q.to(DEV), to_gpu(cache), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                             cu_q=None if decode else torch.tensor(cu, dtype=torch.int32, device=DEV),
                             max_q=None if decode else max(counts), window=window, scale=scale, out=out)
    guard()
    ref = reference_attention(q, cache, table, lens, cu, window, scale or dim ** -0.5)
    check_attention(got, *ref, dtype)
    return got


DECODE = [
    # dtype, hq, hkv, dim, page, lens
    (BF16, 4, 1, 64, 16, [1, 2, 15, 16, 17, 63, 64, 65]),
    (F16, 8, 8, 128, 64, [1, 127, 300]),
    (F32, 6, 2, 128, 32, [1, 33, 255, 700]),
    (BF16, 32, 2, 192, 128, [129, 1000]),
    (F32, 7, 1, 256, 256, [5, 513]),
    (F16, 14, 2, 256, 64, [900, 3]),
    (BF16, 48, 1, 128, 64, [777, 64]),           # more rows than one tile of columns
    (BF16, 32, 8, 128, 64, [9000]),               # a split axis
    (F16, 5, 5, 64, 256, [20000, 1, 4097]),       # split, unevenly
    (F32, 3, 1, 192, 16, [5000, 4999]),
]


@pytest.mark.parametrize("dtype,hq,hkv,dim,page,lens", DECODE)
def test_attention_single_tokens(dtype, hq, hkv, dim, page, lens):
    run_attention(1, dtype, hq, hkv, dim, page, lens, [1] * len(lens), decode=True)


MANY = [
    # dtype, hq, hkv, dim, page, lens, counts, window
    (BF16, 4, 2, 128, 64, [70, 3, 200], [5, 3, 2], 0),
    (F16, 21, 7, 64, 32, [300, 31], [6, 6], 50),
    (F32, 6, 3, 256, 32, [90, 500], [6, 4], 64),
    (BF16, 7, 1, 128, 64, [130, 257], [130, 40], 0),        # whole prompt beside a chunk
    (F16, 2, 2, 64, 256, [700], [300], 0),
    (F16, 6, 2, 192, 128, [333, 65], [100, 65], 37),
    (F32, 4, 2, 64, 16, [200, 129], [200, 1], 0),
    (BF16, 16, 16, 64, 256, [5000], [64], 0),                # a chunk over a long cache: split
    (BF16, 10, 2, 256, 64, [600], [100], 0),
    (F32, 3, 3, 128, 128, [300], [150], 17),
    (BF16, 4, 4, 128, 64, [1, 1, 40, 0], [1, 1, 0, 0], 0),   # sequences without new tokens
    (BF16, 12, 1, 128, 128, [2000, 1500], [33, 21], 1),      # a window of the token itself
    (F16, 8, 1, 128, 64, [1500, 1400], [200, 333], 700),
]


@pytest.mark.parametrize("dtype,hq,hkv,dim,page,lens,counts,window", MANY)
def test_attention_several_tokens(dtype, hq, hkv, dim, page, lens, counts, window):
    run_attention(2, dtype, hq, hkv, dim, page, lens, counts, window)


@pytest.mark.parametrize("dtype,counts", [(BF16, [1, 1, 1]), (F16, [40, 300, 7]), (F32, [3, 50, 1])])
def test_attention_missing_pages_and_empty_rows(dtype, counts):
    def edit(cache, table):
        table[0, :] = -1                       # nothing at all
        table[1, 2] = 1 << 30                  # outside the pool
        table[1, 0] = -7
        table[2, -1] = -1
    run_attention(3, dtype, 8, 2, 128, 32, [100, 300, 130], counts, edit=edit)


def test_attention_lengths_past_the_table():
    """Tokens behind the table's width are not there; the rows see the others."""
    g = torch.Generator().manual_seed(4)
    cache = make_cache(g, 4, 1, 32, 64)
    table = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32)
    q = torch.randn(2, 4, 64, generator=g).to(BF16)
    lens = torch.tensor([1000, -5], dtype=torch.int32)
    got = nv.paged_attention(q.to(DEV), to_gpu(cache), table.to(DEV), lens.to(DEV))
    ref = reference_attention(q[:1], cache, table, [64], [0, 1], 0, 64 ** -0.5)
    check_attention(got[:1], *ref, BF16)
    assert (got[1] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("counts", [[1, 1], [9, 4], [150, 90]])
def test_attention_nan_codes(dtype, counts):
    """NaN codes behind the end and among tokens that only later rows see:
    each row is spoiled exactly by those that it sees."""
    lens, page = [200, 170], 64
    def edit(cache, table):
        k, v, ks, vs = cache
        last = int(table[0, 3])                # tokens 192 .. of sequence 0; 200 on are behind the end
        k[last, :, 8:], v[last, :, :, 8:] = 0x7f, 0xff
        at = int(table[1, 2])                  # token 168 of sequence 1: seen by its last two rows only
        v[at, 0, 5, 40] = 0xff
        k[at, 1, 41, 3] = 0x7f                 # token 169: by the last row only
    run_attention(5, dtype, 6, 2, 128, page, lens, counts, edit=edit)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_attention_scales_far_apart(dtype):
    """Value scales of 2^-14 .. 2^14 and a page of zeros with scale byte 0,
    the weight on one page or spread."""
    def edit(cache, table):
        k, v, ks, vs = cache
        vs[:] = (127 + 4 * ((torch.arange(vs.shape[0]) % 7) - 3)).to(torch.uint8)[:, None]
        i = int(table[0, 1])
        v[i], vs[i] = 0, 0
    for count in (1, 70):
        run_attention(6, dtype, 4, 2, 64, 32, [220, 90], [count, min(count, 20)], edit=edit, spread=1)


def test_attention_strided_and_unaligned_queries():
    g = torch.Generator().manual_seed(7)
    lens, counts, hq, dim = [90, 120], [1, 20], 4, 64
    for dtype, off in ((BF16, 0), (F16, 1), (F32, 3)):
        base = (torch.randn(21, hq * dim + 129 + off, generator=g)).to(dtype)
        q = base[:, off:off + hq * dim].unflatten(1, (hq, dim))
        dq = base.to(DEV)[:, off:off + hq * dim].unflatten(1, (hq, dim))
        table, pages = paging(g, lens, 32)
        cache = make_cache(g, pages, 2, 32, dim)
        cu = [0, 1, 21]
        got = nv.paged_attention(dq, to_gpu(cache), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 cu_q=torch.tensor(cu, dtype=torch.int32, device=DEV))
        check_attention(got, *reference_attention(q, cache, table, lens, cu, 0, dim ** -0.5), dtype)


def test_attention_split_and_whole_agree():
    """The workspace only splits the axis: without one the C entry gives the
    same up to the order of 32-bit sums."""
    g = torch.Generator().manual_seed(8)
    lens, page, dim = [6000], 64, 128
    table, pages = paging(g, lens, page)
    cache = to_gpu(make_cache(g, pages, 2, page, dim))
    q = torch.randn(1, 8, dim, generator=g).to(DEV)
    t, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    lib = nv.load_library()
    assert lib.nvfp4_paged_attention_workspace_size(1, 8, 2, dim, page, 1, 1, t.shape[1], 0, 0) > 0
    a = nv.paged_attention(q, cache, t, n)
    b, guard = guarded((1, 8, dim), F32)
    assert lib.nvfp4_paged_attention(cache._ref, q.data_ptr(), q.stride(0), q.stride(1), 8, 0, 1, None, 1, 1,
                                     t.data_ptr(), t.shape[1], n.data_ptr(), 0, dim ** -0.5, None, 0, b.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    guard()
    assert (a - b).abs().max() <= 1e-4 * a.abs().max()
    assert torch.equal(a, nv.paged_attention(q, cache, t, n))     # and repeats bit for bit


def test_attention_offsets_past_32_bits():
    """A pool of more than 4 GiB a side: pages at its end."""
    heads, page, dim = 8, 256, 256
    pages = (1 << 32) // (heads * page * dim) + 8
    g = torch.Generator().manual_seed(9)
    small = make_cache(g, 3, heads, page, dim)
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    big = nv.KVCache(z(pages, heads, page, dim), z(pages, heads, dim, page), z(pages, heads), z(pages, heads))
    where = [pages - 1, 1, pages - 5]
    for i, p in enumerate(where):
        for dst, src in zip((big.k, big.v, big.k_scales, big.v_scales), small):
            dst[p] = src[i].to(DEV)
    for counts, lens in (([1], [700]), ([50], [600])):
        q = torch.randn(counts[0], heads, dim, generator=g).to(BF16)
        cu = torch.tensor([0] + counts, dtype=torch.int32, device=DEV)
        got = nv.paged_attention(q.to(DEV), big, torch.tensor([where], dtype=torch.int32, device=DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), cu_q=cu)
        ref = reference_attention(q, small, torch.tensor([[0, 1, 2]], dtype=torch.int32), lens, [0] + counts, 0, dim ** -0.5)
        check_attention(got, *ref, BF16)
    # and an append at the end of it
    k = torch.randn(1, heads, dim, generator=g).to(BF16)
    nv.kv_append(k.to(DEV), k.to(DEV), big, torch.tensor([where], dtype=torch.int32, device=DEV),
                 torch.tensor([257], dtype=torch.int32, device=DEV))
    first = big.k[1, :, 0].cpu()
    scale = torch.exp2(big.k_scales[1].cpu().double() - 127)[:, None]
    x = k[0].double()
    assert ((E4M3[first.long()] * scale - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * scale).all()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def rotate(x, pos, inv_freq, interleaved):
    """x [tokens, heads, dim] in 64 bits, rounded to float32 at the end."""
    x = x.double().clone()
    r = 2 * len(inv_freq)
    ang = pos.double()[:, None] * inv_freq.double()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    ia = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    ib = ia + (1 if interleaved else r // 2)
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x.float()


def scale_byte_of(amax):
    """From the definition: the smallest power of two p with amax <= 448 p."""
    if amax == 0:
        return 0
    p = -127
    while amax > math.ldexp(448.0, p):
        p += 1
    return p + 127


def check_codes(codes, want, byte):
    """codes hold `want` (64 bits) at the scale to within half a step; not finite: NaN."""
    scale = math.ldexp(1.0, byte - 127)
    got = E4M3[codes.long()] * scale
    ok = want.isfinite()
    assert torch.equal(got.isnan(), ~ok)
    # the step is relative above 2^-6 and 2^-9 below it
    tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10 * scale)) * (1 + 2.0 ** -20)
    err = torch.where(ok, (got - want).abs() - tol, 0.0)
    assert err.max() <= 0, float(err.max())


def run_append(seed, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved=False, strided=True, edit=None, off=0,
               loud=0.0, missing=()):
    g = torch.Generator().manual_seed(seed)
    lens = [f + c for f, c in zip(firsts, counts)]
    table, pages = paging(g, lens, page)
    for b, i in missing:
        table[b, i] = -1
    cache = make_cache(g, pages, hkv, page, dim, spread=2)
    before = [t.clone() for t in cache]
    tokens = sum(counts)
    width = (hq + 2 * hkv) * dim
    base = (torch.randn(tokens, width + off, generator=g) * math.exp(loud)).to(dtype)
    if edit:
        edit(base[:, off:])
    dev = base.to(DEV)
    parts = lambda t: [p.unflatten(1, (-1, dim)) for p in t[:, off:].split([hq * dim, hkv * dim, hkv * dim], 1)]  # noqa: E731
    q, k, v = parts(base)
    dq, dk, dv = parts(dev)
    inv = (10000.0 ** (-torch.arange(0, rot, 2).float() / max(rot, 1))) if rot else None
    cu = [0] + list(np.cumsum(counts))
    c = to_gpu(cache)
    print("append", seed, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved, flush=True)
    out, guard = guarded((tokens, hq, dim), dtype)
    nv.kv_append(dk, dv, c, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), q=dq,
                 cu_q=torch.tensor(cu, dtype=torch.int32, device=DEV), max_q=max(counts),
                 inv_freq=None if inv is None else inv.to(DEV), interleaved=interleaved, out=out)
    guard()
    pos = torch.cat([torch.arange(f, f + n) for f, n in zip(firsts, counts)] + [torch.zeros(0, dtype=torch.long)])
    inv_t = inv if inv is not None else torch.zeros(0)
    qr, kr = rotate(q, pos, inv_t, interleaved), rotate(k, pos, inv_t, interleaved)
    got_q = out.cpu().double()
    h = torch.finfo(dtype).eps / 2
    size = (q.double().abs().amax(-1, keepdim=True))
    fin = qr.isfinite()
    assert torch.equal(got_q.isfinite(), fin)
    assert (torch.where(fin, (got_q - qr.double()).abs(), 0.0) <= h * qr.double().abs().nan_to_num() * (1 + 2.0 ** -10)
            + 2.0 ** -24 * 2 * size.nan_to_num() + torch.finfo(dtype).smallest_normal * h).all()
    after = [t.cpu() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    touched = torch.zeros(pages, dtype=torch.bool)
    for b, (f, n) in enumerate(zip(firsts, counts)):
        for i in range(f // page, -(-(f + n) // page) if n else f // page):
            pid = int(table[b, i])
            if pid < 0:
                continue
            touched[pid] = True
            lo, hi = max(f, i * page), min(f + n, (i + 1) * page)
            held, rows = lo - i * page, slice(cu[b] + lo - f, cu[b] + hi - f)
            for h_ in range(hkv):
                for side, x in ((0, kr[rows, h_].double()), (1, v[rows, h_].double())):
                    fresh = scale_byte_of(float(torch.where(x.isfinite(), x.abs(), 0.0).max()))
                    old = int(before[2 + side][pid, h_])
                    byte = max(fresh, old) if held else fresh
                    assert int(after[2 + side][pid, h_]) == byte
                    was, now = before[side][pid, h_], after[side][pid, h_]
                    if side:
                        was, now = was.T, now.T
                    check_codes(now[held:held + hi - lo], x, byte)
                    if held:
                        kept = E4M3[was[:held].long()] * math.ldexp(1.0, old - 127)
                        if byte == old:
                            assert torch.equal(now[:held], was[:held])
                        else:
                            check_codes(now[:held], kept, byte)
                    assert torch.equal(now[held + hi - lo:], was[held + hi - lo:])   # behind the end: untouched
    for t, u in zip(after, before):
        assert torch.equal(t[~touched], u[~touched])


APPEND = [
    # dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved
    (BF16, 4, 2, 128, 64, [0, 63, 64, 1000], [1, 1, 1, 1], 128, False),
    (F16, 6, 1, 64, 16, [0, 5, 31], [40, 1, 18], 64, True),
    (F32, 2, 2, 256, 32, [7, 100], [60, 3], 128, False),
    (F32, 3, 3, 192, 256, [250, 0], [20, 300], 96, True),
    (BF16, 42, 6, 128, 128, [15], [260], 96, True),
    (BF16, 1, 1, 256, 256, [3], [510], 256, False),          # more values of a page than the threads hold
    (F16, 8, 4, 128, 64, [0, 1, 0], [0, 0, 5], 0, False),     # no rotation; sequences without new tokens
    (F16, 2, 2, 64, 64, [70], [9], 10, False),                # pairs that no 16-byte access fits
    (BF16, 2, 1, 64, 32, [30], [40], 6, True),
]


@pytest.mark.parametrize("dtype,hq,hkv,dim,page,firsts,counts,rot,interleaved", APPEND)
def test_append(dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved):
    run_append(11, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_append_unaligned_rows(dtype):
    run_append(12, dtype, 3, 2, 64, 32, [20, 0], [30, 1], 64, off=1)


@pytest.mark.parametrize("loud", [-6.0, 0.0, 5.0])
def test_append_rescales_what_a_page_holds(loud):
    """Quieter, equal and louder values than the page's: in the last case the
    held codes are rounded anew at the grown scale."""
    run_append(13, F32, 2, 2, 128, 64, [1, 33, 62], [1, 5, 70], 128, loud=loud)
    run_append(14, BF16, 2, 2, 64, 32, [3, 29], [1, 1], 64, loud=loud)


def test_append_values_that_are_not_finite_and_zeros():
    def edit(x):
        x[0, 70] = math.inf
        x[1, 200] = math.nan
        x[2, 150:] = 0.0
        x[3, 300] = -math.inf
    run_append(15, F32, 1, 2, 64, 32, [10, 0, 40], [2, 1, 3], 0, edit=edit)


def test_append_extreme_magnitudes():
    run_append(16, F32, 1, 1, 64, 32, [0, 5], [3, 1], 64, loud=-80.0)
    run_append(17, F32, 1, 1, 64, 32, [0, 5], [3, 1], 64, loud=80.0)


def test_append_far_positions():
    run_append(18, F32, 2, 1, 64, 256, [131071, 500000], [1, 3], 64)


def test_append_missing_pages():
    run_append(19, BF16, 2, 1, 64, 32, [10, 30], [60, 2], 64, missing=((0, 1), (1, 0)))


def test_append_one_token_without_offsets():
    """cu_q left out, no queries: the same cache as with them."""
    g = torch.Generator().manual_seed(20)
    table, pages = paging(g, [40, 1, 33], 32)
    a, b = [to_gpu(make_cache(torch.Generator().manual_seed(1), pages, 2, 32, 64)) for _ in range(2)]
    k, v = (torch.randn(3, 2, 64, generator=g).to(DEV) for _ in range(2))
    t, n = table.to(DEV), torch.tensor([40, 1, 33], dtype=torch.int32, device=DEV)
    inv = (10000.0 ** (-torch.arange(0, 64, 2).float() / 64)).to(DEV)
    assert nv.kv_append(k, v, a, t, n, inv_freq=inv) is None
    nv.kv_append(k, v, b, t, n, inv_freq=inv, q=k, cu_q=torch.arange(4, dtype=torch.int32, device=DEV), max_q=1)
    for x, y in ((a.k, b.k), (a.v, b.v), (a.k_scales, b.k_scales), (a.v_scales, b.v_scales)):
        assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

def reference_sample(x, u, t, k, p, m):
    """(token, probability) of one row, from the definition in 64 bits."""
    x = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
    top = x.max()
    if top == -np.inf:
        return -1, 0.0
    with np.errstate(all="ignore"):
        w = np.exp((x - top) / t)
    w[x == top] = 1.0
    w[x == -np.inf] = 0.0
    order = np.argsort(-x, kind="stable")
    if k > 0:
        order = order[:k]
    if p < 1:
        before = np.cumsum(w[order]) - w[order]
        keep = before < p * w[order].sum()
        keep[0] = True
        order = order[keep]
    keep = w[order] >= m
    keep[0] = True
    order = np.sort(order[keep & (w[order] > 0)])
    c = np.cumsum(w[order])
    i = min(int(np.searchsorted(c, u * c[-1], side="right")), len(order) - 1)
    return int(order[i]), float(w[order[i]] / c[-1])


def run_sample(x, u, t=None, k=None, p=None, m=None, dev=None):
    batch = x.shape[0]
    f = lambda a: None if a is None else torch.tensor(a, dtype=F32, device=DEV)  # noqa: E731
    print("sample", tuple(x.shape), x.dtype, flush=True)
    token, prob = nv.sample(x.to(DEV) if dev is None else dev, f(u), temperature=f(t),
                            top_k=None if k is None else torch.tensor(k, dtype=torch.int32, device=DEV), top_p=f(p),
                            min_p=f(m), return_prob=True)
    token, prob = token.cpu(), prob.cpu()
    f32 = lambda a, i, d: d if a is None else float(np.float32(a[i]))  # noqa: E731
    for i in range(batch):
        want, pr = reference_sample(x[i].double().numpy(), f32(u, i, 0), f32(t, i, 1.0), 0 if k is None else k[i],
                                    f32(p, i, 1.0), f32(m, i, 0.0))
        assert int(token[i]) == want, (i, int(token[i]), want)
        assert abs(float(prob[i]) - pr) <= pr * (2.0 ** -24 + 1e-10) + 1e-40, (i, float(prob[i]), pr)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 1000, 4099, 50001])
def test_sample_filters(dtype, vocab):
    g = torch.Generator().manual_seed(vocab)
    batch = 12
    x = (torch.randn(batch, vocab, generator=g) * 2.5).to(dtype)
    u = torch.rand(batch, generator=g).tolist()
    t = (torch.rand(batch, generator=g) + 0.5).tolist()
    k = torch.randint(0, 60, (batch,), generator=g).tolist()
    p = (torch.rand(batch, generator=g) * 0.6 + 0.4).tolist()
    m = (torch.rand(batch, generator=g) * 0.1).tolist()
    run_sample(x, u)
    run_sample(x, u, t)
    run_sample(x, u, t, k=k)
    run_sample(x, u, t, p=p)
    run_sample(x, u, t, m=m)
    run_sample(x, u, t, k, p, m)


def test_sample_large_vocabulary():
    g = torch.Generator().manual_seed(30)
    for dtype, vocab in ((BF16, 262144), (F32, 151936), (F16, 300001)):
        x = (torch.randn(3, vocab, generator=g) * 2).to(dtype)
        u = torch.rand(3, generator=g).tolist()
        run_sample(x, u)
        run_sample(x, u, [0.7, 1.0, 1.4], k=[50, 0, 5000], p=[0.9, 0.5, 0.97], m=[0.0, 0.01, 0.0])


def test_sample_ties():
    """Equal logits at every border: the lowest indices stay."""
    x = torch.zeros(6, 1000)
    u = [0.0, 0.5, 0.999, 0.25, 0.75, 0.1]
    run_sample(x, u, k=[1, 10, 999, 64, 65, 1000])
    run_sample(x, u, p=[0.5, 0.25, 0.125, 0.9, 0.001, 0.75])
    run_sample(x, u, k=[7] * 6, p=[0.5] * 6)
    y = (torch.arange(3000) % 7).float().repeat(6, 1)
    run_sample(y, u, k=[1, 428, 429, 430, 1000, 2999], p=[1.0, 0.9, 0.5, 0.99, 0.7, 0.8])
    run_sample(y.to(BF16), u, [0.5] * 6, k=[300] * 6, m=[0.1, 0.2, 0.9, 1.0, 1.5, 0.0])


def test_sample_extremes():
    inf, nan = math.inf, math.nan
    rows = torch.tensor([[nan, -inf, -inf, -inf, -inf], [-inf, 3.0, nan, 3.0, -inf], [inf, 0.0, inf, nan, 1.0],
                         [-0.0, 0.0, -1e30, 0.0, -0.0], [1e38, -1e38, 0.0, 3e38, 3e38], [1e-40, 0.0, -1e-40, 2e-40, 0.0]])
    u = [0.3, 0.6, 0.6, 0.9, 0.2, 0.7]
    run_sample(rows, u)
    run_sample(rows, u, p=[0.5] * 6, k=[2] * 6)
    run_sample(rows, [0.0] * 6, p=[0.0] * 6)
    run_sample(rows, [0.99] * 6, m=[0.5] * 6, t=[0.01] * 6)
    # a weight that the row's sum swallows is still the first by index at u = 0
    far = torch.full((2, 700), -600.0)
    far[:, 300] = 0.0
    run_sample(far, [0.0, 0.5])
    run_sample(torch.tensor([[1.0, 5.0, 5.0, 2.0]] * 3), [0.0, 0.4, 0.6], t=[0.0] * 3)


def test_sample_peaked_rows_and_strides():
    g = torch.Generator().manual_seed(31)
    base = torch.randn(5, 40000, generator=g)
    base[:, 12345] += 60
    for off, n in ((0, 32000), (3, 33333)):
        x = base[:, off:off + n]
        dev = base.to(DEV)[:, off:off + n]
        run_sample(x, torch.rand(5, generator=g).tolist(), p=[0.9] * 5, dev=dev)
        h = base.to(F16)
        run_sample(h[:, off:off + n], torch.rand(5, generator=g).tolist(), k=[40] * 5, dev=h.to(DEV)[:, off:off + n])


def test_sample_repeats_and_refuses():
    x = torch.randn(4, 100000, device=DEV)
    u = torch.rand(4, device=DEV)
    p = torch.full((4,), 0.95, device=DEV)
    a = nv.sample(x, u, top_p=p, return_prob=True)
    for _ in range(5):
        b = nv.sample(x, u, top_p=p, return_prob=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        nv.sample(x, u[:3])
    with pytest.raises(TypeError):
        nv.sample(x, u.double())
    with pytest.raises(TypeError):
        nv.sample(x, u, top_k=p)
    with pytest.raises(ValueError):
        nv.sample(x.T, u)
    with pytest.raises(ValueError):
        nv.sample(torch.zeros(4, 0, device=DEV), u)
    assert nv.sample(torch.zeros(0, 10, device=DEV), u[:0]).shape == (0,)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_refusals_on_the_gpu():
    c = nv.KVCache.empty(4, 2, 32, 64)
    t = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    n = torch.ones(2, dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 4, 64, device=DEV)
    k = torch.zeros(2, 2, 64, device=DEV)
    for bad in (dict(q=q[:, :3]), dict(q=q[:1]), dict(q=q.cpu()), dict(table=t.long()), dict(lens=n[:1]), dict(q=q[..., :32]),
                dict(table=t[:, ::2]), dict(out=q.half()), dict(out=q[:1]), dict(cu_q=n), dict(q=q.double()),
                dict(cu_q=torch.zeros(3, dtype=torch.int32, device=DEV), max_q=0),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            nv.paged_attention(**{**dict(q=q, cache=c, table=t, lens=n), **bad})
    for bad in (dict(k=k.half()), dict(v=k[:, :1]), dict(inv_freq=torch.zeros(40, device=DEV)),
                dict(inv_freq=torch.zeros(4, device=DEV).double()), dict(q=q.half()), dict(out=q), dict(v=k[:1])):
        with pytest.raises((ValueError, TypeError)):
            nv.kv_append(**{**dict(k=k, v=k, cache=c, table=t, lens=n), **bad})
    with pytest.raises(ValueError):
        nv.KVCache(c.k, c.v, c.k_scales.T.contiguous().T, c.v_scales)
    assert nv.paged_attention(q[:0], c, t[:0], n[:0]).shape == (0, 4, 64)
    empty = nv.KVCache.empty(0, 2, 32, 64)
    assert (nv.paged_attention(q + 1, empty, t, n) == 0).all()
    assert nv.kv_append(k, k, empty, t, n, q=q).shape == q.shape


def _step(s):
    q = nv.kv_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], q=s["q"], inv_freq=s["inv"])
    o = nv.paged_attention(q, s["cache"], s["table"], s["lens"])
    logits = o.reshape(o.shape[0], -1).float()
    return o, nv.sample(logits, s["u"], top_p=s["p"])


def _state(seed):
    g = torch.Generator().manual_seed(seed)
    lens = [3000, 70]
    table, pages = paging(g, lens, 64)
    return {"cache": to_gpu(make_cache(g, pages, 2, 64, 128)), "table": table.to(DEV),
            "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "q": torch.randn(2, 8, 128, generator=g).to(BF16).to(DEV), "k": torch.randn(2, 2, 128, generator=g).to(BF16).to(DEV),
            "v": torch.randn(2, 2, 128, generator=g).to(BF16).to(DEV), "u": torch.rand(2, generator=g).to(DEV),
            "p": torch.full((2,), 0.9, device=DEV), "inv": (10000.0 ** (-torch.arange(0, 128, 2).float() / 128)).to(DEV)}


def test_step_on_another_stream_and_in_a_graph():
    s = _state(40)
    o, token = _step(s)
    torch.cuda.synchronize()
    want, want_token = o.clone(), token.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, t2 = _step(s)
    side.synchronize()
    assert torch.equal(o2, want) and torch.equal(t2, want_token)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gt = _step(s)
    for i in range(4):
        fresh = _state(41 + i)
        for name in ("q", "k", "v", "u"):
            s[name].copy_(fresh[name])
        graph.replay()
        torch.cuda.synchronize()
        got, got_token = go.clone(), gt.clone()
        eo, et = _step(s)               # appends the same values again: the cache does not change
        assert torch.equal(got, eo) and torch.equal(got_token, et), i

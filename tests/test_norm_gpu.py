"""The cache append with norms of the queries' and keys' heads, against plain
64-bit implementations on the CPU.

Norm and rotation are in 64 bits on both sides and agree to 1e-12 of a head's
largest value (sums of 256 squares, sines and cosines good to 4e-13); what is
left is one rounding to 32 bits, 2^-24 of the value, and one to the type, half
a step, or to the code, half a step of it.
"""

import itertools
import math

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded
from test_serving_gpu import BF16, E4M3, F16, F32, check_codes, make_cache, paging, scale_byte_of, to_gpu

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def normed(x, weight, eps):
    x = x.double()
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def turned(x, pos, inv, interleaved):
    """Channels [0, 2 len(inv)) of x [tokens, heads, dim] rotated by the positions' angles, in 64 bits."""
    if inv is None:
        return x
    half = inv.numel()
    angle = pos[:, None].double() * inv.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    i = torch.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.clone()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    return y


def run(seed, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved=False, off=0, sides="qk", per_head=False, eps=1e-6,
        loud=0.0, edit=None, max_q=None, decode=False):
    g = torch.Generator().manual_seed(seed)
    lens = [f + c for f, c in zip(firsts, counts)]
    table, pages = paging(g, lens, page)
    cache = make_cache(g, pages, hkv, page, dim, spread=2)
    before = [t.clone() for t in cache]
    tokens = sum(counts)
    base = (torch.randn(tokens, (hq + 2 * hkv) * dim + off, generator=g) * math.exp(loud)).to(dtype)
    if edit:
        edit(base[:, off:])
    dev = base.to(DEV)
    parts = lambda t: [p.unflatten(1, (-1, dim)) for p in t[:, off:].split([hq * dim, hkv * dim, hkv * dim], 1)]  # noqa: E731
    q, k, v = parts(base)
    dq, dk, dv = parts(dev)
    inv = (10000.0 ** (-torch.arange(0, rot, 2).float() / rot)) if rot else None
    weights = [1.0 + 0.4 * torch.randn((h, dim) if per_head else (dim,), generator=g) if side in sides else None
               for side, h in (("q", hq), ("k", hkv))]
    if off:      # unaligned weights too
        dw = [None if w is None else torch.cat((torch.zeros(1), w.flatten())).to(DEV)[1:].view(w.shape) for w in weights]
    else:
        dw = [None if w is None else w.to(DEV) for w in weights]
    cu = [0] + [int(x) for x in np.cumsum(counts)]
    c = to_gpu(cache)
    print("append", seed, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved, off, sides, per_head, flush=True)
    out, guard = guarded((tokens, hq, dim), dtype)
    nv.kv_append(dk, dv, c, table.to(DEV), i32(lens), q=dq, cu_q=None if decode else i32(cu),
                 max_q=None if decode else max_q or max(counts), inv_freq=None if inv is None else inv.to(DEV),
                 interleaved=interleaved, out=out, q_norm=dw[0], k_norm=dw[1], eps=eps)
    guard()
    pos = torch.cat([torch.arange(f, f + n) for f, n in zip(firsts, counts)])
    qr = turned(normed(q, weights[0], eps), pos, inv, interleaved)
    kr = turned(normed(k, weights[1], eps), pos, inv, interleaved).float()
    taken = torch.cat([torch.arange(n) < (max_q or n) for n in counts])
    got, want = out.cpu().double()[taken], qr[taken]
    if not taken.all():
        assert (out.cpu().float()[~taken] == torch.tensor(-12345.0, dtype=dtype).float()).all()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.float().to(dtype).isinf())
    h = torch.finfo(dtype).eps / 2
    size = want.abs().nan_to_num().amax(-1, keepdim=True)
    step = h if dtype != F32 else 0.0
    tol = want.abs() * (step + 2.0 ** -24) * (1 + 2.0 ** -20) + 1e-12 * size + torch.finfo(dtype).smallest_normal * h
    err = torch.where(got.isfinite() & want.isfinite(), (got - want).abs() - tol, 0.0)
    assert err.max() <= 0, float(err.max())
    if dtype != F32:
        assert (got != want.float().to(dtype).double()).logical_and(want.isfinite()).sum() == 0
    after = [t.cpu() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    touched = torch.zeros(pages, dtype=torch.bool)
    for b, (f, n) in enumerate(zip(firsts, counts)):
        n = min(n, max_q or n)
        for i in range(f // page, -(-(f + n) // page) if n else f // page):
            pid = int(table[b, i])
            touched[pid] = True
            lo, hi = max(f, i * page), min(f + n, (i + 1) * page)
            held, rows = lo - i * page, slice(cu[b] + lo - f, cu[b] + hi - f)
            for head in range(hkv):
                for side, x in ((0, kr[rows, head].double()), (1, v[rows, head].double())):
                    fresh = scale_byte_of(float(torch.where(x.isfinite(), x.abs(), 0.0).max()))
                    old = int(before[2 + side][pid, head])
                    byte = max(fresh, old) if held else fresh
                    assert int(after[2 + side][pid, head]) == byte
                    was, now = before[side][pid, head], after[side][pid, head]
                    if side:
                        was, now = was.T, now.T
                    check_codes(now[held:held + hi - lo], x, byte)
                    if held and byte == old:
                        assert torch.equal(now[:held], was[:held])
                    elif held:
                        check_codes(now[:held], E4M3[was[:held].long()] * math.ldexp(1.0, old - 127), byte)
                    assert torch.equal(now[held + hi - lo:], was[held + hi - lo:])
    for t, u in zip(after, before):
        assert torch.equal(t[~touched], u[~touched])


CASES = [
    # dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved
    (BF16, 4, 2, 128, 64, [0, 63, 64, 1000], [1, 1, 1, 1], 128, False),
    (F16, 6, 1, 64, 16, [0, 5, 31], [40, 1, 18], 64, True),
    (F32, 2, 2, 256, 32, [7, 100], [60, 3], 128, False),
    (F32, 3, 3, 192, 256, [250, 0], [20, 300], 96, True),
    (BF16, 42, 6, 128, 128, [15], [260], 96, True),
    (BF16, 1, 1, 256, 256, [3], [510], 256, False),          # more tokens of a page than the lanes hold
    (F16, 8, 4, 128, 64, [0, 1, 0], [0, 0, 5], 0, False),     # no rotation; sequences without new tokens
    (F16, 2, 2, 64, 64, [70], [9], 10, False),                # pairs that no 16-byte access fits
    (BF16, 2, 1, 64, 32, [30], [40], 6, True),
    (F32, 1, 1, 64, 16, [100000], [3], 64, False),
    (F16, 5, 1, 192, 16, [2, 30], [17, 64], 192, False),
    (BF16, 3, 1, 256, 256, [0], [256], 0, True),
    (BF16, 4, 1, 64, 64, [9], [1100], 64, False),
    (F32, 1, 1, 64, 256, [60000], [300], 64, False),          # angles of far positions, turned on over eight rounds
    (F16, 2, 1, 128, 256, [20003], [400], 96, True),
]


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype,hq,hkv,dim,page,firsts,counts,rot,interleaved", CASES)
def test_norms(dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved, off, per_head):
    run(1, dtype, hq, hkv, dim, page, firsts, counts, rot, interleaved, off, per_head=per_head)


@pytest.mark.parametrize("sides", ["q", "k"])
@pytest.mark.parametrize("dtype,off", itertools.product([BF16, F16, F32], [0, 1]))
def test_one_side(sides, dtype, off):
    run(2, dtype, 6, 2, 128, 32, [5, 90], [70, 1], 128, off=off, sides=sides, per_head=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("loud", [-40.0, -12.0, 0.0, 40.0, 80.0])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-2])
def test_sizes_of_values(dtype, loud, eps):
    """Squares far below and above 32 bits' range, against eps that counts and that does not."""
    run(3, dtype, 4, 2, 64, 16, [3, 40], [20, 5], 64, loud=loud, eps=eps)


@pytest.mark.parametrize("dtype,off", [(BF16, 0), (F16, 1), (F32, 0), (F32, 1)])
def test_rows_of_zeros_infinities_and_nan(dtype, off):
    def edit(x):
        dim = 64
        x[2] = 0.0                                            # all heads' rows are zeros
        x[4, :dim] = 0.0
        x[5, 3], x[6, 70], x[7, 5 * dim - 1] = math.inf, -math.inf, math.nan
        x[8, 4 * dim + 1], x[9, 4 * dim + 40] = math.nan, math.inf     # keys
    run(4, dtype, 4, 2, 64, 16, [13], [12], 64, off=off, edit=edit)
    run(4, dtype, 4, 2, 64, 16, [13], [12], 0, off=off, edit=edit)


def test_zeros_without_eps_are_nan():
    run(5, BF16, 2, 1, 64, 16, [0], [6], 0, eps=0.0, edit=lambda x: x[3].zero_())


def test_one_token_each_and_rows_past_max_q():
    run(6, BF16, 8, 2, 128, 64, [5, 0, 130, 63], [1, 1, 1, 1], 128, decode=True)
    run(7, F16, 3, 1, 64, 16, [5, 33], [40, 9], 64, max_q=7)
    run(8, F32, 2, 1, 64, 16, [5, 700], [1500, 9], 32, interleaved=True, max_q=20)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_unit_weights_leave_normed_rows_to_the_plain_append(dtype, interleaved):
    """The norm of one side changes nothing of the other, bit for bit."""
    g = torch.Generator().manual_seed(9)
    base = torch.randn(50, 8 * 128, generator=g).to(dtype).to(DEV)
    q, k, v = (p.unflatten(1, (-1, 128)) for p in base.split([512, 256, 256], 1))
    table, lens, cu = i32([[3, 0, 1, 2]]), i32([100]), i32([0, 50])
    inv = 10000.0 ** (-torch.arange(0, 128, 2, device=DEV).float() / 128)
    ones = torch.ones(128, device=DEV)
    caches = [nv.KVCache.empty(4, 2, 32, 128) for _ in range(3)]
    call = lambda c, **n: nv.kv_append(k, v, c, table, lens, q=q, cu_q=cu, max_q=50, inv_freq=inv, interleaved=interleaved, **n)  # noqa: E731
    plain, only_k, only_q = call(caches[0]), call(caches[1], k_norm=ones), call(caches[2], q_norm=ones)
    assert torch.equal(plain, only_k) and not torch.equal(plain, only_q)
    assert torch.equal(caches[0].k, caches[2].k) and not torch.equal(caches[0].k, caches[1].k)
    assert torch.equal(caches[0].v, caches[1].v) and torch.equal(caches[0].v, caches[2].v)


def test_rows_of_no_sequence():
    """Rows behind the last sequence: queries are normed and stay where they are, keys go nowhere."""
    g = torch.Generator().manual_seed(11)
    for dtype, tokens in ((BF16, 30), (F32, 1300)):
        q, k = torch.randn(tokens, 3, 64, generator=g).to(dtype), torch.randn(tokens, 1, 64, generator=g).to(dtype)
        w = 1.0 + 0.3 * torch.randn(64, generator=g)
        inv = 10000.0 ** (-torch.arange(0, 64, 2).float() / 64)
        cache = nv.KVCache.empty(4, 1, 16, 64)
        out, guard = guarded((tokens, 3, 64), dtype)
        nv.kv_append(k.to(DEV), k.to(DEV), cache, i32([[2, 1], [0, 3]]), i32([20, 9]), q=q.to(DEV), cu_q=i32([0, 11, 13]),
                     max_q=11, inv_freq=inv.to(DEV), q_norm=w.to(DEV), k_norm=w.to(DEV), out=out)
        guard()
        pos = torch.cat((torch.arange(9, 20), torch.arange(7, 9), torch.zeros(tokens - 13, dtype=torch.long)))
        want = turned(normed(q, w, 1e-6), pos, inv, False).float().to(dtype)
        ulps = 0.0 if dtype != F32 else 2.0 ** -23
        assert ((out.cpu().double() - want.double()).abs() <= ulps * want.double().abs()).all()
        assert (cache.k[3] == 0).all() and (cache.k[1, :, 4:] == 0).all() and (cache.k[0, :, 9:] == 0).all()


def test_refusals():
    z = lambda *s, t=BF16: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    cache = nv.KVCache.empty(2, 2, 16, 64)
    k, q, table, lens = z(1, 2, 64), z(1, 4, 64), i32([[0]]), i32([1])
    for bad, error in [
        (dict(q_norm=z(64)), TypeError), (dict(q_norm=z(63, t=F32)), ValueError), (dict(q_norm=z(2, 64, t=F32)), ValueError),
        (dict(k_norm=z(4, 64, t=F32)), ValueError), (dict(k_norm=z(64, t=F32).cpu()), ValueError),
        (dict(k_norm=z(2, 128, t=F32)[:, ::2]), ValueError), (dict(k_norm=z(64, t=F32), eps=-1e-6), nv.NVFP4Error),
        (dict(k_norm=z(64, t=F32), eps=math.nan), nv.NVFP4Error), (dict(k_norm=z(64, t=F32), eps=math.inf), nv.NVFP4Error),
        (dict(q=None, q_norm=z(64, t=F32)), ValueError),
    ]:
        with pytest.raises(error):
            nv.kv_append(k, k, cache, table, lens, **{"q": q, **bad})

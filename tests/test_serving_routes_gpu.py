"""Routes of the serving operators that sizes choose, against the references and
tolerances of test_serving_gpu.py."""

import math

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV
from test_serving_gpu import BF16, E4M3, F16, F32, run_append, run_attention, run_sample

pytestmark = pytest.mark.gpu


# past 1024 tokens a block turns the queries of four rows: a last block of one
# to three, and sequences that begin and end inside a block
@pytest.mark.parametrize("dtype,dim,rot,interleaved,off", [
    (BF16, 64, 64, False, 0), (F16, 128, 96, True, 0), (F32, 64, 0, False, 0), (F16, 64, 32, False, 1),
    (BF16, 128, 128, True, 3), (F32, 64, 64, True, 1), (F16, 64, 10, False, 0), (BF16, 256, 256, False, 0)])
@pytest.mark.parametrize("counts", [[1025], [1, 2, 3, 0, 1030, 5, 6], [513, 514]])
def test_append_of_more_than_1024_tokens(dtype, dim, rot, interleaved, off, counts):
    firsts = [(37 * i) % 100 for i in range(len(counts))]
    run_append(31, dtype, 3, 1, dim, 64, firsts, counts, rot, interleaved, off=off)


@pytest.mark.parametrize("dtype,hq,hkv,dim,count,lens", [
    (BF16, 1, 1, 128, 40, [9000]), (F16, 2, 1, 64, 60, [20000]), (BF16, 4, 2, 192, 20, [12000]), (F16, 2, 1, 256, 33, [9500])])
def test_attention_of_many_rows_in_more_than_16_splits(dtype, hq, hkv, dim, count, lens):
    run_attention(32, dtype, hq, hkv, dim, 64, lens, [count])


@pytest.mark.parametrize("dtype,count,window", [(BF16, 1, 0), (F32, 1, 0), (F16, 40, 0), (BF16, 3, 100), (F16, 50, 300)])
def test_attention_with_a_table_far_wider_than_the_lengths(dtype, count, window):
    """As of a captured graph: the table holds the longest context that there may be."""
    run_attention(33, dtype, 8, 2, 128, 64, [1003, 70, 500, 64], [count] * 4, window=window, width=2048)


@pytest.mark.parametrize("dtype,vocab", [(BF16, 20000), (F16, 40000), (F32, 9000), (F32, 33000)])
def test_sample_of_130_rows(dtype, vocab):
    """From 128 rows on each runs in one block as long as its rounds allow."""
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(130, vocab, generator=g) * 2.5).to(dtype)
    u = torch.rand(130, generator=g).tolist()
    t = (torch.rand(130, generator=g) + 0.5).tolist()
    run_sample(x, u, t)
    run_sample(x, u, t, m=[0.05] * 130)
    run_sample(x, u, t, p=[0.9] * 130)


def e4m3(x):
    """The codes of x (at most 448), nearest, ties to even."""
    return x.float().to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("page,step,growth", [(16, 1, 2.5), (32, 3, 1.3), (64, 5, 0.8)])
def test_append_token_by_token(dtype, page, step, growth):
    """Pages that fill with ever larger values: each growth of the scale rounds
    the codes held so far anew, exactly as the definition in 64 bits."""
    g = torch.Generator().manual_seed(34)
    heads, dim, tokens = 2, 64, 2 * page + 3
    loud = (growth ** (torch.arange(tokens) % page)).clamp(2.0 ** -14, 2.0 ** 13)[:, None, None]
    k, v = ((torch.randn(tokens, heads, dim, generator=g).clamp(-3, 3) * loud).to(dtype) for _ in range(2))
    pages = -(-tokens // page)
    cache = nv.KVCache.empty(pages, heads, page, dim)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    codes = torch.zeros(2, pages, heads, page, dim, dtype=torch.uint8)
    scales = torch.zeros(2, pages, heads, dtype=torch.int64)
    for lo in range(0, tokens, step):
        hi = min(lo + step, tokens)
        nv.kv_append(k[lo:hi].to(DEV), v[lo:hi].to(DEV), cache, table, torch.tensor([hi], dtype=torch.int32, device=DEV),
                     cu_q=torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV))
        for p in range(lo // page, (hi - 1) // page + 1):
            a, b = max(lo, p * page), min(hi, (p + 1) * page)
            for side, x in enumerate((k, v)):
                for h in range(heads):
                    new = x[a:b, h].double()
                    m, e = math.frexp(float(new.abs().max()))      # amax = m 2^e, 448 = 0.875 * 2^9
                    byte = max(e - 9 + (m > 0.875) + 127, 0)
                    old = int(scales[side, p, h])
                    if a > p * page:
                        byte = max(byte, old)
                        if byte > old:
                            held = E4M3[codes[side, p, h, :a - p * page].long()] * math.ldexp(1.0, old - byte)
                            codes[side, p, h, :a - p * page] = e4m3(held)
                    codes[side, p, h, a - p * page:b - p * page] = e4m3(new * math.ldexp(1.0, 127 - byte))
                    scales[side, p, h] = byte
    assert torch.equal(cache.k.cpu(), codes[0])
    assert torch.equal(cache.v.cpu().transpose(2, 3), codes[1])
    assert torch.equal(cache.k_scales.cpu().long(), scales[0]) and torch.equal(cache.v_scales.cpu().long(), scales[1])

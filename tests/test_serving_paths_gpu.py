"""The serving operators' routes that depend on sizes and on what a row holds:
sampling in tiles, in one block and by digits, attention at the borders of the
kernels' tiles, and a decoder that uses all of them.  Tolerances are those of
test_serving_gpu.py."""

import math
import os
import sys

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV
from test_serving_gpu import BF16, F16, F32, make_cache, paging, run_attention, run_sample, to_gpu

pytestmark = pytest.mark.gpu


def filters(g, batch):
    u = torch.rand(batch, generator=g).tolist()
    t = (torch.rand(batch, generator=g) + 0.5).tolist()
    k = torch.randint(1, 300, (batch,), generator=g).tolist()
    p = (torch.rand(batch, generator=g) * 0.6 + 0.39).tolist()
    return u, t, k, p


# one block's rounds end at 65536 tokens of a 2-byte type and 32768 of float32
@pytest.mark.parametrize("dtype,vocab", [(F32, 32767), (F32, 32768), (F32, 32769), (BF16, 65536), (BF16, 65537),
                                         (F16, 65543), (F32, 98304), (BF16, 131072 + 1)])
def test_sample_around_the_tiles(dtype, vocab):
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(3, vocab, generator=g) * 2.5).to(dtype)
    x[1, : vocab // 2] = -math.inf
    x[2, :-1] = -math.inf                        # one token, the last
    u, t, k, p = filters(g, 3)
    run_sample(x, u)
    run_sample(x, u, t, k=k)
    run_sample(x, u, t, p=p)
    run_sample(x, u, t, k, p, [0.01, 0.0, 0.5])
    run_sample(x, u, m=[0.02, 2.0, 0.3])         # above 1: the first one alone


@pytest.mark.parametrize("vocab", [20000, 100000])
def test_sample_rows_with_too_many_in_a_bin(vocab):
    """Ties, few distinct values and nearly flat rows: the borders' bins hold
    more tokens than are gathered."""
    g = torch.Generator().manual_seed(vocab + 1)
    rows = torch.stack([torch.zeros(vocab), torch.randint(0, 5, (vocab,), generator=g).float(),
                        torch.randint(0, 2, (vocab,), generator=g) * -500.0, torch.randn(vocab, generator=g) * 1e-30,
                        torch.where(torch.arange(vocab) % 1000 == 7, 3.0, -3.0)])
    u, t, k, p = filters(g, 5)
    run_sample(rows, u, t, k=[2500, 3000, vocab - 1, 10, 50])
    run_sample(rows, u, t, p=p)
    run_sample(rows, u, t, [5000, 40, 7000, vocab // 2, 15], p)


@pytest.mark.parametrize("vocab", [30000, 150000])
def test_sample_masked_by_large_numbers(vocab):
    """Masks by a type's lowest value and by -100, a low temperature: they widen
    the row's range, not what is chosen."""
    g = torch.Generator().manual_seed(vocab + 2)
    for dtype in (F32, BF16, F16):
        x = (torch.randn(4, vocab, generator=g) * 2.5).to(dtype)
        x[0, ::3] = torch.finfo(dtype).min
        x[1, 1::2] = -100.0
        x[2, 100:] = torch.finfo(dtype).min
        x[3, 5] = math.nan
        u, t, k, p = filters(g, 4)
        run_sample(x, u, t, k, p)
        run_sample(x, u, [0.02, 0.05, 1.0, 0.0], k, p)


def test_sample_without_a_workspace():
    """The C entry without one: each row in one block, the same tokens."""
    lib = nv.load_library()
    g = torch.Generator().manual_seed(50)
    x = (torch.randn(2, 120000, generator=g) * 2.5).to(BF16).to(DEV)
    u = torch.rand(2, generator=g).to(DEV)
    k = torch.tensor([40, 0], dtype=torch.int32, device=DEV)
    p = torch.tensor([0.9, 0.8], device=DEV)
    want = nv.sample(x, u, top_k=k, top_p=p)
    token = torch.empty(2, dtype=torch.int32, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.nvfp4_sample(x.data_ptr(), 1, 2, 120000, 120000, u.data_ptr(), None, k.data_ptr(), p.data_ptr(), None,
                            None, 0, token.data_ptr(), None, stream) == 0
    assert torch.equal(token, want)
    want = nv.sample(x[:, :50000], u)            # tiles with one, a block without
    assert lib.nvfp4_sample(x.data_ptr(), 1, 2, 50000, 120000, u.data_ptr(), None, None, None, None, None, 0,
                            token.data_ptr(), None, stream) == 0
    assert torch.equal(token, want)


def test_sample_min_p_above_one_in_tiles():
    """Alone, without top-k and top-p: the first of the largest logits stays."""
    g = torch.Generator().manual_seed(52)
    x = torch.randn(3, 60000, generator=g)
    x[1, 30000], x[1, 50000] = 9.0, 9.0
    run_sample(x, [0.1, 0.9, 0.5], m=[1.5, 1.001, 0.5])


def test_sample_in_a_graph():
    """Tiles, gathering and counters repeat in replays, between eager calls."""
    g = torch.Generator().manual_seed(51)
    make = lambda: (torch.randn(2, 140000, generator=g) * 2.5).to(BF16).to(DEV)  # noqa: E731
    x, u = make(), torch.rand(2, device=DEV)
    p = torch.full((2,), 0.9, device=DEV)
    nv.sample(x, u, top_p=p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token = nv.sample(x, u, top_p=p)
    for _ in range(4):
        x.copy_(make())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, nv.sample(x, u, top_p=p))


@pytest.mark.parametrize("scale", [1e-30, 0.7, 3.0])
@pytest.mark.parametrize("dtype,counts", [(BF16, [1, 1]), (F16, [40, 33]), (F32, [5, 2])])
def test_attention_scales(dtype, counts, scale):
    run_attention(60, dtype, 4, 2, 64, 64, [200, 131], counts, scale=scale)


@pytest.mark.parametrize("dtype,count", [(BF16, 1), (F16, 40), (F32, 5)])
def test_attention_negative_scale(dtype, count):
    """The same bits as negated queries."""
    g = torch.Generator().manual_seed(65)
    table, pages = paging(g, [200], 64)
    cache, table = to_gpu(make_cache(g, pages, 2, 64, 64)), table.to(DEV)
    q = torch.randn(count, 4, 64, generator=g).to(dtype).to(DEV)
    lens, cu = (torch.tensor(n, dtype=torch.int32, device=DEV) for n in ([200], [0, count]))
    a = nv.paged_attention(q, cache, table, lens, cu_q=cu, scale=-0.3)
    assert torch.equal(a, nv.paged_attention(-q, cache, table, lens, cu_q=cu, scale=0.3))


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_attention_many_rows_pages(page, dim):
    """Tiles of one page and of several, ends inside a tile, a missing page."""
    def edit(cache, table):
        if table.shape[1] > 2:
            table[1, 1] = -1
    run_attention(61, BF16, 4, 1, dim, page, [257, 640, 63], [70, 129, 63], edit=edit)
    run_attention(62, F16, 4, 2, dim, page, [1000], [40], window=130)


@pytest.mark.parametrize("page", [16, 128])
def test_attention_few_rows_missing_pages_at_the_end(page):
    def edit(cache, table):
        table[0, -1] = -1
        table[1, 0] = 1 << 20
    run_attention(63, BF16, 8, 2, 128, page, [1030, 300], [1, 1], edit=edit, decode=True)
    run_attention(64, F32, 4, 2, 64, page, [1030, 300], [3, 2], window=100, edit=edit)


def test_attention_window_far_below_zero_is_none():
    lib = nv.load_library()
    c = nv.KVCache.empty(4, 1, 32, 64)
    c.v.fill_(0x38)                               # ones
    c.v_scales.fill_(127)
    q = torch.ones(1, 1, 64, device=DEV)
    out = torch.zeros_like(q)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([100], dtype=torch.int32, device=DEV)
    assert lib.nvfp4_paged_attention(c._ref, q.data_ptr(), 64, 64, 1, 0, 1, None, 1, 1,
                                     table.data_ptr(), 4, lens.data_ptr(), -(1 << 32) + 5, 0.125, None, 0,
                                     out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert (out == 1).all()
    c.v[0] = 0                                    # as a window of 5 the first page would have no part
    assert lib.nvfp4_paged_attention(c._ref, q.data_ptr(), 64, 64, 1, 0, 1, None, 1, 1,
                                     table.data_ptr(), 4, lens.data_ptr(), -(1 << 32) + 5, 0.125, None, 0,
                                     out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    # keys are all alike: 68 of 100 weights, to the sums' 32-bit roundings
    assert ((out - 0.68).abs() <= 100 * 2.0 ** -24).all()


def test_generate_example():
    """Tokens of the vocabulary, and the same ones again."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
    import generate
    prompts = [[1, 2, 3], list(range(70))]
    out = generate.generate(prompts, 5)
    assert out.shape == (2, 5) and out.dtype == torch.int32
    assert ((out >= 0) & (out < generate.VOCAB)).all()
    assert torch.equal(out, generate.generate(prompts, 5))

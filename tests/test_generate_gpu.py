"""The generation example over a pool of pages: whichever pages sequences have,
share, copy and give back, the tokens are those of caches that are never moved."""

import os
import sys

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import generate  # noqa: E402

pytestmark = pytest.mark.gpu

PROMPTS = [[1, 2, 3], list(range(100)), [7] * 65, list(range(50, 114))]


def apart(prompts, steps, seed=1, window=0, sinks=0, norm=False, samples=1):
    """The example's tokens with pages of its own for each sequence, given once and kept; samples get copies."""
    model = generate.Decoder(DEV, norm=norm, window=window, sinks=sinks)
    counts, n = [len(p) for p in prompts], len(prompts) * samples
    width = -(-(max(counts) + steps) // generate.PAGE)
    table = torch.randperm(n * width, generator=torch.Generator().manual_seed(5)).int().view(n, width).to(DEV)
    caches = [nv.KVCache.empty(n * width, generate.KV_HEADS, generate.PAGE, generate.DIM, DEV) for _ in range(generate.LAYERS)]
    u = torch.rand(steps, n, generator=torch.Generator().manual_seed(seed)).to(DEV)
    row = lambda value, dtype: torch.full((n,), value, dtype=dtype, device=DEV)  # noqa: E731
    settings = {"temperature": row(0.8, torch.float32), "top_k": row(50, torch.int32), "top_p": row(0.95, torch.float32)}
    ends = torch.tensor(counts).cumsum(0)
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), ends)).int().to(DEV)
    lens = torch.tensor(counts, dtype=torch.int32, device=DEV)
    own = torch.arange(len(prompts), device=DEV) * samples           # the rows whose pages the prompts are written to
    x = model(torch.tensor(sum(prompts, []), device=DEV), caches, table[own].contiguous(), lens, cu_q=cu, max_q=max(counts))
    parent = own.repeat_interleave(samples)
    for c in caches:
        for pages in (c.k, c.v, c.k_scales, c.v_scales):
            pages[table.flatten().long()] = pages[table[parent].flatten().long()]
    x, lens = x[(ends - 1).to(DEV)].repeat_interleave(samples, 0), lens.repeat_interleave(samples)
    out = []
    for i in range(steps):
        out.append(nv.sample(nv.qmm(x, *model.head), u[i], **settings))
        if i + 1 < steps:
            lens = lens + 1
            x = model(out[-1], caches, table, lens)
    return torch.stack(out, 1)


def test_pages_from_the_pool():
    assert torch.equal(generate.generate(PROMPTS, 70), apart(PROMPTS, 70))


@pytest.mark.parametrize("window,sinks", [(64, 4), (20, 0), (100, 70)])
def test_pages_behind_the_window_are_given_back(window, sinks):
    """A pool that holds little more than windows and sinks."""
    steps = 150
    most = sum(-(-len(p) // 64) for p in PROMPTS)                  # the prompts
    held = len(PROMPTS) * ((window + 62) // 64 + 1 + -(-sinks // 64))
    got = generate.generate(PROMPTS, steps, window=window, sinks=sinks, norm=True, pages=max(most, held) + 1)
    assert torch.equal(got, apart(PROMPTS, steps, window=window, sinks=sinks, norm=True))


def test_samples_share_their_prompt():
    """Three samples each, in fewer pages than they would fill apart."""
    got = generate.generate(PROMPTS, 70, samples=3, pages=32)
    assert torch.equal(got, apart(PROMPTS, 70, samples=3))
    assert torch.equal(generate.generate(PROMPTS, 90, samples=3, window=70, sinks=9), apart(PROMPTS, 90, samples=3, window=70, sinks=9))


def test_a_pool_that_is_too_small():
    with pytest.raises(RuntimeError, match="too small"):
        generate.generate(PROMPTS, 70, pages=7)


def test_a_decode_step_in_a_graph():
    """Freeing, reserving, normed appends and attention with sinks of both layers, captured on a stream of their own and
    replayed as lengths grow over pages, against the same steps run eagerly."""
    n, window, sinks, width, pages = 3, 40, 3, 6, 14
    model = generate.Decoder(DEV, norm=True, window=window, sinks=sinks)
    start = torch.tensor([5, 60, 100], dtype=torch.int32, device=DEV)

    def state():
        return {"caches": [nv.KVCache.empty(pages, generate.KV_HEADS, generate.PAGE, generate.DIM, DEV) for _ in range(generate.LAYERS)],
                "table": torch.full((n, width), -1, dtype=torch.int32, device=DEV),
                "refs": torch.zeros(pages, dtype=torch.int32, device=DEV), "lens": start.clone(),
                "tokens": torch.tensor([1, 2, 3], device=DEV)}

    def prefill(s):
        counts = start.tolist()
        cu = torch.tensor([0, 5, 65, 165], dtype=torch.int32, device=DEV)
        assert nv.kv_reserve(s["caches"], s["table"], s["lens"], s["refs"], cu_q=cu, tokens=165).tolist() == [0] * n
        model(torch.arange(165, device=DEV) % 97, s["caches"], s["table"], s["lens"], cu_q=cu, max_q=max(counts))

    def step(s):
        s["lens"].add_(1)
        nv.kv_free(s["table"], s["lens"], s["refs"], generate.PAGE, keep=window, sinks=sinks)
        missing = nv.kv_reserve(s["caches"], s["table"], s["lens"], s["refs"])
        x = model(s["tokens"], s["caches"], s["table"], s["lens"])
        s["tokens"].add_(1)
        return x, missing

    eager, captured = state(), state()
    prefill(eager), prefill(captured)
    warm = state()
    prefill(warm), step(warm)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        got, missing = step(captured)
    for i in range(150):
        graph.replay()
        torch.cuda.synchronize()
        want, _ = step(eager)
        assert torch.equal(got, want) and missing.tolist() == [0] * n, i
        assert torch.equal(captured["table"], eager["table"]) and torch.equal(captured["refs"], eager["refs"]), i
    for a, b in zip(captured["caches"], eager["caches"]):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert (eager["refs"] > 0).sum() <= n * 3          # sinks, and the one or two pages of a window

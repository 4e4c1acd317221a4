"""The generation example's handling of pages, without a GPU: the operators that
compute are stubs, those that keep the pages are their definitions on lists, and
the append checks that nothing is written where another sequence reads."""

import os
import sys

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from test_pages_gpu import ref_fork, ref_free, ref_reserve

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import generate  # noqa: E402

I32 = torch.int32


class Pool:
    """What stands in for the operators."""

    def __init__(self):
        self.refs, self.waited, self.appends = None, [], 0

    def kv_reserve(self, caches, table, lens, refs, cu_q=None, tokens=None):
        rows = table.shape[0]
        offsets = cu_q.tolist() if cu_q is not None else list(range(rows + 1))
        t, r, missing, _ = ref_reserve(table.tolist(), lens.tolist(), refs.tolist(), generate.PAGE, offsets, offsets[-1])
        table.copy_(torch.tensor(t))
        refs.copy_(torch.tensor(r))
        self.refs = refs
        self.waited.append(sum(m > 0 for m in missing))
        return torch.tensor(missing, dtype=I32)

    def kv_free(self, table, lens, refs, page, keep=0, sinks=0):
        t, r = ref_free(table.tolist(), lens.tolist(), refs.tolist(), page, keep, sinks)
        table.copy_(torch.tensor(t))
        refs.copy_(torch.tensor(r))

    def kv_fork(self, table, lens, refs, parent):
        t, n, r = ref_fork(table.tolist(), lens.tolist(), refs.tolist(), parent.tolist())
        refs.copy_(torch.tensor(r))
        return torch.tensor(t, dtype=I32), torch.tensor(n, dtype=I32)

    def kv_append(self, k, v, cache, table, lens, q=None, cu_q=None, **_):
        """Every new token has an entry that names a page which no other sequence has."""
        self.appends += 1
        new = cu_q.diff().tolist() if cu_q is not None else [1] * table.shape[0]
        for row, n, count in zip(table.tolist(), lens.tolist(), new):
            for t in range(max(n - count, 0), n):
                page = row[t // generate.PAGE]
                assert page >= 0, "a token without a page"
                assert self.refs[page] == 1, "a token for a page that another sequence reads"
        return q


@pytest.fixture
def pool(monkeypatch):
    p = Pool()
    zeros = lambda x, planes: torch.zeros(x.shape[0], planes.shape[0], dtype=x.dtype)  # noqa: E731
    for name, stub in {
        "quantize": lambda w: (w,), "qmm": zeros, "qmm_glu": lambda x, gate, up, act: zeros(x, gate),
        "paged_attention": lambda q, *_, **__: torch.zeros_like(q),
        "sample": lambda logits, u, **_: torch.zeros(logits.shape[0], dtype=I32),
        "kv_append": p.kv_append, "kv_reserve": p.kv_reserve, "kv_free": p.kv_free, "kv_fork": p.kv_fork,
    }.items():
        monkeypatch.setattr(nv, name, stub)
    monkeypatch.setattr(nv.KVCache, "empty", classmethod(lambda cls, *_: None))
    return p


PROMPTS = [list(range(64)), [1, 2, 3], list(range(100))]      # 4 pages; three samples of each: 9 pages more


@pytest.mark.parametrize("window", [0, 64])
def test_a_pool_that_is_large_enough(pool, window):
    assert generate.generate(PROMPTS, 5, samples=3, window=window, device="cpu", pages=13).shape == (9, 5)
    assert sum(pool.waited) == 0 and pool.appends == 5 * generate.LAYERS


@pytest.mark.parametrize("window", [0, 64])
@pytest.mark.parametrize("pages,waited", [(12, 1), (11, 2), (8, 5)])
def test_sequences_without_pages_wait(pool, pages, waited, window):
    """Their tokens are appended nowhere, neither without a page nor into the page that they share."""
    with pytest.raises(RuntimeError, match="too small"):
        generate.generate(PROMPTS, 5, samples=3, window=window, device="cpu", pages=pages)
    assert pool.waited[1] == waited and pool.appends == 5 * generate.LAYERS


def test_prompts_without_pages(pool):
    """Nothing is decoded from a prompt that is not in the cache."""
    with pytest.raises(RuntimeError, match="too small"):
        generate.generate(PROMPTS, 5, device="cpu", pages=3)
    assert pool.appends == 0

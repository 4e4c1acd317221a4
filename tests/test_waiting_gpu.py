"""Decoding from a pool that is too small: sequences that got no pages wait, and
the others go on as in a pool that is large enough, bit for bit."""

import os
import sys

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import generate  # noqa: E402

pytestmark = pytest.mark.gpu

HEADS, KV, PAGE, DIM = 4, 2, 16, 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Decode:
    """Two layers over one table; `held` is the token that the prompts have before they are forked."""

    def __init__(self, pages, held, parent, norm, new):
        g = torch.Generator().manual_seed(3)
        rnd = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
        self.norm = {side: (1 + 0.3 * rnd(DIM)).to(DEV) for side in ("q_norm", "k_norm")} if norm else {}
        self.new = new                                    # tokens of a step
        self.inv = (100.0 ** (-torch.arange(0, DIM, 2).float() / DIM)).to(DEV)
        self.caches = [nv.KVCache.empty(pages, KV, PAGE, DIM, DEV) for _ in range(2)]
        self.refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        table, lens = torch.full((len(held), 6), -1, dtype=torch.int32, device=DEV), i32(held)
        cu = [0]
        for n in held:
            cu.append(cu[-1] + n)
        assert not nv.kv_reserve(self.caches, table, lens, self.refs, cu_q=i32(cu), tokens=cu[-1]).any()
        for c in self.caches:
            k, v = (rnd(cu[-1], KV, DIM).bfloat16().to(DEV) for _ in range(2))
            nv.kv_append(k, v, c, table, lens, cu_q=i32(cu), inv_freq=self.inv)
        self.table, self.lens = nv.kv_fork(table, lens, self.refs, i32(parent))
        # louder with each step, so that pages' scales grow and their codes are rounded anew
        self.rows = [[4.0 ** step * rnd(len(parent) * new, HEADS + 2 * KV, DIM).bfloat16().to(DEV) for _ in range(2)] for step in range(3)]

    def step(self, i):
        """The outputs of both layers [sequences, new, heads, dim] and who waited."""
        n, new = self.lens.shape[0], self.new
        rows = {"cu_q": torch.arange(0, n * new + 1, new, dtype=torch.int32, device=DEV)}
        self.lens += new
        nv.kv_free(self.table, self.lens, self.refs, PAGE)
        waits = nv.kv_reserve(self.caches, self.table, self.lens, self.refs, tokens=n * new, **rows) > 0
        step, out = torch.where(waits, 0, self.lens), []
        for c, x in zip(self.caches, self.rows[i]):
            q, k, v = x.split([HEADS, KV, KV], 1)
            q = nv.kv_append(k, v, c, self.table, step, q=q, inv_freq=self.inv, max_q=new, **rows, **self.norm)
            out.append(nv.paged_attention(q, c, self.table, step, max_q=new, **rows).view(n, new, HEADS, DIM))
        self.lens -= new * waits.int()
        return torch.stack(out, 1), waits.tolist()

    def page(self, p):
        return [t[p].clone() for c in self.caches for t in (c.k, c.v, c.k_scales, c.v_scales)]


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("new", [1, 3])
@pytest.mark.parametrize("pages,waiting", [(4, [2, 3]), (5, [3]), (3, [1, 2, 3]), (2, [0, 1, 2, 3])])
def test_a_shared_page_stays_as_it_was(pages, waiting, new, norm):
    """Four samples of one prompt go on in its last page, which is half full; of the four copies that they need there are as
    many as free pages, two of the pool being in use."""
    small, ample = Decode(pages, [16 + 9], [0] * 4, norm, new), Decode(20, [16 + 9], [0] * 4, norm, new)
    shared = int(small.table[0, 1])
    before = small.page(shared)
    got, waits = small.step(0)
    want, none = ample.step(0)
    assert [b for b, w in enumerate(waits) if w] == waiting and not any(none)
    for b in range(4):
        if b in waiting:
            assert not got[b].any() and small.table[b].tolist() == [int(small.table[0, 0]), shared] + [-1] * 4
        else:
            assert torch.equal(got[b], want[b])
    for a, b in zip(small.page(shared), before):
        assert torch.equal(a, b)
    assert small.lens.tolist() == [25 if b in waiting else 25 + new for b in range(4)]


def test_who_waited_goes_on():
    """A sequence that gets its pages later has the outputs that it would have had."""
    small, ample = Decode(5, [12, 16], [0, 0, 1, 1], False, 1), Decode(20, [12, 16], [0, 0, 1, 1], False, 1)
    first, waits = small.step(0)
    want, _ = ample.step(0)
    assert waits == [False, False, False, True]        # two copies and two new pages, three of four
    assert torch.equal(first[:3], want[:3])
    second, waits = small.step(0)                      # sequence 3 with the same token, from the page that both copies left
    assert waits == [False] * 4 and torch.equal(second[3], want[3])


def test_the_example_lets_sequences_wait(monkeypatch):
    """Tokens of the sequences that never wait are those of a large pool."""
    prompts = [[1, 2, 3], list(range(100)), [7] * 65]
    want = generate.generate(prompts, 6, samples=3, pages=20)
    tokens, waits = [], []
    sample, reserve = nv.sample, nv.kv_reserve

    def recorded(*args, **kw):
        tokens.append(sample(*args, **kw))
        return tokens[-1]

    def watched(*args, **kw):
        missing = reserve(*args, **kw)
        waits.append((missing > 0).tolist())
        return missing

    monkeypatch.setattr(nv, "sample", recorded)
    monkeypatch.setattr(nv, "kv_reserve", watched)
    with pytest.raises(RuntimeError, match="too small"):
        generate.generate(prompts, 6, samples=3, pages=12)
    waited = torch.tensor(waits[1:]).any(0)
    assert 0 < waited.sum() < 9 and torch.tensor(waits[1]).sum() == 2
    assert torch.equal(torch.stack(tokens, 1).cpu()[~waited], want.cpu()[~waited])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("counts", [[100, 40, 70], [1, 3, 2]])
@pytest.mark.parametrize("width", [10, 200])                 # one share of the axis, or several
def test_prompts_wait(counts, width, norm, window, sinks, dtype):
    """Length 0 with new tokens: nothing of them is written, seen or changed for the others."""
    g = torch.Generator().manual_seed(11)
    pages, tokens = 40, sum(counts)
    table = torch.full((3, width), -1, dtype=torch.int32)
    table[:, :10] = torch.randperm(30, generator=g).view(3, 10).int()
    ample = table.clone()
    ample[1, :10] = torch.arange(30, 40)
    table[1, :8] = table[0, :8]                               # the one that waits shares pages with the first
    lens = i32([130, 120, 75])
    ends = torch.tensor(counts).cumsum(0).tolist()
    cu = i32([0] + ends)
    codes = lambda *shape: torch.randint(0, 120, shape, generator=g).to(torch.uint8).to(DEV)  # noqa: E731
    full = [codes(pages, KV, PAGE, DIM), codes(pages, KV, DIM, PAGE), codes(pages, KV), codes(pages, KV)]
    rows = torch.randn(tokens, HEADS + 2 * KV, DIM, generator=g).to(dtype).to(DEV)
    q, k, v = rows.split([HEADS, KV, KV], 1)
    weight = {"k_norm": (1 + torch.rand(DIM, generator=g)).to(DEV)} if norm else {}

    def run(table, step):
        caches = nv.KVCache(*[t.clone() for t in full])
        out = nv.kv_append(k, v, caches, table.to(DEV), step, q=q, cu_q=cu, max_q=max(counts), **weight)
        return nv.paged_attention(out, caches, table.to(DEV), step, cu_q=cu, max_q=max(counts), window=window, sinks=sinks), caches

    got, after = run(table, torch.where(i32([0, 1, 0]) > 0, 0, lens))
    want, others = run(ample, lens)
    for x, y in zip((after.k, after.v, after.k_scales, after.v_scales), (others.k, others.v, others.k_scales, others.v_scales)):
        assert torch.equal(x[:30], y[:30])
    waits = slice(ends[0], ends[1])
    assert want[waits].any() and not got[waits].any()
    assert torch.equal(got[:ends[0]], want[:ends[0]]) and torch.equal(got[ends[1]:], want[ends[1]:])

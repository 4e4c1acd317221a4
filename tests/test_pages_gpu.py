"""The pages' operators against plain implementations on the host: every
result is a whole number or a copy, and has to be equal."""

import itertools

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV, guarded

pytestmark = pytest.mark.gpu

I32 = torch.int32
FAR = 2 ** 31 - 1


def held(values, dtype=I32):
    """A device tensor inside a larger one whose surroundings must not change, and their check."""
    x = torch.as_tensor(values, dtype=dtype)
    view, check = guarded(tuple(x.shape), dtype)
    view.copy_(x)
    return view, check


# ---------------------------------------------------------------------------
# the definitions, on lists
# ---------------------------------------------------------------------------

def ref_free(table, lens, refs, page, keep, sinks):
    table, refs = [r[:] for r in table], refs[:]
    for row, n in zip(table, lens):
        for i, e in enumerate(row):
            needed = i * page < n and (keep <= 0 or (i + 1) * page > n - keep or i * page < sinks)
            if not needed and 0 <= e < len(refs):
                row[i] = -1
                refs[e] -= 1
    return table, refs


def ref_reserve(table, lens, refs, page, cu, tokens):
    """table, refs, missing and the copies (from, to)."""
    before, refs = refs[:], refs[:]
    table = [r[:] for r in table]
    free = [p for p, r in enumerate(refs) if r <= 0]
    missing, copies, taken = [], [], 0
    for b, row in enumerate(table):
        lo, hi = (min(max(c, 0), tokens) for c in (cu[b], cu[b + 1]))
        n, length = max(hi - lo, 0), max(lens[b], 0)
        first = max(length - n, 0)
        wants = [i for i in range(first // page, -(-length // page)) if n and i < len(row)
                 and not (0 <= row[i] < len(refs) and before[row[i]] <= 1)]
        taken += len(wants)
        missing.append(0 if taken <= len(free) else len(wants))
        if taken > len(free):
            continue
        for i, p in zip(wants, free[taken - len(wants):]):
            old = row[i]
            row[i], refs[p] = p, 1
            if 0 <= old < len(refs):
                refs[old] -= 1
                if i * page < first:
                    copies.append((old, p))
    return table, refs, missing, copies


def ref_fork(table, lens, refs, parent):
    refs = refs[:]
    out, lens_out = [], []
    for p in parent:
        ok = 0 <= p < len(table)
        out.append(table[p][:] if ok else [-1] * len(table[0]))
        lens_out.append(lens[p] if ok else 0)
    for rows, by in ((out, 1), (table, -1)):
        for e in itertools.chain(*rows):
            if 0 <= e < len(refs):
                refs[e] += by
    return out, lens_out, refs


def ref_compact(table, refs):
    inside = [p for p, r in enumerate(refs) if r > 0]
    used, refs = len(inside), refs[:]
    holes = [p for p in range(used) if refs[p] <= 0]
    where = [p if r > 0 else -1 for p, r in enumerate(refs)]
    copies = list(zip([p for p in inside if p >= used], holes))
    for a, b in copies:
        where[a], refs[b], refs[a] = b, refs[a], 0
    table = [[where[e] if 0 <= e < len(refs) else e for e in row] for row in table]
    return table, refs, used, where, copies


def counts(table, pages):
    refs = [0] * pages
    for e in itertools.chain(*table):
        if 0 <= e < pages:
            refs[e] += 1
    return refs


def make_caches(g, layers, pages, heads, page, dim):
    u8 = lambda *shape: torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8)  # noqa: E731
    return [(u8(pages, heads, page, dim), u8(pages, heads, dim, page), u8(pages, heads), u8(pages, heads))
            for _ in range(layers)]


def check_caches(got, was, copies):
    for c, before in zip(got, was):
        for x, y in zip((c.k, c.v, c.k_scales, c.v_scales), before):
            y = y.clone()
            for a, b in copies:
                y[b] = y[a]
            assert torch.equal(x.cpu(), y)


def scattered(g, lens, page, width, pages, share=()):
    """A table of random pages, one for each of `page` tokens; rows (a, b) in `share` have the same first pages."""
    order = torch.randperm(pages, generator=g).tolist()
    table = []
    for n in lens:
        need = min(-(-max(n, 0) // page), width)
        table.append([order.pop() for _ in range(need)] + [-1] * (width - need))
    for a, b, n in share:
        for e in table[b][:n]:
            if e >= 0:
                order.append(e)
        table[b][:n] = table[a][:n]
    return table


# ---------------------------------------------------------------------------
# freeing
# ---------------------------------------------------------------------------

def run_free(table, lens, pages, page, keep, sinks, refs=None):
    refs = counts(table, pages) if refs is None else refs
    t, check_t = held(table)
    r, check_r = held(refs)
    print("free", len(table), len(table[0]), pages, page, keep, sinks, flush=True)
    nv.kv_free(t, torch.tensor(lens, dtype=I32, device=DEV), r, page, keep=keep, sinks=sinks)
    check_t(), check_r()
    want = ref_free(table, lens, refs, page, keep, sinks)
    assert t.tolist() == want[0] and r.tolist() == want[1]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("keep,sinks", [(0, 0), (0, 70), (1, 0), (1, 1), (64, 0), (65, 64), (300, 17), (10 ** 6, 3), (FAR, 0),
                                        (2 ** 40, 5), (-5, 0), (100, 10 ** 12)])
def test_free(page, keep, sinks):
    g = torch.Generator().manual_seed(page + keep % 1000)
    lens = [1, 0, 1000, 999, 64, 65, 640, 1024, 129]
    table = scattered(g, lens, page, 70, 700)
    ended = [1, 0, 0, 998, 60, 65, 1, 1024, 0]       # some went back, some ended
    run_free(table, ended, 700, page, keep, sinks)


def test_free_of_a_table_that_holds_anything():
    g = torch.Generator().manual_seed(1)
    table = scattered(g, [500, 500, 500, 500], 16, 33, 200, [(0, 1, 20), (0, 2, 5)])
    table[3][:6] = [-1, -7, 200, FAR, -FAR - 1, table[3][5]]
    run_free(table, [0, 300, -5, 100], 200, 16, 0, 0)
    run_free(table, [FAR, FAR - 1, -FAR - 1, 100], 200, 16, 50, 20)
    run_free(table, [0, 0, 0, 0], 0, 16, 0, 0, [])                    # no pages: no entry names one
    run_free([[-1, 3]], [5], 4, 16, 0, 0)


@pytest.mark.parametrize("batch,width", [(1, 1), (1, 4097), (3, 1023), (5, 1024), (1025, 1), (1500, 3)])
def test_free_sizes(batch, width):
    g = torch.Generator().manual_seed(width)
    lens = torch.randint(0, width * 16 + 1, (batch,), generator=g).tolist()
    table = scattered(g, lens, 16, width, batch * width + 3)
    now = [n // 2 for n in lens]
    run_free(table, now, batch * width + 3, 16, 0, 0)
    run_free(table, lens, batch * width + 3, 16, 33, 20)


# ---------------------------------------------------------------------------
# sharing
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("given_out", [False, True])
@pytest.mark.parametrize("batch,width,parent", [
    (1, 1, [0]), (1, 5, [0, 0, 0, 0]), (4, 7, [3, 2, 1, 0]), (4, 7, [0, 1, 2, 3]), (4, 7, [1, 1, 1, 1]),
    (5, 1030, [4, -1, 5, FAR, 0, 0, -FAR - 1, 2]), (3, 2050, [2]), (2, 3, [-1, -1]), (3, 4, []), (600, 3, None),
])
def test_fork(batch, width, parent, given_out):
    g = torch.Generator().manual_seed(batch * 100 + width)
    if parent is None:
        parent = torch.randint(-1, batch + 1, (1300,), generator=g).tolist()
    lens = torch.randint(0, width * 16 + 1, (batch,), generator=g).tolist()
    pages = batch * width + 2
    table = scattered(g, lens, 16, width, pages, [(0, batch - 1, width // 2)] if batch > 1 else [])
    table[0][0] = pages                # names no page
    refs = counts(table, pages)
    refs[-1] += 3                      # counted by the caller too
    r, check_r = held(refs)
    out, check_out = guarded((len(parent), width), I32)
    t = torch.tensor(table, dtype=I32, device=DEV)
    got, got_lens = nv.kv_fork(t, torch.tensor(lens, dtype=I32, device=DEV), r,
                               torch.tensor(parent, dtype=I32, device=DEV), out=out if given_out else None)
    check_r(), check_out()
    want = ref_fork(table, lens, refs, parent)
    assert got.tolist() == want[0] and got_lens.tolist() == want[1] and r.tolist() == want[2]
    assert t.tolist() == table


def test_fork_without_entries():
    refs = torch.ones(3, dtype=I32, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=I32, device=DEV)  # noqa: E731
    table, lens = nv.kv_fork(torch.empty(2, 0, dtype=I32, device=DEV), i32([5, 6]), refs, i32([1, 0, 7]))
    assert table.shape == (3, 0) and lens.tolist() == [6, 5, 0] and refs.tolist() == [1, 1, 1]
    table, lens = nv.kv_fork(torch.empty(0, 4, dtype=I32, device=DEV), i32([]).int(), refs, i32([0]))
    assert table.tolist() == [[-1] * 4] and lens.tolist() == [0]


# ---------------------------------------------------------------------------
# reserving
# ---------------------------------------------------------------------------

def run_reserve(g, table, lens, pages, page, new=None, refs=None, layers=1, heads=1, dim=64, tokens=None, cu=None):
    refs = counts(table, pages) if refs is None else refs
    was = make_caches(g, layers, pages, heads, page, dim)
    caches = [nv.KVCache(*[x.to(DEV) for x in c]) for c in was]
    t, check_t = held(table)
    r, check_r = held(refs)
    offsets = cu
    if offsets is None and new is not None:
        offsets = [0] + list(itertools.accumulate(new))
    tokens = tokens if tokens is not None else offsets[-1] if offsets else len(table)
    print("reserve", len(table), len(table[0]), pages, page, lens[:8], (new or [])[:8], layers, heads, dim, flush=True)
    got = nv.kv_reserve(caches if layers > 1 else caches[0], t, torch.tensor(lens, dtype=I32, device=DEV), r,
                        cu_q=None if offsets is None else torch.tensor(offsets, dtype=I32, device=DEV),
                        tokens=None if offsets is None else tokens)
    check_t(), check_r()
    want = ref_reserve(table, lens, refs, page, offsets or list(range(len(table) + 1)), tokens)
    assert got.tolist() == want[2]
    assert t.tolist() == want[0] and r.tolist() == want[1]
    check_caches(caches, was, want[3])
    return want


@pytest.mark.parametrize("page,heads,dim,layers", [(16, 1, 64, 1), (32, 3, 192, 2), (64, 8, 128, 3), (128, 2, 256, 1),
                                                   (256, 5, 64, 2), (16, 2, 64, 70)])
def test_reserve_one_token_each(page, heads, dim, layers):
    g = torch.Generator().manual_seed(page)
    before = [page, page - 1, 3 * page, 0, 5, page + 1, 0]
    table = scattered(g, before, page, 5, 40, [(1, 6, 1)])
    before[6] = before[1]                       # shares the page that it goes on in
    want = run_reserve(g, table, [n + 1 for n in before], 40, page, layers=layers, heads=heads, dim=dim)
    assert len(want[3]) == 2


@pytest.mark.parametrize("page", [16, 64])
def test_reserve_ragged(page):
    g = torch.Generator().manual_seed(page)
    before = [0, 100, 100, 33, 64, 7, 0, 1000, 3]
    new = [500, 1, 0, 70, 64, 8, 0, 17, 1]
    table = scattered(g, before, page, 70, 300, [(1, 2, 7), (4, 5, 1)])
    before[2], before[5] = 100, min(page, 64)
    lens = [a + b for a, b in zip(before, new)]
    run_reserve(g, table, lens, 300, page, new)
    run_reserve(g, table, lens, 130, page, new, refs=counts(table, 300)[:130])   # a pool cut short: entries behind it name none
    run_reserve(g, table, lens, 300, page, new, tokens=600)             # rows behind the tokens are left out
    run_reserve(g, [r[:20] for r in table], lens, 300, page, new)       # lengths past the table


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 5, 8])
def test_reserve_from_too_few(spare):
    """Sequences are served in order as long as the sum of needs is there, whole or not at all."""
    g = torch.Generator().manual_seed(spare)
    before, new = [16, 10, 0, 32, 5, 48], [17, 3, 40, 0, 30, 16]
    table = scattered(g, before, 16, 6, 20, [(0, 1, 1)])
    refs = counts(table, 20)
    for p in [p for p in range(20) if refs[p] == 0][spare:]:
        refs[p] = 1                              # the caller's
    want = run_reserve(g, table, [a + b for a, b in zip(before, new)], 20, 16, new, refs)
    assert sum(want[2]) > 0


def test_reserve_many_entries_and_pages():
    """More entries than threads and more pages than a round looks at, scattered and aligned or not."""
    g = torch.Generator().manual_seed(7)
    pages = 40000
    refs = (torch.rand(pages, generator=g) < 0.9).int().tolist()
    new = [30000, 5, 0, 12000, 1]
    table = [[-1] * 2000 for _ in new]
    run_reserve(g, table, new, pages, 16, new, refs[:], dim=64)
    assert sum(r == 0 for r in refs) > sum(-(-n // 16) for n in new)
    refs = [1] * pages
    refs[-1500:] = [0] * 1500                     # the last ones alone, and too few of them
    run_reserve(g, table, new, pages, 16, new, refs)
    run_reserve(g, [[-1] for _ in range(3000)], [1] * 3000, 5000, 16)
    run_reserve(g, [[-1] for _ in range(3000)], [1] * 3000, 2000, 16)


def test_reserve_from_pools_that_are_counted_first():
    """Pools of more than 65536 pages: free ones in few rounds of 16384, in the last one, all over, and too few."""
    g = torch.Generator().manual_seed(8)
    pages = 150001
    for free in ([3, 16383, 16384, 70000, 70001, 131072, 150000], list(range(149990, 150001)), list(range(0, 150001, 97))):
        refs = [1] * pages
        for p in free:
            refs[p] = 0
        for new in ([16 * len(free) // 2, 5], [3, 1, 16 * len(free)]):
            run_reserve(g, [[-1] * 1600 for _ in new], new, pages, 16, new, refs[:])


def test_compact_to_the_border_of_a_round():
    """As many pages in use as one or two rounds have."""
    for used in (16384, 32768, 16383, 16385):
        g = torch.Generator().manual_seed(used)
        pages = 50000
        inside = sorted(torch.randperm(pages, generator=g)[:used].tolist())
        refs = [0] * pages
        for p in inside:
            refs[p] = 1
        was = make_caches(g, 1, pages, 1, 16, 64)
        cache = nv.KVCache(*[x.to(DEV) for x in was[0]])
        table = [inside[-5:], inside[:5]]
        t, r = torch.tensor(table, dtype=I32, device=DEV), torch.tensor(refs, dtype=I32, device=DEV)
        got, where = nv.kv_compact(cache, t, r)
        want = ref_compact(table, refs)
        assert got.item() == used == want[2] and where.tolist() == want[3]
        assert t.tolist() == want[0] and r.tolist() == want[1]
        check_caches([cache], was, want[4])


def test_tables_without_entries():
    i32 = lambda *shape: torch.zeros(shape, dtype=I32, device=DEV)  # noqa: E731
    cache, refs = nv.KVCache.empty(4, 1, 16, 64), i32(4)
    assert nv.kv_reserve(cache, i32(2, 0), i32(2) + 5, refs).tolist() == [0, 0]
    assert nv.kv_reserve(cache, i32(0, 3), i32(0), refs).tolist() == []
    nv.kv_free(i32(2, 0), i32(2), refs, 16)
    nv.kv_free(i32(0, 2), i32(0), refs, 16)
    none = nv.KVCache.empty(0, 1, 16, 64)
    used, where = nv.kv_compact(none, i32(2, 3), i32(0))
    assert used.item() == 0 and where.tolist() == [] and refs.tolist() == [0] * 4


def test_reserve_of_a_table_that_holds_anything():
    g = torch.Generator().manual_seed(3)
    table = scattered(g, [64, 64, 64, 64, 64], 16, 6, 30)
    table[0][4], table[1][4], table[2][4], table[3][3] = 30, FAR, -FAR - 1, -3
    lens = [65, 65, 70, 60, -4]
    run_reserve(g, table, lens, 30, 16)
    run_reserve(g, table, [FAR, FAR - 1, 96, 97, 0], 30, 16)
    run_reserve(g, table, lens, 30, 16, cu=[5, -3, 900, 2, 2, 4], tokens=7)
    run_reserve(g, table, [3, 3, 3, 3, 3], 30, 16, new=[9, 9, 9, 9, 9])       # more new tokens than the length
    refs = counts(table, 30)
    refs[table[0][0]], refs[29 if table[0][0] != 29 else 28] = 0, -4          # counts that do not match
    run_reserve(g, table, lens, 30, 16, refs=refs)
    run_reserve(g, [[-1, -1]] * 3, [1, 5, 17], 0, 16, refs=[])                # no pages at all


# ---------------------------------------------------------------------------
# compacting
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("pages,filled,layers,heads,page,dim", [
    (1, 0.0, 1, 1, 16, 64), (1, 1.0, 1, 1, 16, 64), (17, 0.5, 2, 3, 16, 64), (100, 0.9, 1, 2, 64, 192), (64, 1.0, 1, 1, 32, 64),
    (64, 0.0, 1, 1, 32, 64), (333, 0.3, 3, 1, 128, 128), (50, 0.6, 40, 1, 16, 64), (16384, 0.5, 1, 1, 16, 64),
    (16385, 0.7, 1, 1, 16, 64), (40007, 0.2, 1, 1, 16, 64), (60, 0.5, 1, 5, 256, 256), (49152, 0.9, 1, 1, 16, 64),
    (32768, 1.0, 1, 1, 16, 64), (32768, 0.0, 1, 1, 16, 64), (301, 0.5, 2, 3, 16, 64), (77, 0.4, 1, 3, 32, 192),
])
def test_compact(pages, filled, layers, heads, page, dim):
    g = torch.Generator().manual_seed(pages)
    inside = [p for p in range(pages) if torch.rand(1, generator=g).item() < filled]
    order = [inside[i] for i in torch.randperm(len(inside), generator=g).tolist()]
    width = max(3, len(order) // 3)
    table = [order[i * width:(i + 1) * width] for i in range(4)]
    table = [r + [-1] * (width - len(r)) for r in table]
    table[3][-2:] = [pages, FAR]
    table[2][-1] = table[0][0]
    refs = counts(table, pages)
    for p in order[4 * width:]:
        refs[p] += 1
    if pages > 20:
        refs[pages - 1] += 2                     # the caller's alone, perhaps
        refs[3] = -1 if refs[3] == 0 else refs[3]
    was = make_caches(g, layers, pages, heads, page, dim)
    caches = [nv.KVCache(*[x.to(DEV) for x in c]) for c in was]
    t, check_t = held(table)
    r, check_r = held(refs)
    print("compact", pages, filled, layers, heads, page, dim, flush=True)
    used, where = nv.kv_compact(caches, t, r)
    check_t(), check_r()
    want = ref_compact(table, refs)
    assert used.tolist() == [want[2]] and where.tolist() == want[3]
    assert t.tolist() == want[0] and r.tolist() == want[1]
    check_caches(caches, was, want[4])


def test_compact_without_a_table():
    g = torch.Generator().manual_seed(2)
    was = make_caches(g, 1, 9, 1, 16, 64)
    cache = nv.KVCache(*[x.to(DEV) for x in was[0]])
    refs = torch.tensor([0, 1, 0, 0, 2, 0, 0, 0, 5], dtype=I32, device=DEV)
    used, where = nv.kv_compact(cache, torch.empty(0, 4, dtype=I32, device=DEV), refs)
    assert used.item() == 3 and refs.tolist() == [2, 1, 5, 0, 0, 0, 0, 0, 0]
    assert where.tolist() == [-1, 1, -1, -1, 0, -1, -1, -1, 2]
    check_caches([cache], was, [(4, 0), (8, 2)])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(4))
def test_a_life_of_a_pool(seed):
    """Sequences come, grow, fork, lose what is behind a window, end; the pool is compacted now and then."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    page, pages, width, rows = 16, 60, 12, 6
    was = make_caches(g, 2, pages, 1, page, 64)
    caches = [nv.KVCache(*[x.to(DEV) for x in c]) for c in was]
    table, lens, refs = [[-1] * width for _ in range(rows)], [0] * rows, [0] * pages
    t = torch.full((rows, width), -1, dtype=I32, device=DEV)
    r = torch.zeros(pages, dtype=I32, device=DEV)
    keep, sinks = (0, 0) if seed % 2 else (50, 5)
    for _ in range(40):
        new = [rnd(0, 20) if n + 20 <= width * page else 0 for n in lens]
        lens = [a + b for a, b in zip(lens, new)]
        if rnd(0, 3) == 0:
            i = rnd(0, rows - 1)
            lens[i] = new[i] = 0
        dl = torch.tensor(lens, dtype=I32, device=DEV)
        nv.kv_free(t, dl, r, page, keep=keep, sinks=sinks)
        table, refs = ref_free(table, lens, refs, page, keep, sinks)
        cu = [0] + list(itertools.accumulate(new))
        missing = nv.kv_reserve(caches, t, dl, r, cu_q=torch.tensor(cu, dtype=I32, device=DEV), tokens=cu[-1])
        table, refs, lack, copies = ref_reserve(table, lens, refs, page, cu, cu[-1])
        assert missing.tolist() == lack
        for c in was:
            for x in c:
                for a, b in copies:
                    x[b] = x[a]
        lens = [n - m if k else n for n, m, k in zip(lens, new, lack)]
        if rnd(0, 2) == 0:
            parent = [rnd(-1, rows - 1) if rnd(0, 2) == 0 else i for i in range(rows)]
            t, dl = nv.kv_fork(t, torch.tensor(lens, dtype=I32, device=DEV), r, torch.tensor(parent, dtype=I32, device=DEV))
            table, lens, refs = ref_fork(table, lens, refs, parent)
            assert dl.tolist() == lens
        if rnd(0, 5) == 0:
            used, _ = nv.kv_compact(caches, t, r)
            table, refs, n, _, copies = ref_compact(table, refs)
            assert used.item() == n
            for c in was:
                for x in c:
                    for a, b in copies:
                        x[b] = x[a]
        assert t.tolist() == table and r.tolist() == refs and refs == counts(table, pages)
    check_caches(caches, was, [])


def test_offsets_past_32_bits():
    """Caches of more than 4 GiB: pages at their ends are copied."""
    pages, heads, page, dim = 1100, 64, 256, 256             # 4.3 GiB a side
    z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=DEV)  # noqa: E731
    cache = nv.KVCache(z(pages, heads, page, dim), z(pages, heads, dim, page), z(pages, heads), z(pages, heads))
    g = torch.Generator().manual_seed(0)
    part = make_caches(g, 1, 1, heads, page, dim)[0]
    for x, y in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), part):
        x[pages - 2] = y[0].to(DEV)
    table = torch.tensor([[pages - 2], [pages - 2]], dtype=I32, device=DEV)
    refs = torch.ones(pages, dtype=I32, device=DEV)
    refs[pages - 2], refs[pages - 1] = 2, 0
    refs[5] = 0
    missing = nv.kv_reserve(cache, table, torch.tensor([7, 9], dtype=I32, device=DEV), refs)
    assert missing.tolist() == [0, 0] and table.tolist() == [[5], [pages - 1]]
    for x, y in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), part):
        assert torch.equal(x[5].cpu(), y[0]) and torch.equal(x[pages - 1].cpu(), y[0])


def test_refusals():
    i32 = lambda *shape: torch.zeros(shape, dtype=I32, device=DEV)  # noqa: E731
    table, lens, refs = i32(2, 3), i32(2), i32(8)
    cache = nv.KVCache.empty(8, 1, 16, 64)
    for call, error in [
        (lambda: nv.kv_free(table.float(), lens, refs, 16), TypeError),
        (lambda: nv.kv_free(table, lens.long(), refs, 16), TypeError),
        (lambda: nv.kv_free(table, lens, refs, 48), ValueError),
        (lambda: nv.kv_free(table, i32(3), refs, 16), ValueError),
        (lambda: nv.kv_free(table.t(), i32(3), refs, 16), ValueError),
        (lambda: nv.kv_free(table, lens.cpu(), refs, 16), ValueError),
        (lambda: nv.kv_free(table[0], lens, refs, 16), ValueError),
        (lambda: nv.kv_fork(table, lens, refs, i32(2, 1)), ValueError),
        (lambda: nv.kv_fork(table, lens, refs, i32(2), out=i32(2, 4)), ValueError),
        (lambda: nv.kv_fork(table, lens, refs, i32(2), out=table), nv.NVFP4Error),
        (lambda: nv.kv_reserve([], table, lens, refs), ValueError),
        (lambda: nv.kv_reserve([cache, nv.KVCache.empty(8, 2, 16, 64)], table, lens, refs), ValueError),
        (lambda: nv.kv_reserve(cache, table, lens, i32(9)), ValueError),
        (lambda: nv.kv_reserve(cache, table, lens, refs, cu_q=i32(3)), ValueError),
        (lambda: nv.kv_reserve(cache, table, lens, refs, tokens=3), ValueError),
        (lambda: nv.kv_reserve(cache, table, lens, refs, cu_q=i32(2), tokens=2), ValueError),
        (lambda: nv.kv_reserve(cache, table, lens, refs, cu_q=i32(3), tokens=-1), nv.NVFP4Error),
        (lambda: nv.kv_compact(cache, table, i32(7)), ValueError),
    ]:
        with pytest.raises(error):
            call()


def test_in_a_graph_and_on_another_stream():
    """A step of freeing, reserving and forking, captured on a side stream and replayed over moving lengths."""
    g = torch.Generator().manual_seed(4)
    page, pages, rows, width = 16, 64, 4, 10
    was = make_caches(g, 2, pages, 1, page, 64)
    caches = [nv.KVCache(*[x.to(DEV) for x in c]) for c in was]
    start = scattered(g, [20, 16, 40, 3], page, width, pages, [(0, 1, 1)])
    t = torch.tensor(start, dtype=I32, device=DEV)
    r = torch.tensor(counts(start, pages), dtype=I32, device=DEV)
    lens = torch.tensor([20, 16, 40, 3], dtype=I32, device=DEV)
    parent = torch.tensor([0, 1, 0, 3], dtype=I32, device=DEV)
    out = torch.empty_like(t)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()

    def step():
        lens.add_(1)
        nv.kv_free(t, lens, r, page, keep=30, sinks=4)
        missing = nv.kv_reserve(caches, t, lens, r)
        _, forked = nv.kv_fork(t, lens, r, parent, out=out)
        t.copy_(out)
        lens.copy_(forked)
        return missing

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        missing = step()
    table, n, refs = start, [20, 16, 40, 3], counts(start, pages)
    for i in range(25):
        graph.replay()
        torch.cuda.synchronize()
        n = [x + 1 for x in n]
        table, refs = ref_free(table, n, refs, page, 30, 4)
        table, refs, lack, copies = ref_reserve(table, n, refs, page, list(range(rows + 1)), rows)
        for c in was:
            for x in c:
                for a, b in copies:
                    x[b] = x[a]
        table, n, refs = ref_fork(table, n, refs, [0, 1, 0, 3])
        assert missing.tolist() == lack and t.tolist() == table and r.tolist() == refs and lens.tolist() == n, i
        check_caches(caches, was, [])
        torch.randn(1000, device=DEV).sum().item()      # other work between replays

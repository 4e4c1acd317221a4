"""Reserving for more sequences than a block has threads, all of them going on
in pages that they share: what the entries held, their counts and the copies are
then worked out anew past the first 1024."""

import pytest
import torch

from test_pages_gpu import counts, run_reserve

pytestmark = pytest.mark.gpu

BATCH, GROUP = 1500, 3


def shared_table(g, pages, width, before, page):
    """Sequences in groups of three that share all pages of their tokens, and the free pages."""
    order = torch.randperm(pages, generator=g).tolist()
    table = []
    for b in range(BATCH):
        if b % GROUP == 0:
            row = [order.pop() for _ in range(-(-before // page))]
            row += [-1] * (width - len(row))
        table.append(row[:])
    return table, len(order)


# new tokens, whether with offsets, tokens before, bytes of a page, pages of the pool
CASES = [(1, False, 9, 1, 2100), (1, True, 9, 1, 2100), (3, True, 30, 1, 6000), (20, True, 9, 1, 6000), (1, False, 9, 1, 70000),
         (1, False, 70, 16, 2600)]


@pytest.mark.parametrize("short", [0, 1, 200, 1400])
@pytest.mark.parametrize("new,offsets,before,size,pages", CASES)
def test_sequences_go_on_in_shared_pages(new, offsets, before, size, pages, short):
    """short: free pages that are missing; the last sequences are not served then."""
    g = torch.Generator().manual_seed(new + size)
    page, heads, dim = (64, 2, 128) if size == 16 else (16, 1, 64)       # 16 or 1 KB a side
    width = -(-(before + new) // page) + 1
    table, free = shared_table(g, pages, width, before, page)
    lens = [before + new] * BATCH
    need = BATCH * (-(-(before + new) // page) - before // page)
    refs = counts(table, pages)
    spare = [p for p in range(pages) if refs[p] == 0][need - short:]
    assert len(spare) == free - need + short
    for p in spare:
        refs[p] = 1                                                      # the caller's
    _, _, missing, copies = run_reserve(g, table, lens, pages, page, [new] * BATCH if offsets else None, refs, heads=heads, dim=dim)
    served = sum(m == 0 for m in missing)
    each = need // BATCH
    assert served == BATCH - -(-short // each) and len(copies) == served

"""Limits of the serving operators' launches, checked before anything is
enqueued: every call here is refused."""

import pytest

from test_serving_host import BF16, FAKE, GRID, SHAPE, append, attention, cache, lib  # noqa: F401

FAR = 1 << 42     # never dereferenced; apart from each other, so that nothing overlaps


def apart(heads=2, page=64):
    return cache(k=FAR, v=2 * FAR, heads=heads, page=page)


@pytest.mark.parametrize("sizes", [
    dict(tokens=1 << 20, batch=1 << 12, max_q=1 << 18),              # 4096 tiles of rows each: 2^25 blocks
    dict(tokens=1 << 20, batch=1 << 20, max_q=1 << 3),               # one each
    dict(tokens=1 << 25, batch=1, max_q=1, hq=2, width=1 << 16),     # 2^26 rows that a split axis would join
])
def test_attention_grids_in_threads(lib, sizes):  # noqa: F811
    """A dimension holds less than 2^32 threads, 2^24 blocks of 256."""
    sizes = {**dict(hq=64, qt=64 * 128), **sizes}
    assert attention(lib, c=apart(heads=2 if sizes["hq"] == 2 else 32), out=4 * FAR, **sizes) == GRID


@pytest.mark.parametrize("heads_q", [(1 << 20) + 1, (1 << 24) - 1, 1 << 27])
def test_append_query_heads(lib, heads_q):  # noqa: F811
    """4 tokens of 2^24 heads and more have more items than a 32-bit index counts."""
    assert append(lib, c=apart(), tokens=1, batch=1, max_q=1, hq=heads_q, out=4 * FAR, q=8 * FAR) == SHAPE


@pytest.mark.parametrize("sizes,heads", [
    (dict(tokens=1 << 18, batch=2, max_q=1 << 18), 4096),
    (dict(tokens=1 << 18, batch=1 << 18, max_q=1), 32),
    (dict(tokens=1 << 18, batch=1 << 22, max_q=1), 2),
])
def test_append_grids_in_threads(lib, sizes, heads):  # noqa: F811
    assert append(lib, c=apart(heads=heads), kt=heads * 128, vt=heads * 128, out=4 * FAR, q=8 * FAR, **sizes) == GRID

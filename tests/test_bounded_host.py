"""Host-side checks of the append with norms and of attention with sinks that
need no GPU: every call here is refused, or is a no-op, before anything is
launched."""

import ctypes
import math

import pytest

from test_serving_host import ALIGN, BF16, DTYPE, FAKE, GRID, OK, SHAPE, UNSUP, cache, lib  # noqa: F401

FAR = 1 << 42     # never dereferenced; apart from each other, so that nothing overlaps


def append(lib, c=None, hq=4, q=3 * FAR, out=4 * FAR, tokens=3, qn=5 * FAR, qn_head=0, kn=6 * FAR, kn_head=0, eps=1e-6, rot=128, dt=BF16):  # noqa: F811
    c = c or cache(k=FAR, v=2 * FAR)
    return lib.nvfp4_kv_append_norm(ctypes.addressof(c), FAKE, 256, 128, FAKE, 256, 128, q, 512, 128, hq, out, dt, tokens, FAKE,
                                    2, 2, FAKE, 4, FAKE, FAKE, rot, 0, qn, qn_head, kn, kn_head, eps, None)


def attention(lib, c=None, dt=BF16, tokens=3, width=4, window=100, sinks=4, ws=None, ws_bytes=0, hq=4):  # noqa: F811
    c = c or cache(k=FAR, v=2 * FAR)
    return lib.nvfp4_paged_attention_sinks(ctypes.addressof(c), FAKE, 512, 128, hq, dt, tokens, FAKE, 2, 2, FAKE, width, FAKE,
                                           window, sinks, 1.0, ws, ws_bytes, 4 * FAR, None)


@pytest.mark.parametrize("bad,status", [
    (dict(eps=-1e-9), SHAPE), (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE), (dict(qn=5 * FAR + 2), ALIGN),
    (dict(kn=6 * FAR + 1), ALIGN), (dict(qn_head=64), SHAPE), (dict(kn_head=-128), SHAPE), (dict(kn_head=1), SHAPE),
    (dict(q=None, out=None), SHAPE), (dict(out=5 * FAR - 64), SHAPE), (dict(out=6 * FAR - 64), SHAPE),
    (dict(qn_head=128, out=5 * FAR + 4 * 128 * 3), SHAPE), (dict(kn_head=128, out=6 * FAR + 128 * 4 + 16), SHAPE),
    (dict(rot=130), SHAPE), (dict(dt=9), DTYPE), (dict(hq=(1 << 20) + 1), SHAPE),
])
def test_append_refusals(lib, bad, status):  # noqa: F811
    assert append(lib, **bad) == status


def test_append_without_tokens(lib):  # noqa: F811
    assert append(lib, tokens=0) == OK
    assert append(lib, tokens=0, qn=None, kn=None, qn_head=7) == OK     # strides of weights that are not there


@pytest.mark.parametrize("bad,status", [
    (dict(dt=7), DTYPE), (dict(hq=3), SHAPE), (dict(tokens=-1), SHAPE), (dict(ws_bytes=-1), SHAPE), (dict(ws_bytes=64), SHAPE),
    (dict(ws=FAKE + 8, ws_bytes=64), ALIGN), (dict(width=-1), SHAPE), (dict(width=1 << 25), SHAPE),
])
def test_attention_refusals(lib, bad, status):  # noqa: F811
    assert attention(lib, **bad) == status


def test_attention_workspace(lib):  # noqa: F811
    size = lib.nvfp4_paged_attention_sinks_workspace_size
    plain = lib.nvfp4_paged_attention_workspace_size
    for sizes in ((1, 32, 8, 128, 64, 1, 1, 2000), (64, 16, 2, 128, 64, 64, 1, 128), (4096, 8, 8, 64, 64, 1, 4096, 64)):
        for window in (0, 100, 4096, 1 << 40):
            assert size(*sizes, window, 0, BF16) == size(*sizes, window, -5, BF16) == plain(*sizes, window, BF16)
            assert size(*sizes, window, 1 << 50, BF16) >= 0
        assert size(*sizes, 0, 500, BF16) == plain(*sizes, 0, BF16)           # no window: the sinks say nothing
    assert size(1, 32, 8, 128, 48, 1, 1, 2000, 100, 4, BF16) == UNSUP
    assert size(1, 31, 8, 128, 64, 1, 1, 2000, 100, 4, BF16) == SHAPE
    assert size(1, 32, 8, 128, 64, 1, 1, 2000, 100, 4, 3) == DTYPE


def test_attention_grid(lib):  # noqa: F811
    c = cache(k=FAR, v=2 * FAR, heads=32)
    assert lib.nvfp4_paged_attention_sinks(ctypes.addressof(c), FAKE, 64 * 128, 128, 64, BF16, 1 << 20, FAKE, 1 << 12, 1 << 18,
                                           FAKE, 4, FAKE, 100, 4, 1.0, None, 0, 4 * FAR, None) == GRID

"""Host-side checks of the pages' operators that need no GPU: every call here
is refused, or is a no-op, before anything is launched."""

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from nvfp4_quantized_matmul_amd.serving import _CacheStruct

OK, NULLPTR, SHAPE, UNSUP, ALIGN = 0, -1, -2, -6, -8
A = 1 << 32          # addresses that are never dereferenced, far apart
TABLE, LENS, REFS, CU, WS, MISSING, PARENT, OUT, LENS_OUT, USED, WHERE = (A * i for i in range(8, 19))


@pytest.fixture(scope="module")
def lib():
    return nv.load_library()


def caches(n=1, **changed):
    base = dict(k=A, v=2 * A, k_scales=3 * A, v_scales=4 * A, pages=8, heads=2, page=64, dim=128)
    return (_CacheStruct * n)(*[_CacheStruct(**(dict(base, **changed) if i == n - 1 else base)) for i in range(n)])


def free(lib, table=TABLE, batch=2, width=4, lens=LENS, page=64, keep=0, sinks=0, refs=REFS, pages=8):
    return lib.nvfp4_kv_free(table, batch, width, lens, page, keep, sinks, refs, pages, None)


def reserve(lib, c=None, count=1, table=TABLE, batch=2, width=4, lens=LENS, cu=CU, tokens=3, refs=REFS, ws=WS,
            ws_bytes=1 << 20, missing=MISSING):
    return lib.nvfp4_kv_reserve(c or caches(), count, table, batch, width, lens, cu, tokens, refs, ws, ws_bytes, missing, None)


def fork(lib, table=TABLE, batch=2, width=4, lens=LENS, parent=PARENT, rows=3, refs=REFS, pages=8, out=OUT,
         lens_out=LENS_OUT):
    return lib.nvfp4_kv_fork(table, batch, width, lens, parent, rows, refs, pages, out, lens_out, None)


def compact(lib, c=None, count=1, table=TABLE, batch=2, width=4, refs=REFS, ws=WS, ws_bytes=1 << 20, used=USED, where=WHERE):
    return lib.nvfp4_kv_compact(c or caches(), count, table, batch, width, refs, ws, ws_bytes, used, where, None)


TABLE_REFUSALS = [
    (dict(batch=-1), SHAPE), (dict(width=-1), SHAPE), (dict(batch=1 << 20, width=1 << 12), SHAPE),
    (dict(batch=1 << 31), SHAPE), (dict(table=None), NULLPTR), (dict(refs=None), NULLPTR), (dict(table=TABLE + 2), ALIGN),
    (dict(refs=REFS + 1), ALIGN), (dict(refs=TABLE + 16), SHAPE), (dict(width=1 << 62, batch=4), SHAPE),
]


@pytest.mark.parametrize("call", [free, reserve, fork, compact])
@pytest.mark.parametrize("bad,status", TABLE_REFUSALS)
def test_table_refusals(lib, call, bad, status):
    assert call(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(page=48), UNSUP), (dict(page=0), UNSUP), (dict(pages=-1), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(lens=None), NULLPTR), (dict(lens=LENS + 2), ALIGN), (dict(lens=TABLE + 4), SHAPE), (dict(lens=REFS), SHAPE),
    (dict(width=1 << 25), SHAPE),
])
def test_free_refusals(lib, bad, status):
    assert free(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(count=0), SHAPE), (dict(count=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(cu=None), SHAPE), (dict(lens=None), NULLPTR), (dict(missing=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(ws=WS + 8), ALIGN), (dict(ws_bytes=16), SHAPE), (dict(cu=CU + 1), ALIGN), (dict(missing=MISSING + 1), ALIGN),
    (dict(missing=LENS), SHAPE), (dict(missing=CU + 4), SHAPE), (dict(ws=TABLE + 16), SHAPE), (dict(lens=REFS + 4), SHAPE),
    (dict(batch=0, cu=None), SHAPE), (dict(width=1 << 25), SHAPE), (dict(batch=1 << 30, width=1), SHAPE),
])
def test_reserve_refusals(lib, bad, status):
    assert reserve(lib, **bad) == status


@pytest.mark.parametrize("call", [reserve, compact])
@pytest.mark.parametrize("bad,status", [
    (dict(page=48), UNSUP), (dict(dim=80), UNSUP), (dict(k=None), NULLPTR), (dict(v=2 * A + 8), ALIGN),
    (dict(pages=9), SHAPE), (dict(heads=3), SHAPE), (dict(page=32), SHAPE), (dict(dim=64), SHAPE), (dict(heads=0), SHAPE),
])
def test_cache_refusals(lib, call, bad, status):
    assert call(lib, c=caches(3, **bad), count=3) == status
    assert call(lib, c=caches(1, k_scales=None)) == NULLPTR
    assert call(lib, c=caches(1, heads=(1 << 19) + 1)) == SHAPE


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(parent=None), NULLPTR),
    (dict(out=None), NULLPTR), (dict(lens_out=None), NULLPTR), (dict(lens=None), NULLPTR), (dict(parent=PARENT + 2), ALIGN),
    (dict(out=OUT + 1), ALIGN), (dict(out=TABLE), SHAPE), (dict(out=TABLE + 16), SHAPE), (dict(lens_out=LENS), SHAPE),
    (dict(lens_out=PARENT), SHAPE), (dict(parent=OUT + 32), SHAPE), (dict(pages=-1), SHAPE),
])
def test_fork_refusals(lib, bad, status):
    assert fork(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(count=0), SHAPE), (dict(used=None), NULLPTR), (dict(where=None), NULLPTR), (dict(ws=None), NULLPTR),
    (dict(ws_bytes=15), SHAPE), (dict(ws=WS + 4), ALIGN), (dict(where=REFS), SHAPE), (dict(used=WHERE + 8), SHAPE),
    (dict(where=WHERE + 2), ALIGN), (dict(ws=REFS + 16), SHAPE),
])
def test_compact_refusals(lib, bad, status):
    assert compact(lib, **bad) == status


def test_nothing_to_do(lib):
    assert free(lib, batch=0) == OK and free(lib, width=0, table=None) == OK
    assert free(lib, batch=0, table=None, refs=None, pages=0, lens=None) == OK
    assert reserve(lib, batch=0, tokens=0) == OK
    assert fork(lib, batch=0, rows=0, table=None, out=None, parent=None, lens=None, lens_out=None) == OK


def test_workspace_sizes(lib):
    size = lib.nvfp4_kv_reserve_workspace_size
    assert size(64, 64, 64, 100) >= (4 + 2 * 64 + 2 * (64 + 2 * 64 // 64) + 1) * 4
    assert size(64, 64, 64, 1 << 24) >= size(64, 64, 64, 100) + 4 * (1 << 24) // 16384 - 256
    assert size(0, 0, 64, 8) == 0
    assert size(-1, 1, 64, 8) == size(1, -1, 64, 8) == size(1, 1, 64, -1) == size(1, 1, 64, 1 << 31) == SHAPE
    assert size((1 << 31) - 1, 1 << 30, 16, 8) == SHAPE
    assert size(1, 1, 63, 8) == UNSUP
    assert lib.nvfp4_kv_compact_workspace_size(1000) >= 4016
    assert lib.nvfp4_kv_compact_workspace_size(-1) == SHAPE
    assert lib.nvfp4_kv_compact_workspace_size(1 << 31) == SHAPE


def test_python_refusals():
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    for call in (lambda: nv.kv_free(i32(2, 3), i32(2), i32(8), 64), lambda: nv.kv_fork(i32(2, 3), i32(2), i32(8), i32(2))):
        with pytest.raises(ValueError, match="on the GPU"):
            call()


def test_current_device_is_switched(monkeypatch):
    """A stream's handle of 0 is the current device's: a call for another device makes that one current."""
    seen = []

    class Guard:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            seen.append(("in", self.index))

        def __exit__(self, *_):
            seen.append(("out", self.index))

    monkeypatch.setattr(nv, "_CURRENT_DEVICE", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    assert nv._on_device(0, lambda x: x, 5) == 5 and seen == []
    assert nv._on_device(3, lambda x: seen.append(x) or 7, "call") == 7
    assert seen == [("in", 3), "call", ("out", 3)]

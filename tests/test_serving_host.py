"""Host-side checks of the serving operators (cache append, paged attention,
sampling) that need no GPU: every call here is refused, or is a no-op, before
anything is launched."""

import ctypes

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from nvfp4_quantized_matmul_amd.serving import _CacheStruct

OK, NULLPTR, SHAPE, DTYPE, GRID, UNSUP, ALIGN = 0, -1, -2, -3, -4, -6, -8
F32, BF16 = 0, 1
FAKE, ODD = 0x10000000, 0x10000001     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return nv.load_library()


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, pages=8, heads=2, page=64, dim=128):
    return _CacheStruct(k, v, ks, vs, pages, heads, page, dim)


def append(lib, c=None, k=FAKE, kt=256, kh=128, v=FAKE, vt=256, vh=128, q=FAKE + (1 << 20), qt=512, qh=128, hq=4,
           out=FAKE + (1 << 24), dt=BF16, tokens=3, cu=FAKE, batch=2, max_q=2, table=FAKE, width=4, lens=FAKE,
           freq=FAKE, rot=128, inter=0):
    c = c or cache(k=FAKE + (1 << 28), v=FAKE + (1 << 29))
    return lib.nvfp4_kv_append(ctypes.addressof(c), k, kt, kh, v, vt, vh, q, qt, qh, hq, out, dt, tokens, cu, batch,
                               max_q, table, width, lens, freq, rot, inter, None)


def attention(lib, c=None, q=FAKE, qt=512, qh=128, hq=4, dt=BF16, tokens=3, cu=FAKE, batch=2, max_q=2, table=FAKE,
              width=4, lens=FAKE, window=0, ws=None, ws_bytes=0, out=FAKE + (1 << 24)):
    c = c or cache(k=FAKE + (1 << 28), v=FAKE + (1 << 29))
    return lib.nvfp4_paged_attention(ctypes.addressof(c), q, qt, qh, hq, dt, tokens, cu, batch, max_q, table, width,
                                     lens, window, 1.0, ws, ws_bytes, out, None)


def sample(lib, x=FAKE, dt=BF16, batch=2, vocab=100, stride=100, u=FAKE, t=None, k=None, p=None, m=None, ws=None,
           ws_bytes=0, token=FAKE, prob=None):
    return lib.nvfp4_sample(x, dt, batch, vocab, stride, u, t, k, p, m, ws, ws_bytes, token, prob, None)


@pytest.mark.parametrize("call", [append, attention])
@pytest.mark.parametrize("bad,status", [
    (dict(pages=-1), SHAPE), (dict(heads=0), SHAPE), (dict(page=48), UNSUP), (dict(page=8), UNSUP),
    (dict(page=512), UNSUP), (dict(dim=80), UNSUP), (dict(dim=512), UNSUP), (dict(k=None), NULLPTR),
    (dict(vs=None), NULLPTR), (dict(k=FAKE + 8), ALIGN), (dict(v=ODD), ALIGN), (dict(pages=2 ** 31), SHAPE),
    (dict(pages=2 ** 31 - 1, heads=2 ** 31 - 1), SHAPE),
])
def test_cache_refusals(lib, call, bad, status):
    assert call(lib, c=cache(**bad)) == status


@pytest.mark.parametrize("call", [append, attention])
@pytest.mark.parametrize("bad,status", [
    (dict(dt=7), DTYPE), (dict(tokens=-1), SHAPE), (dict(batch=-1), SHAPE), (dict(max_q=-1), SHAPE),
    (dict(max_q=0), SHAPE), (dict(width=-1), SHAPE), (dict(width=1 << 26), SHAPE), (dict(qt=-1), SHAPE),
    (dict(qh=-128), SHAPE), (dict(cu=None), SHAPE), (dict(lens=None), NULLPTR), (dict(table=None), NULLPTR),
    (dict(table=ODD), ALIGN), (dict(lens=ODD), ALIGN), (dict(cu=ODD), ALIGN), (dict(q=ODD), ALIGN),
    (dict(out=FAKE + (1 << 24) + 8), ALIGN), (dict(tokens=2 ** 31), SHAPE), (dict(qt=2 ** 62), SHAPE),
    (dict(out=FAKE + (1 << 28)), SHAPE), (dict(max_q=1 << 28, hq=64, tokens=1 << 20, cu=FAKE), SHAPE),
])
def test_sequence_refusals(lib, call, bad, status):
    assert call(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(rot=127), SHAPE), (dict(rot=130), SHAPE), (dict(rot=-2), SHAPE), (dict(rot=0), SHAPE),
    (dict(freq=None), SHAPE), (dict(q=None), SHAPE), (dict(out=None), SHAPE), (dict(k=None), NULLPTR),
    (dict(v=None), NULLPTR), (dict(k=ODD), ALIGN), (dict(v=ODD), ALIGN), (dict(freq=ODD), ALIGN),
    (dict(kt=-1), SHAPE), (dict(vh=-1), SHAPE), (dict(out=FAKE), SHAPE), (dict(out=FAKE + (1 << 20)), SHAPE),
])
def test_append_refusals(lib, bad, status):
    assert append(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(hq=5), SHAPE), (dict(q=None), NULLPTR), (dict(out=None), NULLPTR), (dict(out=FAKE), SHAPE),
    (dict(ws=None, ws_bytes=64), SHAPE), (dict(ws=ODD, ws_bytes=64), ALIGN), (dict(ws=FAKE, ws_bytes=-1), SHAPE),
    (dict(ws=FAKE + (1 << 24), ws_bytes=64), SHAPE),
])
def test_attention_refusals(lib, bad, status):
    assert attention(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dt=9), DTYPE), (dict(batch=-1), SHAPE), (dict(vocab=-1), SHAPE), (dict(vocab=0, stride=0), SHAPE),
    (dict(stride=99), SHAPE), (dict(x=None), NULLPTR), (dict(u=None), NULLPTR), (dict(token=None), NULLPTR),
    (dict(x=ODD), ALIGN), (dict(u=ODD), ALIGN), (dict(t=ODD), ALIGN), (dict(k=ODD), ALIGN), (dict(p=ODD), ALIGN),
    (dict(m=ODD), ALIGN), (dict(token=ODD), ALIGN), (dict(prob=ODD), ALIGN), (dict(ws_bytes=16), SHAPE),
    (dict(vocab=2 ** 31, stride=2 ** 31), SHAPE), (dict(batch=70000), GRID),
])
def test_sample_refusals(lib, bad, status):
    assert sample(lib, **bad) == status


def test_empty_calls_launch_nothing(lib):
    assert append(lib, tokens=0) == OK
    assert append(lib, tokens=0, batch=0, cu=None) == OK
    assert attention(lib, tokens=0) == OK
    assert attention(lib, tokens=0, batch=0, cu=None, q=None, out=None) == OK
    assert attention(lib, hq=0) == OK
    assert sample(lib, batch=0, x=None, u=None, token=None) == OK


def test_workspace_sizes(lib):
    size = lib.nvfp4_paged_attention_workspace_size
    assert size(1, 32, 8, 128, 48, 1, 1, 16, 0, BF16) == UNSUP
    assert size(1, 32, 8, 100, 64, 1, 1, 16, 0, BF16) == UNSUP
    assert size(1, 33, 8, 128, 64, 1, 1, 16, 0, BF16) == SHAPE
    assert size(1, 32, 0, 128, 64, 1, 1, 16, 0, BF16) == SHAPE
    assert size(1, 32, 8, 128, 64, 1, 1, 16, 0, 5) == DTYPE
    assert size(0, 32, 8, 128, 64, 1, 1, 16, 0, BF16) == 0
    assert size(1, 32, 8, 128, 64, 1, 1, 2048, 0, BF16) > 0          # one sequence over a long cache is split
    assert lib.nvfp4_sample_workspace_size(1, -1, BF16) == SHAPE
    assert lib.nvfp4_sample_workspace_size(1, 100, 9) == DTYPE
    assert lib.nvfp4_sample_workspace_size(0, 100, BF16) == 0


def test_binding_refuses_on_the_cpu():
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        nv.KVCache(z(2, 1, 64, 64), z(2, 1, 64, 64), z(2, 1), z(2, 1))
    with pytest.raises(ValueError, match="pages, heads, page, dim"):
        nv.KVCache(z(2, 64, 64), z(2, 1, 64, 64), z(2, 1), z(2, 1))
    with pytest.raises(ValueError, match="does not match"):
        nv.KVCache(z(2, 1, 64, 128), z(2, 1, 64, 128), z(2, 1), z(2, 1))
    with pytest.raises(ValueError, match="k_scales"):
        nv.KVCache(z(2, 1, 64, 128), z(2, 1, 128, 64), z(2, 2), z(2, 1))
    with pytest.raises(ValueError, match="page must be"):
        nv.KVCache(z(2, 1, 48, 128), z(2, 1, 128, 48), z(2, 1), z(2, 1))
    with pytest.raises(TypeError, match="uint8"):
        nv.KVCache(z(2, 1, 64, 64, dt=torch.int8), z(2, 1, 64, 64), z(2, 1), z(2, 1))
    with pytest.raises(ValueError, match="GPU"):
        nv.sample(z(2, 8, dt=torch.float32), z(2, dt=torch.float32))
    with pytest.raises(TypeError):
        nv.sample(z(2, 8, dt=torch.float64), z(2, dt=torch.float32))
    with pytest.raises(ValueError, match="batch, vocab"):
        nv.sample(z(8, dt=torch.float32), z(1, dt=torch.float32))

"""Every entry point launches with its tensors' device as the current one, also
where that is another; without a GPU, with a library that only looks."""

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from nvfp4_quantized_matmul_amd import pages, serving

HERE, OTHER = 0, 3      # the tensors' device, and the current one


class On(torch.Tensor):
    """A CPU tensor that says it is on device HERE."""

    def get_device(self):
        return HERE


class Library:
    """Every function notes its name and the device that is current; sizes are 0 and calls succeed."""

    def __init__(self):
        self.current, self.calls, self.sizes = OTHER, [], []

    def __getattr__(self, name):
        def fn(*args):
            (self.sizes if name.endswith("_workspace_size") else self.calls).append((name, self.current))
            return 0
        return fn


@pytest.fixture
def lib(monkeypatch):
    lib = Library()

    class Switch:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            lib.current, self.before = self.index, lib.current

        def __exit__(self, *_):
            lib.current = self.before

    monkeypatch.setattr(torch.cuda, "device", Switch)
    for module in (nv, serving, pages):
        monkeypatch.setattr(module, "load_library", lambda: lib)
        monkeypatch.setattr(module, "_stream", lambda device: 0)
        if hasattr(module, "_CURRENT_DEVICE"):
            monkeypatch.setattr(module, "_CURRENT_DEVICE", lambda: lib.current)
    monkeypatch.setattr(nv, "_require_gpu", lambda *_: torch.device("cpu", HERE))
    monkeypatch.setattr(nv, "_QMM_WS_CACHE", {})
    for module, name in ((serving, "_ATTENTION_WS_CACHE"), (serving, "_SAMPLE_WS_CACHE"), (pages, "_WS_CACHE")):
        monkeypatch.setattr(module, name, {})
    return lib


def on(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(On)


def u8(*shape):
    return on(*shape, dtype=torch.uint8)


def f32(*shape):
    return on(*shape, dtype=torch.float32)


def cache():
    return nv.KVCache(u8(4, 1, 16, 64), u8(4, 1, 64, 16), u8(4, 1), u8(4, 1))


PLANE = lambda *lead: (on(*lead, 32, 8), u8(*lead, 32, 4))      # noqa: E731  (32 rows of 64)

CALLS = {
    "transcode": lambda: nv.transcode(u8(32, 32), u8(32, 4)),
    "dequantize": lambda: nv.dequantize(*PLANE()),
    "quantize": lambda: nv.quantize(f32(32, 64)),
    "qmm": lambda: nv.qmm(f32(2, 64), *PLANE()),
    "qmm_glu": lambda: nv.qmm_glu(f32(2, 64), *PLANE(), None, *PLANE(), None),
    "qmm_batched": lambda: nv.qmm_batched(f32(1, 2, 64), *PLANE(3)),
    "gather_qmm": lambda: nv.gather_qmm(f32(3, 1, 64), *PLANE(3), on(5)),
    "sample": lambda: nv.sample(f32(2, 100), f32(2)),
    "kv_append": lambda: nv.kv_append(f32(2, 1, 64), f32(2, 1, 64), cache(), on(2, 2), on(2)),
    "kv_append with norms": lambda: nv.kv_append(f32(2, 1, 64), f32(2, 1, 64), cache(), on(2, 2), on(2), k_norm=f32(64)),
    "paged_attention": lambda: nv.paged_attention(f32(2, 1, 64), cache(), on(2, 2), on(2)),
    "paged_attention with sinks": lambda: nv.paged_attention(f32(2, 1, 64), cache(), on(2, 2), on(2), window=5, sinks=1),
    "kv_free": lambda: nv.kv_free(on(2, 2), on(2), on(4), 16),
    "kv_reserve": lambda: nv.kv_reserve(cache(), on(2, 2), on(2), on(4)),
    "kv_fork": lambda: nv.kv_fork(on(2, 2), on(2), on(4), on(3)),
    "kv_compact": lambda: nv.kv_compact(cache(), on(2, 2), on(4)),
}


@pytest.mark.parametrize("name", CALLS)
def test_launches_on_the_tensors_device(lib, name):
    CALLS[name]()
    assert len(lib.calls) == 1 and lib.calls[0][0].startswith("nvfp4_" + name.split()[0])
    assert lib.calls[0][1] == HERE and lib.current == OTHER


@pytest.mark.parametrize("name", ["qmm", "qmm_glu", "qmm_batched"])
def test_workspaces_are_sized_for_the_tensors_device(lib, name):
    """The products' splits go by its compute units."""
    CALLS[name]()
    assert len(lib.sizes) == 1 and lib.sizes[0][1] == HERE


@pytest.mark.parametrize("name", ["qmm", "qmm_batched"])
def test_launches_with_a_workspace(lib, name, monkeypatch):
    monkeypatch.setattr(nv, "_qmm_workspace_bytes", lambda *_: 256)
    CALLS[name]()
    assert lib.calls == [(f"nvfp4_{name}_ws", HERE)] and lib.current == OTHER


def test_every_entry_point_is_here():
    """All that the package offers and that launches something."""
    other = {"KVCache", "select_route", "qmv_max_rows", "status_string", "load_library", "library_path", "check_planes"}
    calls = {n for n in nv.__all__ if callable(getattr(nv, n)) and not isinstance(getattr(nv, n), type)} - other
    assert calls == {n.split()[0] for n in CALLS}

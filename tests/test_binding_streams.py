"""A call's `stream` argument: what the call allocates and clears, and the library call itself, belong
to that stream.  Host logic alone: the streams and the library are stand-ins."""
import contextlib
import ctypes

import pytest
import torch

import spmm_tiled_column_b200 as spw

N = K = 64


class Library:
    """Records the stream handle of each call (the last pointer argument); sizes are 64."""

    def __init__(self, world):
        self.world = world

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 64
            self.world.launches.append([a.value for a in args if isinstance(a, ctypes.c_void_p)][-1])
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    class World:
        stream = 0
    w = World()
    w.launches, w.made = [], []

    @contextlib.contextmanager
    def on(stream):
        w.stream, before = stream, w.stream
        yield
        w.stream = before

    def watched(make):
        def call(*a, **kw):
            w.made.append(w.stream)
            return make(*a, **kw)
        return call

    library = Library(w)
    for name in ("zeros", "empty", "empty_strided"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(spw, "_stream", lambda s=None: ctypes.c_void_p(1000 + (w.stream if s is None else s)))
    monkeypatch.setattr(spw, "lib", lambda: library)
    monkeypatch.setattr(spw, "_half", lambda t, name: t)
    monkeypatch.setattr(spw, "_mask_like", lambda m, n, k: (m, K))
    monkeypatch.setattr(spw, "_nbytes", lambda t, name="ws": 1 << 20)
    monkeypatch.setattr(spw, "_need_buf", lambda *a: None)
    monkeypatch.setattr(spw, "_same_device", lambda *a: None)
    monkeypatch.setattr(spw, "spw_format_query", lambda mask, stream=None: (1024, 0))
    return w


def calls():
    h = spw.spw_format()
    h.N, h.K = N, K
    b, x, m = torch.zeros(1024, dtype=torch.uint8), torch.zeros(2, K, dtype=torch.float16), torch.zeros(N, K, dtype=torch.uint8)
    W = torch.zeros(N, K, dtype=torch.float16)
    return {
        "spw_compress": (W, m), "spw_decompress": (h, b), "spw_select_threshold": (x, 0.1), "spw_select_topk": (x, 3),
        "spw_spmv": (h, b, x), "spw_spmv_group": ([h], [b], [x]), "spw_spmv_noalloc": (h, b, x), "spw_spmm": (h, b, x),
        "spw_group_tokens": (x, 0.1, 16), "spw_spmm_tokens": (h, b, x, 0.1), "spw_spmv_tc": (h, b, x),
        "spw_spmv_auto": (h, b, x), "spw_spmv_ffn": (h, b, h, b, x), "spw_split24": (W, m), "spw_spmm24": (h, b, b, x),
        "spw_spmv_ep": (h, b, x), "spw_spmm_ep": (h, b, x), "spw_spmm_ffn": (h, b, h, b, x),
        "spw_spmm_backward": (h, b, x, x), "spw_spmm_ffn_backward": (h, b, h, b, x, x, x, x),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_everything_on_the_named_stream(world, name):
    args = calls()[name]
    world.made.clear()
    getattr(spw, name)(*args, stream=7)
    assert world.made and set(world.made) == {7}
    assert world.launches and set(world.launches) == {1007}
    world.made.clear(), world.launches.clear()
    getattr(spw, name)(*args)
    assert set(world.made) == {0} and set(world.launches) == {1000}


def test_stream_as_the_last_positional_argument(world):
    a = calls()
    spw.spw_spmv(*a["spw_spmv"], 0.0, None, None, None, 5)
    spw.spw_spmm(*a["spw_spmm"], None, None, 5)
    spw.spw_split24(*a["spw_split24"], 5)
    spw.spw_spmm24(*a["spw_spmm24"], None, None, 5)
    spw.spw_decompress(*a["spw_decompress"], None, 5)
    assert set(world.launches) == {1005} and len(world.launches) == 5
    with pytest.raises(TypeError):
        spw.spw_split24(*a["spw_split24"], 5, 6)

"""Which workspace a holder's decode calls use: calls that may run at the same time never share one.
Host logic alone: the streams, the capture and the library calls below are stand-ins."""
import contextlib
import ctypes

import pytest
import torch

import spmm_tiled_column_b200 as spw

K = N = 64


class Lin(spw.SparseLinear):
    def __init__(self):
        self.N, self.K = N, K
        self.buf, self.hdr = torch.zeros(16, dtype=torch.uint8), None
        self._ws = {}
        self._workspaces = spw._Workspaces(self.buf.device)


@pytest.fixture
def world(monkeypatch):
    """The current stream, whether it captures, and (workspace, stream at the call, stream where it
    was cleared) of every call."""
    class World:
        stream, capturing, calls, cleared = 0, False, [], {}
    w = World()
    w.calls, w.cleared = [], {}
    zeros = torch.zeros

    def clear(*a, **kw):
        t = zeros(*a, **kw)
        w.cleared[id(t)] = w.stream
        return t

    @contextlib.contextmanager
    def on(stream):
        w.stream, before = stream, w.stream
        yield
        w.stream = before

    def record(place):
        def call(*args, **kw):
            w.calls.append((args[place], w.stream, w.cleared[id(args[place])]))
        return call

    monkeypatch.setattr(torch, "zeros", clear)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.capturing)
    monkeypatch.setattr(spw, "_stream", lambda s=None: ctypes.c_void_p(1000 + (w.stream if s is None else s)))
    for name, place in (("spw_spmv_ffn", 8), ("spw_spmv_ep", 9), ("spw_spmv", 6), ("spw_spmv_auto", 6)):
        monkeypatch.setattr(spw, name, record(place))
        monkeypatch.setattr(spw, name + "_workspace_bytes", lambda *a: 4096)
    return w


def call_of(kind):
    if kind == "ffn":
        return spw.SparseFFN(Lin(), Lin()).spmv
    return {"ep": Lin().spmv_ep, "spmv": Lin().spmv, "auto": Lin().spmv_auto}[kind]


KINDS = ["ffn", "ep", "spmv", "auto"]


@pytest.mark.parametrize("kind", KINDS)
def test_one_for_each_batch_and_stream(world, kind):
    call = call_of(kind)
    xs = {B: torch.empty(B, K) for B in (1, 2)}
    for stream in (1, 2, None, 1, 2, None):
        for B in (1, 2):
            call(xs[B], stream=stream)
    ws = [id(t) for t, _, _ in world.calls]
    assert ws[:6] == ws[6:] and len(set(ws)) == 6
    # the call runs on the stream that it names, and that stream cleared its workspace
    assert [(at, cleared) for _, at, cleared in world.calls] == [(s, s) for s in (1, 1, 2, 2, 0, 0)] * 2


@pytest.mark.parametrize("kind", KINDS)
def test_a_captured_call_has_its_own(world, kind):
    call = call_of(kind)
    x = torch.empty(1, K)
    for world.capturing in (True, False, True, False, True):
        call(x)
    a, b, c, d, e = [t for t, _, _ in world.calls]
    assert b is d and len({id(t) for t in (a, b, c, e)}) == 4


@pytest.mark.parametrize("kind", KINDS)
def test_stream_as_the_last_positional_argument(world, kind):
    call = call_of(kind)
    args = (0.0, None, None, 0, None, None) if kind == "ep" else (0.0, None, None)
    call(torch.empty(1, K), *args, 7)
    assert world.calls[0][1:] == (7, 7)


@pytest.mark.parametrize("kind", KINDS)
def test_made_anew_after_a_reported_timeout(world, kind, monkeypatch):
    class Library:
        code = spw.SPW_OK

        def spw_last_device_status(self, stream, at):
            at._obj.value = self.code
            return spw.SPW_OK
    library = Library()
    monkeypatch.setattr(spw, "lib", lambda: library)
    call = call_of(kind)
    x = torch.empty(1, K)
    for library.code in (spw.SPW_OK, spw.SPW_ERR_FORMAT, spw.SPW_ERR_TIMEOUT, spw.SPW_OK):
        call(x, stream=1), call(x, stream=2)
        assert spw.spw_last_device_status() == library.code
    call(x, stream=1), call(x, stream=2)
    ws = [id(t) for t, _, _ in world.calls]
    assert ws[0:2] == ws[2:4] == ws[4:6] and ws[6:8] == ws[8:10] and len(set(ws)) == 4

"""Decode calls of one holder that run at the same time: on two streams, in two graphs, captured before
any eager call.  Long sums of few rows: the strips are split, so the workspace's counters and partial
sums are in use.  Results are compared bit by bit with calls made one after the other, and those with
the 64-bit form."""
import pytest
import torch

import ref64
from gpu_util import needs_gpu
from test_gpu_epilogue import half, layer, ok
from test_gpu_ffn_prefill import block
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]

N, K, T = 100, 8200, 0.3


class Gated:
    """SparseFFN.spmv: (h, its column set)."""

    def __init__(self, B):
        self.ffn, self.Wg, self.Wu = block(N, K, 0.5, 0.5, "silu", "holder")
        self.B = B

    def out(self):
        # (rows of 16-byte strides; column sets of a 16-byte size)
        return (torch.zeros(self.B, 104, dtype=torch.float16, device="cuda")[:, :N],
                torch.zeros(4, dtype=torch.int32, device="cuda"))

    def __call__(self, x, out, stream=None):
        return self.ffn.spmv(x, T, out[0], out[1], stream=stream)

    def check(self, x, out):
        h, words = out
        # the decode rounds g and u to fp16 before it multiplies, and adds one product at a time
        (ref, bound), (g, _), (u, _) = ref64.gated(x, self.Wg, self.Wu, "silu")
        a, _ = ref64.act(g, "silu")
        S = x.double().abs() @ self.Wg.double().abs().T * u.abs() + a.abs() * (x.double().abs() @ self.Wu.double().abs().T)
        bound = bound + ref64.HALF * (1.13 * g.abs() * u.abs() + a.abs() * u.abs()) + 1.13 * K * 2.0 ** -24 * S
        ref64.assert_within(h, ref, bound)
        on = ((h != 0) & ~(h.float().abs() < T)).any(0)
        got = (words[:, None].bitwise_right_shift(torch.arange(32, device="cuda", dtype=torch.int32)) & 1).flatten()[:N]
        assert torch.equal(got.bool(), on)


class Plain:
    """SparseLinear.spmv or spmv_auto."""

    def __init__(self, method, B):
        self.lin, self.W = layer(N, K, 0.5, "holder")
        self.method, self.B = getattr(self.lin, method), B

    def out(self):
        return (torch.zeros(self.B, 104, dtype=torch.float16, device="cuda")[:, :N],)

    def __call__(self, x, out, stream=None):
        return self.method(x, 0.0, None, out[0], stream=stream)

    def check(self, x, out):
        z, dz = ref64.product(x, self.W)
        dz = dz + K * 2.0 ** -24 * (x.double().abs() @ self.W.double().abs().T)
        ref64.assert_within(out[0], *ref64.epilogue(z, dz, "none"))


def make(kind, B):
    return Gated(B) if kind == "ffn" else Plain(kind, B)


def inputs(B, n):
    return [half(B, K, "hold", B, i) for i in range(n)]


KINDS = ["ffn", "spmv", "spmv_auto"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [1, 9, 16])
def test_captured_before_any_call(kind, B):
    call = make(kind, B)
    (x,) = inputs(B, 1)
    captured = call.out()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, captured)
    for _ in range(2):
        eager = call.out()
        call(x, eager)
        call.check(x, eager)
        for t in captured:
            t.zero_()
        graph.replay()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)
    ok()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [1, 9, 16])
def test_two_streams_two_graphs_and_a_graph_beside_eager_calls(kind, B):
    call = make(kind, B)
    xs = inputs(B, 2)
    want = [call.out() for _ in xs]
    for x, w in zip(xs, want):
        call(x, w)
        ok()
        call.check(x, w)
    n = 20
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[call.out() for _ in range(n)] for _ in xs]
    torch.cuda.synchronize()

    def compare():
        torch.cuda.synchronize()
        for w, mine in zip(want, outs):
            for o in mine:
                for a, b in zip(o, w):
                    assert torch.equal(a, b)
                    a.zero_()
        torch.cuda.synchronize()

    for r in range(n):
        for x, s, mine in zip(xs, streams, outs):
            call(x, mine[r], stream=s)
    compare()
    graphs = [torch.cuda.CUDAGraph() for _ in xs]
    for g, x, mine in zip(graphs, xs, outs):
        with torch.cuda.graph(g):
            for o in mine:
                call(x, o)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    compare()
    with torch.cuda.stream(streams[0]):
        graphs[0].replay()
    for r in range(n):
        call(xs[1], outs[1][r], stream=streams[1])
    compare()
    ok()


def test_strips_are_split_at_these_sizes():
    c = Gated(1)
    assert spw.spw_spmv_ffn_workspace_bytes(c.ffn.gate.hdr, c.ffn.up.hdr, 1) > 4 * N * 2
    assert c.ffn.gate.hdr.n_ktiles == 129 and c.ffn.gate.hdr.n_strips == 2

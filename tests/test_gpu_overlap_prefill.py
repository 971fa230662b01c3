"""Launch overlap between consecutive calls (spw_set_launch_overlap) with the products with epilogues,
the gated block and the gradients around the decode: every result is bit for bit what it is without."""
import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_epilogue import half, layer, ok
from test_gpu_ffn_prefill import block
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture
def overlap():
    prev = spw.spw_set_launch_overlap(True)
    yield
    spw.spw_set_launch_overlap(prev)


def chain(D, F, M):
    ffn, _, _ = block(F, D, 0.5, 0.5, "silu", "chain")
    down, _ = layer(D, F, 0.5, "chain-down")
    X, dY = half(M, D, "cx", M), half(M, D, "cy", M)

    def run():
        """Each call reads what the one before it wrote; decodes follow each kind of kernel."""
        H, G, U = ffn.spmm(X, save=True)
        d1 = down.spmv(H[:2])
        Y = down.spmm_ep(H, residual=X)
        d2 = ffn.gate.spmv_ep(Y[:1], act="gelu")
        h, bits = ffn.spmv(Y[:2], 0.1)
        d3 = down.spmv_ep(h, 0.1, bits, residual=Y[:2])
        dH, _ = down.spmm_backward(None, dY, need_dv=False)
        d4 = down.spmv(dH[:1])
        dH, dVd = down.spmm_backward(H, dY)
        d5 = down.spmv_ep(dH[:1])
        dX, dVg, dVu = ffn.backward(X, G, U, dH)
        d6 = ffn.gate.spmv(dX[:1])
        only = ffn.backward(None, G, U, dH, need_dv=False)[0]
        d7 = ffn.up.spmv_ep(only[:4], 0.2, bias=None, act="relu")
        return H, G, U, d1, Y, d2, h, bits, d3, dH, d4, dVd, d5, dX, dVg, dVu, d6, only, d7
    return run


# the direct form of every product, and the expanded one
@pytest.mark.parametrize("D,F,M", [(256, 688, 40), (512, 1376, 4096)])
def test_a_chain_of_calls(overlap, D, F, M):
    run = chain(D, F, M)
    got = [run() for _ in range(3)]
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(2):
        graph.replay()
    ok()
    spw.spw_set_launch_overlap(False)
    want = run()
    ok()
    for one in got + [captured]:
        for i, (a, b) in enumerate(zip(one, want)):
            assert torch.equal(a, b), i

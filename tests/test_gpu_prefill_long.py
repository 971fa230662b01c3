"""The prefill products over operands of more than 2^32 elements: offsets in 64 bits throughout.

Rows at both ends and around the 2^31st and 2^32nd element are compared with the 64-bit forms."""
import pytest
import torch

import ref64
import workloads
from gpu_util import dev, needs_gpu
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def layer(N, K, *seed):
    W = dev(workloads.weight(N, K, "long", *seed, std=0.05))
    m = dev(workloads.random_mask(N, K, 0.5, "long", *seed))
    return spw.SparseLinear(W, m), W * m.to(torch.float16)


def some_rows(M, cols):
    """Row numbers at the ends and where offsets of 2^31 and 2^32 elements fall."""
    at = {0, 1, M - 130, M - 1}
    for e in (31, 32):
        r = 2 ** e // cols
        at |= {i for i in (r - 1, r, r + 1, r + 200) if 0 <= i < M}
    return torch.tensor(sorted(at), device="cuda")


def rows(M, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(M, cols, dtype=torch.float16, device="cuda").normal_(generator=g)


def ok():
    torch.cuda.synchronize()
    assert spw.spw_last_device_status() == spw.SPW_OK


def test_long_input_and_its_gradient():
    M, N, K = 300_001, 72, 16384  # X and dX: 4.9e9 elements
    lin, W = layer(N, K, "in")
    X = rows(M, K, 1)
    at = some_rows(M, K)
    Y = lin.spmm_ep(X, act="relu")
    ok()
    ref64.assert_within(Y[at], *ref64.epilogue(*ref64.product(X[at], W), "relu"))
    del X
    dY = rows(M, N, 2)
    dX, _ = lin.spmm_backward(None, dY, need_dv=False)
    ok()
    ref64.assert_within(dX[at], *ref64.dx([(dY[at], None, W)]))


def test_long_output():
    M, N, K = 300_001, 16384, 72  # Y, H, G and U: 4.9e9 elements each
    lin, W = layer(N, K, "out")
    X = rows(M, K, 3)
    at = some_rows(M, N)
    res = rows(M, N, 4)
    keep = res[at].clone()
    Y = lin.spmm_ep(X, act="silu", residual=res, Y=res)
    ok()
    ref64.assert_within(Y[at], *ref64.epilogue(*ref64.product(X[at], W), "silu", None, keep))
    del Y, res
    H, G, U = spw.SparseFFN(lin, lin).spmm(X, save=True)
    ok()
    for got, want in zip((H, G, U), ref64.gated(X[at], W, W, "silu")):
        ref64.assert_within(got[at], *want)

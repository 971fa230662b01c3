"""A gradient beyond fp16 in the gated block's backward: it shows in its token's row of dX and its weight
row's entries of dV, and nowhere else."""
import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_epilogue import half, ok
from test_gpu_ffn_prefill import block
from test_gpu_workspaces import order_of

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("N,K,M", [(200, 128, 30), (512, 512, 1500)])  # direct form of dX, expanded
def test_stays_in_its_row(N, K, M):
    ffn, Wg, Wu = block(N, K, 0.5, 0.5, "silu", "overflow")
    X, dH = half(M, K, "ox", M), half(M, N, "oh", M)
    _, G, U = ffn.spmm(X, save=True)
    G[7, 3], U[7, 3] = 1.0, 100.0
    clean = ffn.backward(X, G, U, dH)
    dH[7, 3] = 60000.0  # dG = 60000 * 100 * SiLU'(1); dU = 60000 * SiLU(1) = 43864, in range
    dX, dVg, dVu = ffn.backward(X, G, U, dH)
    ok()
    rows = torch.arange(M, device="cuda") != 7
    assert torch.equal(dX[rows], clean[0][rows]) and not torch.isfinite(dX[7]).any()
    for got, was, lin, W, spread in ((dVg, clean[1], ffn.gate, Wg, True), (dVu, clean[2], ffn.up, Wu, False)):
        at = order_of(lin, W)
        mine = (at >= 0) & (at // K == 3)
        assert mine.any() and torch.equal(got[~mine], was[~mine])
        if spread:
            assert not torch.isfinite(got[mine]).any()
    # (dU's entries of row 3: finite or beyond fp16 by their own size, never NaN)
    assert not torch.isnan(dVu).any()

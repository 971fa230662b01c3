"""Every operand of the calls that take rows: a view whose rows overlap is refused before a launch."""
import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_epilogue import half, layer, ok
from test_gpu_ffn_prefill import block
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def wide(cols, rows=10):
    """rows x cols that repeat one row."""
    return half(1, cols, "wide").expand(rows, cols)


def test_overlapping_rows():
    N, K, M = 64, 128, 10
    ffn, _, _ = block(N, K, 0.5, 0.5, "silu", "views")
    lin = ffn.gate
    h = (lin.hdr, lin.buf)
    X, R = half(M, K, "vx"), half(M, N, "vr")
    _, G, U = ffn.spmm(X, save=True)
    bad = [
        lambda: lin.spmv_ep(wide(K)), lambda: lin.spmv_ep(X, residual=wide(N)), lambda: lin.spmv_ep(X, y=wide(N)),
        lambda: lin.spmm_ep(wide(K)), lambda: lin.spmm_ep(X, residual=wide(N)), lambda: lin.spmm_ep(X, Y=wide(N)),
        lambda: ffn.spmm(wide(K)), lambda: ffn.spmm(X, H=wide(N)), lambda: ffn.spmm(X, G=wide(N), U=R.clone()),
        lambda: ffn.spmm(X, G=R.clone(), U=wide(N)),
        lambda: lin.spmm_backward(X, torch.ones(N, dtype=torch.float16, device="cuda").expand(M, N)),
        lambda: lin.spmm_backward(wide(K), R), lambda: spw.spw_spmm_backward(*h, X, R, dX=wide(K)),
        lambda: ffn.backward(wide(K), G, U, R), lambda: ffn.backward(X, wide(N), U, R),
        lambda: ffn.backward(X, G, wide(N), R), lambda: ffn.backward(X, G, U, wide(N)),
        lambda: spw.spw_spmm_ffn_backward(*h, ffn.up.hdr, ffn.up.buf, X, G, U, R, dX=wide(K)),
        lambda: lin.spmv(wide(K)), lambda: lin.spmv(X, y=wide(N)), lambda: lin.spmv_auto(wide(K)),
        lambda: lin.spmm(wide(K)), lambda: lin.spmm(X, Y=wide(N)), lambda: lin.spmm_tokens(wide(K)),
        lambda: ffn.spmv(wide(K)), lambda: spw.spw_select_threshold(wide(K), 0.1),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlap"):
            call()
    ok()


def test_a_broadcast_made_contiguous():
    lin, _ = layer(64, 128, 0.5, "views")
    X, r = half(10, 128, "vx"), half(1, 64, "vb")
    a = lin.spmm_ep(X, residual=r.expand(10, 64).contiguous())
    b = lin.spmm_ep(X, residual=r.repeat(10, 1))
    ok()
    assert torch.equal(a, b)

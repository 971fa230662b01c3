"""The caller's workspace of the products with epilogues, the gated block and the gradients: at any
16-byte boundary, of exactly the queried size."""
import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_epilogue import half, ok
from test_gpu_ffn_prefill import block
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def calls(N, K, M):
    """name -> (workspace bytes, call on a given workspace returning its results)."""
    ffn, _, _ = block(N, K, 0.5, 0.5, "silu", "ws")
    lin, h, u = ffn.gate, ffn.gate.hdr, ffn.up.hdr
    X, dY = half(M, K, "wx", M), half(M, N, "wy", M)
    _, G, U = ffn.spmm(X, save=True)
    return {
        "ep": (spw.spw_spmm_ep_workspace_bytes(h, M), lambda ws: (lin.spmm_ep(X, act="gelu", residual=dY, ws=ws),)),
        "ffn": (spw.spw_spmm_ffn_workspace_bytes(h, u, M), lambda ws: ffn.spmm(X, save=True, ws=ws)),
        "backward": (spw.spw_spmm_backward_workspace_bytes(h, M), lambda ws: lin.spmm_backward(X, dY, ws=ws)),
        "ffn_backward": (spw.spw_spmm_ffn_backward_workspace_bytes(h, u, M), lambda ws: ffn.backward(X, G, U, dY, ws=ws)),
    }


def dense_bytes(N, K):
    """The expanded weight: strips and k-tiles of 64, each rounded up to a multiple of four."""
    return -(-N // 256) * 4 * (-(-K // 256) * 4) * 8192


@pytest.mark.parametrize("which", ["ep", "ffn", "backward", "ffn_backward"])
def test_any_16_byte_boundary(which):
    N, K, M = 512, 512, 1500
    need, call = calls(N, K, M)[which]
    assert need >= dense_bytes(N, K)  # the expanded form: 32-byte stores into the workspace
    want = call(None)
    ok()
    for skip in (0, 16, 32, 48, 240, 256):
        room = torch.full((need + skip + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        assert room.data_ptr() % 256 == 0
        got = call(room[skip:skip + need])
        ok()
        for a, b in zip(got, want):
            assert torch.equal(a, b), skip
        assert (room[:skip] == 0x5A).all() and (room[skip + need:] == 0x5A).all(), skip
    with pytest.raises(spw.SpwError) as e:
        call(torch.zeros(need + 16, dtype=torch.uint8, device="cuda")[8:8 + need])
    assert e.value.status == spw.SPW_ERR_ALIGNMENT
    with pytest.raises(spw.SpwError) as e:
        call(torch.zeros(need, dtype=torch.uint8, device="cuda")[:need - 16])
    assert e.value.status == spw.SPW_ERR_BUFFER_TOO_SMALL

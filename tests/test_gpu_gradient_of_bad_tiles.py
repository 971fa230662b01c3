"""The packed gradients of a buffer whose sections disagree: the bad tile's entries are zeros, not what the
memory held before, and every other tile's are what they were."""
import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_corrupt import corrupted
from test_gpu_epilogue import half
from test_gpu_ffn_prefill import block
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def pointers(lin, buf):
    h = lin.hdr
    return buf[h.off_tileptr:h.off_tileptr + 4 * (h.n_strips * h.n_ktiles + 1)].view(torch.int32)


def bad_buffer(lin, what):
    """(buffer, number of tiles from the first on that it spoils)."""
    if what in ("bitmaps", "overclaim", "tileptr"):
        return corrupted(lin, what), 2 if what == "tileptr" else 1
    buf = lin.buf.clone()
    tp = pointers(lin, buf)
    if what == "one unit":    # tile 0's end a unit late
        tp[1] += 1
        return buf, 2
    if what == "negative":    # beyond 2^31, where adding a count passes 2^32
        tp[1] = -1
        return buf, 2
    words = buf[lin.hdr.off_bitmaps:lin.hdr.off_bitmaps + 512]  # "cleared": tile 0 without bits
    words.zero_()
    return buf, 1


@pytest.mark.parametrize("what", ["bitmaps", "overclaim", "tileptr", "one unit", "negative", "cleared"])
@pytest.mark.parametrize("N,K,M", [(256, 512, 40), (300, 450, 5000)])
def test_zeros_for_the_bad_tile_alone(what, N, K, M):
    ffn, _, _ = block(N, K, 0.5, 0.5, "silu", "badgrad")
    lin = ffn.gate
    X, dY = half(M, K, "bx", M), half(M, N, "by", M)
    _, G, U = ffn.spmm(X, save=True)
    n = spw._values_len(lin.hdr)
    good_v = lin.spmm_backward(X, dY, need_dx=False)[1]
    good_g, good_u = ffn.backward(X, G, U, dY, need_dx=False)[1:]
    torch.cuda.synchronize()
    assert spw.spw_last_device_status() == spw.SPW_OK
    buf, tiles = bad_buffer(lin, what)
    end = 8 * int(pointers(lin, lin.buf)[tiles])
    assert 0 < end < n
    dV, dVg = [torch.full((n,), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]
    guard = torch.full((n + 4096,), 7.0, dtype=torch.float16, device="cuda")
    spw.spw_spmm_backward(lin.hdr, buf, X, dY, need_dx=False, dV=dV)
    spw.spw_spmm_backward(lin.hdr, buf, X, dY, need_dx=False, dV=guard)
    _, _, dVu = spw.spw_spmm_ffn_backward(lin.hdr, buf, ffn.up.hdr, ffn.up.buf, X, G, U, dY, need_dx=False, dV_gate=dVg)
    torch.cuda.synchronize()
    assert spw.spw_last_device_status() == spw.SPW_ERR_FORMAT
    for got, good in ((dV, good_v), (dVg, good_g), (guard[:n], good_v)):
        assert not got[:end].any() and torch.equal(got[end:], good[end:])
    assert torch.equal(dVu, good_u) and (guard[n:] == 7).all()

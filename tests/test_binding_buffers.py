"""Raw buffers (workspaces, compressed weights, column sets) of the products with epilogues, the
gated block and the gradients: a tensor with gaps or repeats is refused before the library is
called.  The device check before it is replaced, so that host tensors reach it."""
import pytest
import torch

import spmm_tiled_column_b200 as spw

N, K, M = 64, 64, 4


def half(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


@pytest.fixture
def call(monkeypatch):
    monkeypatch.setattr(spw, "_same_device", lambda *tensors: None)
    h = spw.spw_format()
    h.N, h.K, h.bytes_total = N, K, 4096
    raw = torch.zeros(4096, dtype=torch.uint8)
    x, y = half(M, K), half(M, N)

    def run(which, buf=raw, ws=raw, bits=None):
        if which == "spmv_ep":
            return spw.spw_spmv_ep(h, buf, x, act_bits=bits, ws=ws)
        if which == "spmm_ep":
            return spw.spw_spmm_ep(h, buf, x, ws=ws)
        if which == "ffn":
            return spw.spw_spmm_ffn(h, raw, h, buf, x, ws=ws)
        if which == "ffn_backward":
            return spw.spw_spmm_ffn_backward(h, buf, h, raw, x, y, y, y, ws=ws)
        return spw.spw_spmm_backward(h, buf, x, y, ws=ws)
    return run


@pytest.mark.parametrize("which", ["spmv_ep", "spmm_ep", "ffn", "ffn_backward", "backward"])
@pytest.mark.parametrize("view", ["broadcast", "every other", "window"])
def test_gaps_and_repeats_are_refused(call, which, view):
    t = {"broadcast": torch.zeros(1, dtype=torch.uint8).expand(1 << 20),  # one byte
         "every other": torch.zeros(1 << 13, dtype=torch.uint8)[::2],
         "window": torch.zeros(5000, dtype=torch.uint8).unfold(0, 4096, 1)}[view]
    with pytest.raises(ValueError, match="buf.* must be contiguous"):
        call(which, buf=t)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        call(which, ws=t)


def test_column_set_with_gaps_is_refused(call):
    with pytest.raises(ValueError, match="act_bits must be contiguous"):
        call("spmv_ep", bits=torch.zeros(8, dtype=torch.int32)[::2])


def test_contiguous_buffers_pass_the_check():
    spw._whole("ws buf", None, torch.zeros(64, dtype=torch.uint8)[16:48])

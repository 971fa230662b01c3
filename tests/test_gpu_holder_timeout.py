"""After a reported timeout the holders' decode calls are right again, without the caller touching
their workspaces (as tests/test_gpu_timeout.py for calls with a workspace of the caller's)."""
import pytest
import torch

from gpu_util import needs_gpu
from test_gpu_epilogue import half, layer
from test_gpu_timeout import run_with_tiny_limit
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def status():
    torch.cuda.synchronize()
    return spw.spw_last_device_status()


@pytest.mark.parametrize("kind", ["ep", "spmv", "auto", "ffn"])
def test_right_after_a_timeout(kind):
    # several tiles a warp and split strips: a wait of the pipeline runs out, and the counters of
    # strips whose pieces were cut off may stay behind
    lin, _ = layer(4096, 11008, 0.5, "holder-timeout")
    x = half(1, 11008, "ht")
    assert spw.spw_spmv_ep_path(lin.hdr, 1) == 0
    call = {"ep": lambda: lin.spmv_ep(x, act="silu"), "spmv": lambda: lin.spmv(x), "auto": lambda: lin.spmv_auto(x),
            "ffn": lambda: ffn.spmv(x)[0]}[kind]
    ffn = spw.SparseFFN(lin, lin)
    want = call()
    assert status() == spw.SPW_OK
    held = (ffn if kind == "ffn" else lin)._workspaces._held
    (ws,) = held.values()
    assert run_with_tiny_limit(call) == spw.SPW_ERR_TIMEOUT
    ws.fill_(1)  # what a timeout may leave at worst
    for _ in range(2):
        assert torch.equal(call(), want)
    assert status() == spw.SPW_OK

"""Failure paths of the products with epilogues, the gated block and the gradients: bounded
waits that run out (as tests/test_gpu_timeout.py) and buffers whose sections disagree (as
tests/test_gpu_corrupt.py), for the form that decodes into shared memory and the one that
expands the weight first."""
import pytest
import torch

import ref64
from gpu_util import needs_gpu
from test_gpu_corrupt import corrupted
from test_gpu_epilogue import half, layer
from test_gpu_ffn_prefill import block
from test_gpu_timeout import run_with_tiny_limit
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]

# (N, K, M): the direct form, and the expanded one (its workspace holds the dense weight)
SIZES = [(1024, 2048, 64), (512, 512, 6000)]


def status():
    torch.cuda.synchronize()
    return spw.spw_last_device_status()


def calls(N, K, M):
    ffn, Wg, Wu = block(N, K, 0.5, 0.5, "silu", "faults")
    X, dY = half(M, K, "fx", M), half(M, N, "fy", M)
    _, G, U = ffn.spmm(X, save=True)
    return ffn, X, dY, {
        "ep": lambda: (ffn.gate.spmm_ep(X, act="gelu", residual=dY),),
        "ffn": lambda: (ffn.spmm(X),),
        "dx": lambda: ffn.gate.spmm_backward(None, dY, need_dv=False)[:1],
        "dv": lambda: ffn.gate.spmm_backward(X, dY, need_dx=False)[1:],
        "backward": lambda: ffn.backward(X, G, U, dY),
    }


def test_both_forms_are_taken():
    for (N, K, M), dense in zip(SIZES, (False, True)):
        ffn, _, _, _ = calls(N, K, M)
        h = ffn.gate.hdr
        assert (spw.spw_spmm_ep_workspace_bytes(h, M) >= 2 * N * K) == dense
        assert (spw.spw_spmm_ffn_workspace_bytes(h, ffn.up.hdr, M) >= 4 * N * K) == dense


@pytest.mark.parametrize("N,K,M", SIZES)
@pytest.mark.parametrize("which", ["ep", "ffn", "dx", "dv", "backward"])
def test_timeout_then_recovers(N, K, M, which):
    _, _, _, c = calls(N, K, M)
    want = [t.clone() for t in c[which]()]
    assert status() == spw.SPW_OK
    assert run_with_tiny_limit(lambda: c[which]()) == spw.SPW_ERR_TIMEOUT
    got = c[which]()
    assert status() == spw.SPW_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_decode_timeout_then_recovers():
    lin, _ = layer(1024, 2048, 0.5, "faults")
    x = half(16, 2048, "fd")
    assert spw.spw_spmv_ep_path(lin.hdr, 16) == 1
    want = lin.spmv_ep(x, 0.3, act="silu")
    assert run_with_tiny_limit(lambda: lin.spmv_ep(x, 0.3, act="silu")) == spw.SPW_ERR_TIMEOUT
    assert torch.equal(lin.spmv_ep(x, 0.3, act="silu"), want)
    assert status() == spw.SPW_OK


@pytest.mark.parametrize("what", ["bitmaps", "overclaim", "tileptr"])
@pytest.mark.parametrize("N,K,M", [(256, 512, 40), (512, 512, 6000)])
def test_format_reported_then_recovers(what, N, K, M):
    ffn, X, dY, c = calls(N, K, M)
    want = {k: [t.clone() for t in f()] for k, f in c.items()}
    x = half(16, K, "fd")
    dec = ffn.gate.spmv_ep(x)
    assert status() == spw.SPW_OK
    good, ffn.gate.buf = ffn.gate.buf, corrupted(ffn.gate, what)
    for k, f in c.items():
        f()
        assert status() == spw.SPW_ERR_FORMAT, k
    ffn.gate.spmv_ep(x)
    assert status() == spw.SPW_ERR_FORMAT
    # the strips that the fault does not touch are what they were
    Y = ffn.gate.spmm_ep(X, act="gelu", residual=dY)
    assert torch.equal(Y[:, 64:], want["ep"][0][:, 64:])
    status()
    ffn.gate.buf = good
    for k, f in c.items():
        for a, b in zip(f(), want[k]):
            assert torch.equal(a, b)
    assert torch.equal(ffn.gate.spmv_ep(x), dec)
    assert status() == spw.SPW_OK


def test_large_forms_against_64_bits():
    # the expanded form at ragged sizes, aligned and odd leading dimensions
    for N, K, M, ld in ((1030, 515, 5000, 0), (520, 1000, 4099, 3)):
        ffn, Wg, Wu = block(N, K, 0.4, 0.5, "gelu_tanh", "large", N)
        X, dH = half(M, K, "lx"), half(M, N, "lh")
        assert spw.spw_spmm_ep_workspace_bytes(ffn.gate.hdr, M) >= 2 * N * K
        res = half(M, N, "lr", ld=N + ld)
        Y = torch.full((M + 1, N + ld), 7.0, dtype=torch.float16, device="cuda")
        ffn.gate.spmm_ep(X, act="silu", residual=res, Y=Y[:M, :N])
        ref64.assert_within(Y[:M, :N], *ref64.epilogue(*ref64.product(X, Wg), "silu", None, res))
        assert (Y[M:] == 7).all() and (Y[:, N:] == 7).all()
        H, G, U = ffn.spmm(X, save=True)
        for got, (ref, bound) in zip((H, G, U), ref64.gated(X, Wg, Wu, "gelu_tanh")):
            ref64.assert_within(got, ref, bound)
        dX, _, _ = ffn.backward(X, G, U, dH)
        (dG, eg), (dU, eu) = ref64.gate_grads(G, U, dH, "gelu_tanh")
        ref64.assert_within(dX, *ref64.dx([(dG, eg, Wg), (dU, eu, Wu)]))
    assert status() == spw.SPW_OK

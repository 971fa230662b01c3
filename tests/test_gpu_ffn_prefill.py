"""The gated block for M rows (spw_spmm_ffn) against plain 64-bit forms."""
import pytest
import torch

import ref64
from gpu_util import needs_gpu
from test_gpu_epilogue import half, layer, ok
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def block(N, K, dg, du, act, *seed):
    g, Wg = layer(N, K, dg, "gate", *seed)
    u, Wu = layer(N, K, du, "up", *seed)
    return spw.SparseFFN(g, u, act), Wg, Wu


def check(ffn, Wg, Wu, X, name):
    H, G, U = ffn.spmm(X, save=True)
    ok()
    refs = ref64.gated(X, Wg, Wu, name)
    for got, (ref, bound), what in zip((H, G, U), refs, "HGU"):
        ref64.assert_within(got, ref, bound, f"{what} {name}")
    alone = ffn.spmm(X)
    ok()
    assert torch.equal(alone, H)


@pytest.mark.parametrize("N,K", [(1, 1), (64, 64), (256, 512), (130, 70), (300, 1), (1, 300), (200, 1000)])
@pytest.mark.parametrize("M", [1, 17, 256, 300])
def test_small(N, K, M):
    for name in ref64.ACTS:
        ffn, Wg, Wu = block(N, K, 0.5, 0.4, name)
        check(ffn, Wg, Wu, half(M, K, "f", M), name)


@pytest.mark.parametrize("N,K,M,dg,du", [
    (1030, 1024, 600, 0.5, 0.6),
    (96, 8192, 40, 0.5, 0.5),    # split reduction
    (2730, 1021, 333, 0.3, 0.3),
    (500, 300, 1000, 1.0, 0.0),  # nothing dropped against everything dropped
])
def test_larger(N, K, M, dg, du):
    ffn, Wg, Wu = block(N, K, dg, du, "silu", "larger")
    check(ffn, Wg, Wu, half(M, K, "fl"), "silu")


def test_agrees_with_the_decode_form():
    # the decode rounds g and u to fp16 before it multiplies: each is off by half a step more
    ffn, Wg, Wu = block(512, 1024, 0.5, 0.5, "silu", "decode")
    x = half(8, 1024, "fd")
    h, _ = ffn.spmv(x)
    H = ffn.spmm(x)
    ok()
    (ref, bound), (g, _), (u, _) = ref64.gated(x, Wg, Wu, "silu")
    a, _ = ref64.act(g, "silu")
    bound = bound + ref64.HALF * (1.13 * g.abs() * u.abs() + a.abs() * u.abs())
    # the CUDA-core decode adds one product at a time
    S = x.double().abs() @ Wg.double().abs().T * u.abs() + a.abs() * (x.double().abs() @ Wu.double().abs().T)
    ref64.assert_within(h, ref, bound + 1.13 * 1024 * 2.0 ** -24 * S)
    ref64.assert_within(H, ref, bound)


def test_strides_and_untouched_neighbours():
    N, K, M = 136, 200, 70
    ffn, Wg, Wu = block(N, K, 0.5, 0.5, "silu", "strides")
    X = half(M, K, "xs", ld=K + 24)
    refs = ref64.gated(X, Wg, Wu, "silu")
    for lds in ((N, N + 8, N + 16), (N + 1, N, N + 3)):
        bufs = [torch.full((M + 1, ld), 7.0, dtype=torch.float16, device="cuda") for ld in lds]
        H, G, U = [b[:M, :N] for b in bufs]
        ffn.spmm(X, H=H, G=G, U=U)
        ok()
        for got, (ref, bound), b in zip((H, G, U), refs, bufs):
            ref64.assert_within(got, ref, bound)
            assert (b[M:] == 7).all() and (b[:, N:] == 7).all()


def test_nonfinite_row_stays_in_its_row():
    ffn, _, _ = block(200, 128, 0.5, 0.5, "silu", "nan")
    X = half(30, 128, "xn")
    clean = ffn.spmm(X)
    X[7, 3] = float("nan")
    H = ffn.spmm(X)
    ok()
    assert torch.isnan(H[7]).all()
    keep = torch.arange(30, device="cuda") != 7
    assert torch.equal(H[keep], clean[keep])


def test_refusals():
    ffn, _, _ = block(64, 128, 0.5, 0.5, "silu", "bad")
    other, _ = layer(72, 128, 0.5, "bad")
    with pytest.raises(ValueError):
        spw.SparseFFN(ffn.gate, other)
    X = half(4, 128, "bad")
    with pytest.raises(spw.SpwError) as e:
        spw.spw_spmm_ffn(ffn.gate.hdr, ffn.gate.buf, other.hdr, other.buf, X)
    assert e.value.status == spw.SPW_ERR_INVALID_ARG
    assert spw.spw_spmm_ffn_workspace_bytes(ffn.gate.hdr, other.hdr, 4) == 0
    with pytest.raises(ValueError, match="together"):
        ffn.spmm(X, G=half(4, 64, "g"))
    with pytest.raises(spw.SpwError):
        spw.spw_spmm_ffn(ffn.gate.hdr, ffn.gate.buf, ffn.up.hdr, ffn.up.buf, X, act=9)
    with pytest.raises(ValueError):
        spw.SparseFFN(ffn.gate, ffn.up, "gelu").spmv(X)

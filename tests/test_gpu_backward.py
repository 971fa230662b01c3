"""The gradients of the sparse products (spw_spmm_backward, spw_spmm_ffn_backward): against the
formulas in 64 bits, and against differences of the forward products."""
import numpy as np
import pytest
import torch

import ref64
import workloads
from gpu_util import dev, needs_gpu
from test_gpu_epilogue import half, layer, ok
from test_gpu_ffn_prefill import block
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


def mask_of(W, lin):
    """The pattern, from the buffer's own decompression of all-ones values."""
    ones = lin.buf.clone()
    v = ones[lin.hdr.off_values:lin.hdr.bytes_total].view(torch.float16)
    v.fill_(1.0)
    return (spw.spw_decompress(lin.hdr, ones) != 0).to(torch.uint8)


SHAPES = [(1, 1, 1), (64, 64, 64), (130, 70, 33), (300, 1, 5), (1, 300, 20), (257, 515, 250), (100, 2000, 65),
          (1500, 130, 300), (64, 64, 3000)]


@pytest.mark.parametrize("N,K,M", SHAPES)
def test_linear(N, K, M):
    lin, W = layer(N, K, 0.5, "bwd")
    mask = mask_of(W, lin)
    X, dY = half(M, K, "bx", M), half(M, N, "by", M)
    dX, dV = lin.spmm_backward(X, dY)
    ok()
    ref64.assert_within(dX, *ref64.dx([(dY, None, W)]), "dX")
    order = ref64.packed_order(mask)
    ref, bound = ref64.dw(dY, None, X)
    ref64.assert_within(dV, ref64.pack(ref, order), ref64.pack(bound, order), "dV")
    only, none = lin.spmm_backward(X, dY, need_dv=False)
    assert none is None and torch.equal(only, dX)
    none, only = lin.spmm_backward(X, dY, need_dx=False)
    assert none is None and torch.equal(only, dV)


@pytest.mark.parametrize("N,K,M", SHAPES)
@pytest.mark.parametrize("name", ref64.ACTS)
def test_gated(N, K, M, name):
    ffn, Wg, Wu = block(N, K, 0.5, 0.3, name, "bwd")
    X, dH = half(M, K, "gx", M), half(M, N, "gh", M)
    H, G, U = ffn.spmm(X, save=True)
    dX, dVg, dVu = ffn.backward(X, G, U, dH)
    ok()
    (dG, eg), (dU, eu) = ref64.gate_grads(G, U, dH, name)
    ref64.assert_within(dX, *ref64.dx([(dG, eg, Wg), (dU, eu, Wu)]), "dX")
    for got, d, e, W, lin in ((dVg, dG, eg, Wg, ffn.gate), (dVu, dU, eu, Wu, ffn.up)):
        order = ref64.packed_order(mask_of(W, lin))
        ref, bound = ref64.dw(d, e, X)
        ref64.assert_within(got, ref64.pack(ref, order), ref64.pack(bound, order), "dV")


@pytest.mark.parametrize("density", [0.0, 1.0])
def test_empty_and_full_patterns(density):
    lin, W = layer(200, 300, density, "ends")
    X, dY = half(50, 300, "ex"), half(50, 200, "ey")
    dX, dV = lin.spmm_backward(X, dY)
    ok()
    ref64.assert_within(dX, *ref64.dx([(dY, None, W)]))
    order = ref64.packed_order(torch.full((200, 300), int(density), dtype=torch.uint8, device="cuda"))
    ref, bound = ref64.dw(dY, None, X)
    ref64.assert_within(dV, ref64.pack(ref, order), ref64.pack(bound, order))


def test_against_differences():
    # L = sum(C * H) for fixed C: its derivative along a direction, by central differences of
    # the 64-bit forward, against the gradients' inner product with the direction.  The
    # 64-bit forward's own difference error (h^2 of the third derivative, h = 1e-4) is far
    # below the gradients' rounding: |<g, d>| errors of at most 2^-9 of sum |g||d|.
    N, K, M = 96, 160, 40
    for name in ("silu", "gelu", "gelu_tanh", "none"):
        ffn, Wg, Wu = block(N, K, 0.5, 0.5, name, "diff")
        X, C = half(M, K, "dx"), half(M, N, "dc")
        _, G, U = ffn.spmm(X, save=True)
        dX, dVg, dVu = ffn.backward(X, G, U, C)
        ok()

        def loss(x, wg, wu):
            a, _ = ref64.act(x @ wg.T, name)
            return (C.double() * a * (x @ wu.T)).sum()

        x, wg, wu = X.double(), Wg.double(), Wu.double()
        e = 1e-4
        D = dev(workloads.rng("dir", 1).standard_normal((M, K)))
        num = (loss(x + e * D, wg, wu) - loss(x - e * D, wg, wu)) / (2 * e)
        # G and U enter the gradients as fp16: one more half step of each factor
        assert abs(num - (dX.double() * D).sum()) <= 2.0 ** -9 * (dX.double().abs() * D.abs()).sum()
        for dV, W, lin, which in ((dVg, wg, ffn.gate, 0), (dVu, wu, ffn.up, 1)):
            mask = mask_of(W, lin)
            D = dev(workloads.rng("dir", 2).standard_normal((N, K))) * mask
            p, q = (wg + e * D, wu) if which == 0 else (wg, wu + e * D)
            r, s = (wg - e * D, wu) if which == 0 else (wg, wu - e * D)
            num = (loss(x, p, q) - loss(x, r, s)) / (2 * e)
            d = ref64.pack(D, ref64.packed_order(mask))
            assert abs(num - (dV.double() * d).sum()) <= 2.0 ** -9 * (dV.double().abs() * d.abs()).sum()


def test_strides_and_untouched_neighbours():
    N, K, M = 136, 77, 70
    ffn, Wg, Wu = block(N, K, 0.5, 0.5, "silu", "strides")
    X = half(M, K, "sx", ld=88)
    G, U, dH = half(M, N, "sg", ld=N + 3), half(M, N, "su", ld=N + 8), half(M, N, "sh", ld=N + 1)
    buf = torch.full((M + 1, K + 5), 7.0, dtype=torch.float16, device="cuda")
    n = spw._values_len(ffn.gate.hdr), spw._values_len(ffn.up.hdr)
    vg, vu = [torch.full((k + 9,), 7.0, dtype=torch.float16, device="cuda") for k in n]
    h = ffn.gate.hdr, ffn.gate.buf, ffn.up.hdr, ffn.up.buf
    dX, a, b = spw.spw_spmm_ffn_backward(*h, X, G, U, dH, dX=buf[:M, :K], dV_gate=vg, dV_up=vu)
    ok()
    (dG, eg), (dU, eu) = ref64.gate_grads(G, U, dH, "silu")
    ref64.assert_within(dX, *ref64.dx([(dG, eg, Wg), (dU, eu, Wu)]))
    assert (buf[M:] == 7).all() and (buf[:, K:] == 7).all()
    for got, d, e, W, lin in ((a, dG, eg, Wg, ffn.gate), (b, dU, eu, Wu, ffn.up)):
        order = ref64.packed_order(mask_of(W, lin))
        ref, bound = ref64.dw(d, e, X)
        ref64.assert_within(got[:-9], ref64.pack(ref, order), ref64.pack(bound, order))
        assert (got[-9:] == 7).all()


def test_no_tokens():
    ffn, _, _ = block(64, 72, 0.5, 0.5, "silu", "zero")
    e = lambda n: torch.empty((0, n), dtype=torch.float16, device="cuda")  # noqa: E731
    dX, a, b = ffn.backward(e(72), e(64), e(64), e(64))
    ok()
    assert dX.shape == (0, 72) and not a.any() and not b.any() and a.numel() == spw._values_len(ffn.gate.hdr)
    dX, v = ffn.gate.spmm_backward(e(72), e(64))
    ok()
    assert dX.shape == (0, 72) and not v.any()


def test_training_step_through_a_block():
    # gate/up -> down onto the residual stream, the gradients of the whole, and one step of the
    # kept weights in place: the forward then runs on the new weights without recompressing
    D, F, M = 256, 688, 150
    ffn, Wg, Wu = block(F, D, 0.5, 0.5, "silu", "step")
    down, Wd = layer(D, F, 0.5, "step-down")
    X, dY = half(M, D, "tx"), half(M, D, "ty")
    H, G, U = ffn.spmm(X, save=True)
    Y = down.spmm_ep(H, residual=X)
    dH, dVd = down.spmm_backward(H, dY)
    dX, dVg, dVu = ffn.backward(X, G, U, dH)
    ok()
    ref64.assert_within(Y, *ref64.epilogue(*ref64.product(H, Wd), "none", None, X))
    ref64.assert_within(dH, *ref64.dx([(dY, None, Wd)]))
    (dG, eg), (dU, eu) = ref64.gate_grads(G, U, dH, "silu")
    ref64.assert_within(dX, *ref64.dx([(dG, eg, Wg), (dU, eu, Wu)]))
    for lin, W, dV in ((ffn.gate, Wg, dVg), (ffn.up, Wu, dVu), (down, Wd, dVd)):
        mask = mask_of(W, lin)
        order = ref64.packed_order(mask)
        assert torch.equal(lin.values(), ref64.pack(W, order))
        new = (lin.values().float() - 2.0 ** -12 * dV.float()).to(torch.float16)
        lin.values().copy_(new)
        dense = torch.zeros_like(W).flatten()
        dense[order[order >= 0]] = new[order >= 0]
        assert torch.equal(lin.decompress(), dense.view_as(W))


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_captured_and_replayed(which):
    ffn, Wg, Wu = block(300, 256, 0.5, 0.5, "silu", "graph")
    X = half(90, 256, "cx").contiguous()
    dH = half(90, 300, "ch").contiguous()
    _, G, U = ffn.spmm(X, save=True)
    call = (lambda: (ffn.spmm(X),)) if which == "forward" else (lambda: ffn.backward(X, G, U, dH))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (1, 2):
        X.copy_(half(90, 256, "cx", seed))
        dH.copy_(half(90, 300, "ch", seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, call()):
            assert torch.equal(a, b)
    ok()


def test_two_streams():
    ffn, Wg, Wu = block(512, 512, 0.5, 0.5, "silu", "streams")
    Xs = [half(200, 512, "st", i) for i in range(4)]
    want = [ffn.spmm(X) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = []
    for _ in range(5):
        for s, X in zip(streams, Xs):
            with torch.cuda.stream(s):
                got.append(ffn.spmm(X))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 4])
    ok()


def test_refusals():
    ffn, _, _ = block(64, 128, 0.5, 0.5, "silu", "bad")
    X, G, U, dH = half(4, 128, "x"), half(4, 64, "g"), half(4, 64, "u"), half(4, 64, "h")
    with pytest.raises(ValueError, match="need X"):
        ffn.backward(None, G, U, dH)
    assert ffn.backward(None, G, U, dH, need_dv=False)[1:] == (None, None)
    with pytest.raises(spw.SpwError) as e:
        ffn.backward(X, G, U, dH, need_dx=False, need_dv=False)
    assert e.value.status == spw.SPW_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ffn.backward(X, G, U[:3], dH)
    with pytest.raises(ValueError):
        ffn.backward(X[:, :120], G, U, dH)
    with pytest.raises(spw.SpwError) as e:
        ffn.backward(X, G, U, dH, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == spw.SPW_ERR_BUFFER_TOO_SMALL
    lin = ffn.gate
    with pytest.raises(ValueError, match="columns"):
        lin.spmm_backward(X, half(4, 56, "y"))
    with pytest.raises(spw.SpwError):  # dY rows at a stride that is no multiple of 8
        lin.spmm_backward(X, torch.zeros((4, 65), dtype=torch.float16, device="cuda")[:, :64])
    with pytest.raises(ValueError):
        spw.spw_spmm_backward(lin.hdr, lin.buf, X, dH, dV=torch.zeros(8, dtype=torch.float16, device="cuda"))

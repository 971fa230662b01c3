"""The products with an epilogue (spw_spmv_ep, spw_spmm_ep) against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import ref64
import workloads
from gpu_util import dev, needs_gpu
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]

SHAPES = [(1, 1), (64, 64), (256, 512), (130, 70), (300, 1), (1, 300), (200, 1000), (65, 4097)]


def layer(N, K, density, *seed):
    W = dev(workloads.weight(N, K, "ep", *seed, std=0.05))
    m = dev(workloads.random_mask(N, K, density, "ep", *seed))
    return spw.SparseLinear(W, m), W * m.to(torch.float16)


def half(rows, cols, *seed, ld=None, std=1.0):
    """fp16 rows at a leading dimension (a multiple of 8 unless given)."""
    ld = -(-cols // 8) * 8 if ld is None else ld
    a = workloads.rng("ep-act", rows, cols, *seed).standard_normal((rows, ld)) * std
    return dev(a.astype(np.float16))[:, :cols]


def ok():
    torch.cuda.synchronize()
    assert spw.spw_last_device_status() == spw.SPW_OK


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 33, 257])
def test_prefill_small(N, K, M):
    lin, W = layer(N, K, 0.5)
    X = half(M, K, "x", M)
    bias, res = half(1, N, "b")[0].contiguous(), half(M, N, "r", M, ld=N + 3)
    z, dz = ref64.product(X, W)
    for name in ref64.ACTS:
        for b, r in ((None, None), (bias, res)):
            Y = lin.spmm_ep(X, bias=b, act=name, residual=r)
            ok()
            ref64.assert_within(Y, *ref64.epilogue(z, dz, name, b, r), f"{name} {b is not None}")


@pytest.mark.parametrize("N,K,M,density", [
    (512, 1024, 600, 0.5),      # several row tiles
    (64, 8192, 20, 0.5),        # few tiles, a long sum: the reduction is split
    (1111, 2049, 300, 0.4),     # ragged everywhere
    (4096, 256, 2050, 0.3),     # many column tiles, a last row tile of two rows
    (200, 600, 129, 1.0),       # nothing dropped
    (200, 600, 129, 0.0),       # everything dropped
])
def test_prefill_larger(N, K, M, density):
    lin, W = layer(N, K, density, "larger")
    X, res = half(M, K, "xl"), half(M, N, "rl")
    bias = half(1, N, "bl")[0].contiguous()
    Y = lin.spmm_ep(X, bias=bias, act="silu", residual=res)
    ok()
    ref64.assert_within(Y, *ref64.epilogue(*ref64.product(X, W), "silu", bias, res))


def test_prefill_strides_and_untouched_neighbours():
    N, K, M = 136, 200, 70
    lin, W = layer(N, K, 0.5, "strides")
    X = half(M, K, "xs", ld=K + 56)
    z, dz = ref64.product(X, W)
    for ldy in (N, N + 8, N + 5):  # 16-byte stores and scalar ones
        buf = torch.full((M + 2, ldy), 7.0, dtype=torch.float16, device="cuda")
        Y = buf[:M, :N]
        assert lin.spmm_ep(X, Y=Y) is Y
        ok()
        ref64.assert_within(Y, *ref64.epilogue(z, dz, "none"))
        assert (buf[M:] == 7).all() and (buf[:, N:] == 7).all()


def test_prefill_residual_in_place():
    N, K, M = 256, 4096, 40  # split sum as well
    lin, W = layer(N, K, 0.5, "inplace")
    X, res = half(M, K, "xi"), half(M, N, "ri")
    ref = ref64.epilogue(*ref64.product(X, W), "gelu", None, res)
    Y = res.clone()
    lin.spmm_ep(X, act="gelu", residual=Y, Y=Y)
    ok()
    ref64.assert_within(Y, *ref)


def test_prefill_workspace_of_any_content_and_determinism():
    N, K, M = 128, 4096, 50
    lin, _ = layer(N, K, 0.5, "ws")
    X = half(M, K, "xw")
    need = spw.spw_spmm_ep_workspace_bytes(lin.hdr, M)
    first = None
    for fill in (0, 0xFF, 0x5A):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            Y = lin.spmm_ep(X, act="gelu_tanh", ws=ws)
            ok()
            first = Y if first is None else first
            assert torch.equal(Y, first)


def test_prefill_extreme_values():
    N, K, M = 70, 100, 20
    W = torch.zeros((N, K), dtype=torch.float16, device="cuda")
    W[:, 0] = 1.0
    lin = spw.SparseLinear(W, torch.ones((N, K), dtype=torch.uint8, device="cuda"))
    vals = torch.tensor([0.0, -0.0, 1e-7, -6e-8, 3.0, -3.0, -6.0, -9.0, -20.0, 65504.0, -65504.0, 11.0, -11.5,
                         0.5, -0.5, 88.0, -88.0, 100.0, -104.0, 2.0], dtype=torch.float16, device="cuda")
    X = torch.zeros((M, 104), dtype=torch.float16, device="cuda")[:, :K]
    X[:, 0] = vals
    z = vals.double()[:, None].expand(M, N)
    for name in ref64.ACTS:
        Y = lin.spmm_ep(X, act=name)
        ok()
        a, _ = ref64.act(z, name)
        # the sum is exact here: only the activation's own error and the rounding remain
        ref64.assert_within(Y, a, 2.0 ** -19 * a.abs() + 2.0 ** -23 + ref64.HALF * a.abs() + ref64.TINY, name)
    X[3, 1], X[4, 1] = float("inf"), float("nan")
    Y = lin.spmm_ep(X)
    ok()
    assert not torch.isfinite(Y[3]).any() and torch.isnan(Y[4]).all()
    assert torch.isfinite(Y[[0, 1, 2, 5]]).all()


def test_prefill_zero_rows():
    lin, _ = layer(64, 64, 0.5)
    assert lin.spmm_ep(torch.empty((0, 64), dtype=torch.float16, device="cuda")).shape == (0, 64)


@pytest.mark.parametrize("N,K", SHAPES + [(512, 2048)])
@pytest.mark.parametrize("B", [1, 3, 8, 16])
def test_decode(N, K, B):
    lin, W = layer(N, K, 0.5)
    x = half(B, K, "d", B)
    bias, res = half(1, N, "b")[0].contiguous(), half(B, N, "r", B, ld=N + 1)
    cols = dev((workloads.rng("cols", K).random(K) < 0.7).astype(np.uint8)).bool()
    w = torch.zeros((K + 31) // 32 * 32, dtype=torch.int64, device="cuda")
    w[:K] = cols.long()
    w = (w.view(-1, 32) << torch.arange(32, device="cuda")).sum(1).to(torch.int32)
    for t, on in ((0.0, None), (0.4, w)):
        xt = torch.where((x != 0) & ~(x.float().abs() < t), x, torch.zeros_like(x))
        if on is not None:
            xt = torch.where(cols, xt, torch.zeros_like(xt))
        z, dz = ref64.product(xt, W)
        # CUDA-core sums add one product at a time
        dz = K * 2.0 ** -24 * (xt.double().abs() @ W.double().abs().T) + dz
        for name, b, r in (("none", None, res), ("gelu", bias, None), ("silu", bias, res), ("relu", None, None),
                           ("none", None, None)):
            y = lin.spmv_ep(x, t, on, bias=b, act=name, residual=r)
            ok()
            ref64.assert_within(y, *ref64.epilogue(z, dz, name, b, r), f"{name} t={t}")
    if spw.spw_spmv_ep_path(lin.hdr, B) == 0:
        assert torch.equal(lin.spmv_ep(x), lin.spmv(x))  # no epilogue: the plain decode
    Y = res.clone()
    lin.spmv_ep(x, bias=bias, residual=Y, y=Y)  # in place
    ok()
    assert torch.equal(Y, lin.spmv_ep(x, bias=bias, residual=res))


def test_refusals():
    lin, _ = layer(64, 128, 0.5)
    X = half(4, 128, "bad")
    with pytest.raises(ValueError, match="unknown activation"):
        lin.spmm_ep(X, act="swish")
    for act in (-1, 5):
        with pytest.raises(spw.SpwError) as e:
            lin.spmm_ep(X, act=act)
        assert e.value.status == spw.SPW_ERR_INVALID_ARG
        with pytest.raises(spw.SpwError):
            lin.spmv_ep(X, act=act)
    with pytest.raises(ValueError, match="bias"):
        lin.spmm_ep(X, bias=half(1, 63, "b")[0])
    with pytest.raises(ValueError, match="residual"):
        lin.spmm_ep(X, residual=half(3, 64, "r"))
    with pytest.raises(ValueError, match="columns"):
        lin.spmm_ep(half(4, 120, "x"))
    with pytest.raises(ValueError, match="current CUDA device"):
        lin.spmm_ep(X, bias=torch.zeros(64, dtype=torch.float16))
    big, _ = layer(2048, 2048, 0.5)
    need = spw.spw_spmm_ep_workspace_bytes(big.hdr, 8192)
    assert need >= 2 * 2048 * 2048
    with pytest.raises(spw.SpwError) as e:  # workspace too small
        big.spmm_ep(half(8192, 2048, "bad"), ws=torch.zeros(need - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == spw.SPW_ERR_BUFFER_TOO_SMALL
    with pytest.raises(spw.SpwError) as e:  # bias not 16-byte aligned
        lin.spmm_ep(X, bias=half(1, 72, "b")[0][1:65])
    assert e.value.status == spw.SPW_ERR_ALIGNMENT
    with pytest.raises(spw.SpwError):  # X rows at a stride that is no multiple of 8
        lin.spmm_ep(torch.zeros((4, 129), dtype=torch.float16, device="cuda")[:, :128])
    with pytest.raises(spw.SpwError):
        lin.spmv_ep(half(17, 128, "x"))


@pytest.mark.parametrize("name", ref64.ACTS)
def test_activation_of_every_finite_value(name):
    """Weight = identity, so the product is the operand itself: every finite fp16 through the
    activation of both products.  Bound: half a step, and 2^-16 of the value.  (Wherever the
    result is not below 2^-25, the exponentials' arguments stay below 18; five fp32 roundings
    of one are 18 * 5 * 2^-24 < 5.4e-6 of its exponential, __expf's own error (2 + 18) 2^-23 <
    2.4e-6, the normal tail's fit 1.3e-6, divisions and products a few 2^-23: 1.1e-5 < 2^-16.)"""
    eye = torch.eye(64, device="cuda")
    lin = spw.SparseLinear(eye.to(torch.float16), eye.to(torch.uint8))
    bits = torch.arange(65536, dtype=torch.int32, device="cuda")
    x = bits[(bits & 0x7C00) != 0x7C00].to(torch.int16).view(torch.float16).view(-1, 64)
    a, _ = ref64.act(x.double(), name)
    bound = (ref64.HALF + 2.0 ** -16) * a.abs() + ref64.TINY
    ref64.assert_within(lin.spmm_ep(x, act=name), a, bound, "spmm_ep " + name)
    for i in range(0, x.shape[0], 16):
        ref64.assert_within(lin.spmv_ep(x[i:i + 16], act=name), a[i:i + 16], bound[i:i + 16], "spmv_ep " + name)
    ok()


# Long sums of few rows: the reduction is split, and the workspace's counters are in use (the
# CUDA-core decode at 1 row, the tensor cores at 9).
@pytest.mark.parametrize("B", [1, 9])
def test_decode_captured_before_any_call(B):
    """The first call of a weight is captured; an eager call then comes before the first replay."""
    lin, W = layer(100, 8200, 0.5, "capture")
    x, y0 = half(B, 8200, "cap", B), torch.empty(B, 100, dtype=torch.float16, device="cuda")
    want = ref64.epilogue(*ref64.product(x, W), "silu")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.spmv_ep(x, act="silu", y=y0)
    for _ in range(2):
        ref64.assert_within(lin.spmv_ep(x, act="silu"), *want)
        y0.zero_()
        graph.replay()
        ref64.assert_within(y0, *want)
    ok()


@pytest.mark.parametrize("B", [1, 9])
def test_decode_on_two_streams_and_in_two_graphs(B):
    """Calls of one weight that overlap: eager ones on two streams, then two graphs."""
    lin, W = layer(100, 8200, 0.5, "streams")
    xs = [half(B, 8200, "two", B, i) for i in range(2)]
    want = [ref64.epilogue(*ref64.product(x, W), "relu") for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ys = [torch.zeros(20, B, 104, dtype=torch.float16, device="cuda")[:, :, :100] for _ in xs]  # 16-byte rows
    torch.cuda.synchronize()
    for r in range(20):
        for x, y, s in zip(xs, ys, streams):
            lin.spmv_ep(x, act="relu", y=y[r], stream=s)
    torch.cuda.synchronize()
    for y, (a, bound) in zip(ys, want):
        ref64.assert_within(y, a.expand_as(y), bound.expand_as(y))
    graphs = [torch.cuda.CUDAGraph() for _ in xs]
    for g, x, y in zip(graphs, xs, ys):
        y.zero_()
        with torch.cuda.graph(g):
            for r in range(20):
                lin.spmv_ep(x, act="relu", y=y[r])
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for y, (a, bound) in zip(ys, want):
        ref64.assert_within(y, a.expand_as(y), bound.expand_as(y))
    ok()


def test_decode_splits_at_these_sizes():
    lin, _ = layer(100, 8200, 0.5, "streams")
    assert spw.spw_spmv_ep_workspace_bytes(lin.hdr, 1) > 0


@pytest.mark.parametrize("B", [2, 16])
def test_decode_threshold_boundaries(B):
    """Weight = identity: the result is x~ itself.  Thresholds at, just above and just below fp16
    values, below the smallest and above the largest one; non-finite entries only where the column
    set is off (there they must leave no trace, on the tensor cores either)."""
    eye = torch.eye(64, device="cuda")
    lin = spw.SparseLinear(eye.to(torch.float16), eye.to(torch.uint8))
    assert spw.spw_spmv_ep_path(lin.hdr, 16) == 1 and spw.spw_spmv_ep_path(lin.hdr, 2) == 0
    base = torch.tensor([0.5, 0.4998, 0.50049, 6e-8, 1.2e-7, 6.1e-5, 6.2e-5, 65504.0, 65472.0, 1.0, 0.0, -0.0, 2.0,
                         1e-4, 3.0, 0.25], dtype=torch.float16, device="cuda")
    x = torch.stack([base.repeat(4).roll(b) * (1 if b % 2 else -1) for b in range(B)])
    on = torch.ones(64, dtype=torch.bool, device="cuda")
    on[[3, 17, 40]] = False
    x[:, 3], x[:, 17], x[:, 40] = float("nan"), float("inf"), 1.0
    words = (on.view(2, 32).long() << torch.arange(32, device="cuda")).sum(1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    for t in (0.0, 1e-9, 6e-8, 5.96e-8, 6.1e-5, 0.5, 0.50001, 0.49999, 1.0, 65504.0, 65503.9, 1e6):
        keep = on & ~(x.double().abs() < float(np.float32(t)))
        want = torch.where(keep, x.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
        assert torch.equal(lin.spmv_ep(x, t, words).double(), want), t
    ok()

"""The workspace of the products with epilogues, the gated block and the gradients: at any
16-byte boundary, of exactly the queried size."""
import pytest
import torch

import ref64
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


def grads_bytes(N, M):
    """dG and dU of the gated block's gradients."""
    return 2 * (-(-2 * M * (-(-N // 8) * 8) // 256) * 256)


# Sizes at which the expanded form is taken and its sum is split: the workspace then holds fp32
# partial sums (256 KB and more) behind the dense weight, and counters of arrived pieces.
@pytest.mark.parametrize("which,N,K,M", [
    ("ep", 136, 5000, 3000), ("ffn", 136, 5000, 2500),
    ("backward", 8192, 256, 2000),       # dX: 128 steps for 8 tiles of 256 x 256
    ("backward", 512, 512, 5000),        # dV: 79 steps for 4 tiles
    ("ffn_backward", 8192, 256, 2000), ("ffn_backward", 512, 512, 5000),
])
def test_split_sums_with_any_content(which, N, K, M):
    need, call = calls(N, K, M)[which]
    gated = which.startswith("ffn")
    rest = need - dense_bytes(N, K) * (2 if gated else 1) - (grads_bytes(N, M) if which == "ffn_backward" else 0)
    assert rest >= 1 << 18  # expanded, and partial sums beside it
    first = None
    for fill in (0, 0xFF, 0x5A):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):  # (the second finds what the first left)
            got = [t.clone() for t in call(ws)]
            ok()
            first = first or got
            for a, b in zip(got, first):
                assert torch.equal(a, b), fill
    check(which, N, K, M, first)


def check(which, N, K, M, got):
    """Results of calls() against the 64-bit forms."""
    ffn, Wg, Wu = block(N, K, 0.5, 0.5, "silu", "ws")
    X, dY = half(M, K, "wx", M), half(M, N, "wy", M)

    def packed(v, lin, W, d, e):
        at = order_of(lin, W)
        ref, bound = ref64.dw(d, e, X)
        kept = at >= 0
        ref64.assert_within(v[kept], ref.flatten()[at[kept]], bound.flatten()[at[kept]], "dV")
        assert not v[~kept].any()

    if which == "ep":
        ref64.assert_within(got[0], *ref64.epilogue(*ref64.product(X, Wg), "gelu", None, dY))
    elif which == "ffn":
        for t, want in zip(got, ref64.gated(X, Wg, Wu, "silu")):
            ref64.assert_within(t, *want)
    elif which == "backward":
        ref64.assert_within(got[0], *ref64.dx([(dY, None, Wg)]))
        packed(got[1], ffn.gate, Wg, dY, None)
    else:
        _, G, U = ffn.spmm(X, save=True)
        (dG, eg), (dU, eu) = ref64.gate_grads(G, U, dY, "silu")
        ref64.assert_within(got[0], *ref64.dx([(dG, eg, Wg), (dU, eu, Wu)]))
        packed(got[1], ffn.gate, Wg, dG, eg)
        packed(got[2], ffn.up, Wu, dU, eu)


def order_of(lin, W):
    """For each entry of the values section its index in the flattened weight, -1 for filling: read
    from the layout by decompressing numbers of places instead of weights."""
    n = lin.values().numel()
    place = torch.arange(n, device="cuda")
    order = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    digits = []
    for d in range(3):  # three digits to the base 1024, plus one: exact in fp16, and never zero
        buf = lin.buf.clone()
        v = buf[lin.hdr.off_values:lin.hdr.bytes_total].view(torch.float16)
        v.copy_((place // 1024 ** d % 1024 + 1).to(torch.float16))
        digits.append(spw.spw_decompress(lin.hdr, buf).flatten().long())
    kept = digits[0] != 0
    index = sum((t - 1) * 1024 ** d for d, t in enumerate(digits))[kept]
    order[index] = kept.nonzero().squeeze(1)
    assert torch.equal(lin.values()[index], W.flatten()[kept])
    return order


@pytest.mark.parametrize("which", ["backward", "ffn_backward"])
@pytest.mark.parametrize("N,K,M", [(1030, 515, 5000), (520, 1000, 4099)])
def test_gradients_of_large_runs(which, N, K, M):
    need, call = calls(N, K, M)[which]
    assert need >= dense_bytes(N, K)  # (dX by the expanded form as well)
    got = call(None)
    ok()
    check(which, N, K, M, got)

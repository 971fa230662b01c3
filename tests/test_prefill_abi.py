"""Host-side argument checks of the products with epilogues, the gated block and the gradients:
every refusal comes before any device call, so they run without a GPU."""
import ctypes

import pytest

from spmm_tiled_column_b200 import build as spw_build
from test_abi import valid_header

P = ctypes.c_void_p
GOOD, ODD, S = P(0x10000), P(0x10008), P(0)
WS = ctypes.c_uint64(1 << 30)
INVALID, ALIGN, FORMAT = 1, 2, 4


@pytest.fixture(scope="module")
def spw():
    spw_build.build()
    import spmm_tiled_column_b200 as m
    return m


def by(h):
    return ctypes.byref(h)


def bad_header(spw):
    h = valid_header(spw)
    h.version = 7
    return h


def epilogue(spw, bias=None, residual=None, ldr=0, act=0):
    return spw.spw_epilogue(bias, residual, ldr, act)


def test_epilogue_arguments(spw):
    L, h = spw.lib(), valid_header(spw)  # 128 x 128

    def mm(hd=h, buf=GOOD, X=GOOD, M=4, ldx=128, ep=None, Y=GOOD, ldy=128):
        return L.spw_spmm_ep(by(hd), buf, X, M, ldx, None if ep is None else by(ep), Y, ldy, GOOD, WS, S)

    def mv(hd=h, buf=GOOD, x=GOOD, B=4, ldx=128, t=0.0, bits=None, ep=None, y=GOOD, ldy=128):
        return L.spw_spmv_ep(by(hd), buf, x, B, ldx, t, bits, None if ep is None else by(ep), y, ldy, GOOD, WS, S)

    for call in (mm, mv):
        assert call(hd=bad_header(spw)) == FORMAT
        assert call(buf=None) == INVALID
        assert call(ldx=100) == INVALID and call(ldx=132) == INVALID and call(ldy=127) == INVALID
        assert call(buf=ODD) == ALIGN
        for act in (-1, 5, 99):
            assert call(ep=epilogue(spw, act=act)) == INVALID
        assert call(ep=epilogue(spw, residual=0x20000, ldr=127)) == INVALID
        assert call(ep=epilogue(spw, bias=0x20008)) == ALIGN
        assert call(ep=epilogue(spw, residual=0x20002, ldr=128)) == ALIGN
    assert mm(X=None) == INVALID and mm(Y=None) == INVALID and mm(M=-1) == INVALID
    assert mm(X=ODD) == ALIGN and mm(Y=ODD) == ALIGN
    assert mm(M=0, X=None, Y=None) == 0  # nothing to do
    assert mm(M=0, ep=epilogue(spw, act=9)) == INVALID
    for B in (0, 17):
        assert mv(B=B) == INVALID
    for t in (-1.0, float("nan"), float("inf")):
        assert mv(t=t) == INVALID
    assert mv(bits=ODD) == ALIGN
    assert L.spw_spmv_ep_path(by(h), 0) == -1 and L.spw_spmv_ep_path(by(h), 17) == -1
    assert L.spw_spmv_ep_path(by(bad_header(spw)), 1) == -1
    assert L.spw_spmv_ep_workspace_bytes(by(h), 17) == 0
    assert L.spw_spmm_ep_workspace_bytes(by(h), 0) == 0
    assert L.spw_spmm_ep_workspace_bytes(by(bad_header(spw)), 5) == 0


def test_gated_block_arguments(spw):
    L, h, other = spw.lib(), valid_header(spw), valid_header(spw, N=192)

    def f(hg=h, hu=h, bg=GOOD, bu=GOOD, X=GOOD, M=4, ldx=128, act=2, H=GOOD, ldh=128, G=None, ldg=0, U=None, ldu=0):
        return L.spw_spmm_ffn(by(hg), bg, by(hu), bu, X, M, ldx, act, H, ldh, G, ldg, U, ldu, GOOD, WS, S)

    assert f(hu=other) == INVALID and f(hg=bad_header(spw)) == FORMAT and f(hu=bad_header(spw)) == FORMAT
    assert f(bg=None) == INVALID and f(bu=None) == INVALID and f(X=None) == INVALID and f(H=None) == INVALID
    assert f(M=-1) == INVALID and f(act=5) == INVALID and f(act=-1) == INVALID
    assert f(G=GOOD, ldg=128) == INVALID and f(U=GOOD, ldu=128) == INVALID  # both or neither
    assert f(G=GOOD, ldg=127, U=GOOD, ldu=128) == INVALID and f(G=GOOD, ldg=128, U=GOOD, ldu=100) == INVALID
    assert f(ldx=132) == INVALID and f(ldh=127) == INVALID
    for name in ("bg", "bu", "X", "H"):
        assert f(**{name: ODD}) == ALIGN
    assert f(G=ODD, ldg=128, U=GOOD, ldu=128) == ALIGN
    assert f(M=0, X=None, H=None) == 0
    assert L.spw_spmm_ffn_workspace_bytes(by(h), by(other), 4) == 0


def test_gradient_arguments(spw):
    L, h, other = spw.lib(), valid_header(spw), valid_header(spw, K=192)

    def f(hg=h, hu=h, bg=GOOD, bu=GOOD, X=GOOD, M=4, ldx=128, act=2, G=GOOD, ldg=128, U=GOOD, ldu=128, dH=GOOD,
          lddh=128, dX=GOOD, lddx=128, vg=GOOD, vu=GOOD):
        return L.spw_spmm_ffn_backward(by(hg), bg, by(hu), bu, X, M, ldx, act, G, ldg, U, ldu, dH, lddh, dX, lddx,
                                       vg, vu, GOOD, WS, S)

    assert f(hu=other) == INVALID and f(hg=bad_header(spw)) == FORMAT
    assert f(act=7) == INVALID and f(M=-3) == INVALID
    assert f(vg=None) == INVALID and f(vu=None) == INVALID  # both or neither
    assert f(dX=None, vg=None, vu=None) == INVALID          # nothing asked for
    for name in ("bg", "bu", "G", "U", "dH", "X"):
        assert f(**{name: None}) == INVALID, name
    for name in ("bg", "bu", "G", "U", "dH", "X", "dX", "vg", "vu"):
        assert f(**{name: ODD}) == ALIGN, name
    assert f(ldg=127) == INVALID and f(ldu=127) == INVALID and f(lddh=127) == INVALID and f(lddx=127) == INVALID
    assert f(ldx=132) == INVALID
    assert f(M=0, dX=None, vg=None, vu=None) == 0

    def b(hd=h, buf=GOOD, X=GOOD, M=4, ldx=128, dY=GOOD, lddy=128, dX=GOOD, lddx=128, v=GOOD):
        return L.spw_spmm_backward(by(hd), buf, X, M, ldx, dY, lddy, dX, lddx, v, GOOD, WS, S)

    assert b(hd=bad_header(spw)) == FORMAT and b(M=-1) == INVALID
    assert b(dX=None, v=None) == INVALID and b(X=None) == INVALID and b(dY=None) == INVALID and b(buf=None) == INVALID
    assert b(lddy=132) == INVALID and b(lddy=100) == INVALID and b(lddx=100) == INVALID and b(ldx=132) == INVALID
    for name in ("buf", "X", "dY", "dX", "v"):
        assert b(**{name: ODD}) == ALIGN, name
    assert b(M=0, v=None, dX=None) == 0
    assert L.spw_spmm_backward_workspace_bytes(by(h), 0) == 0


def test_activation_names(spw):
    assert [spw._act(n) for n in ("none", "relu", "silu", "gelu", "gelu_tanh")] == [0, 1, 2, 3, 4]
    assert ctypes.sizeof(spw.spw_epilogue) == 24
    with pytest.raises(ValueError):
        spw._act("swish")


def test_equal_outputs_and_largest_sizes(spw):
    L, h = spw.lib(), valid_header(spw)
    UNSUPPORTED = 5
    A, B, C = (P(0x10000 * i) for i in (2, 3, 4))

    def f(H, G, U):
        return L.spw_spmm_ffn(by(h), GOOD, by(h), GOOD, GOOD, 4, 128, 2, H, 128, G, 128, U, 128, GOOD, WS, S)

    assert f(A, B, B) == INVALID and f(A, A, B) == INVALID and f(A, B, A) == INVALID
    assert h.bytes_total > h.off_values
    assert L.spw_spmm_ffn_backward(by(h), GOOD, by(h), GOOD, GOOD, 4, 128, 2, GOOD, 128, GOOD, 128, GOOD, 128, A, 128,
                                   B, B, GOOD, WS, S) == INVALID
    M = 0x7ffff001  # the last tile's rows would pass 2^31
    assert L.spw_spmm_ep(by(h), GOOD, GOOD, M, 128, None, A, 128, GOOD, WS, S) == UNSUPPORTED
    assert L.spw_spmm_ffn(by(h), GOOD, by(h), GOOD, GOOD, M, 128, 2, A, 128, B, 128, C, 128, GOOD, WS, S) == UNSUPPORTED
    assert L.spw_spmm_backward(by(h), GOOD, GOOD, M, 128, GOOD, 128, A, 128, B, GOOD, WS, S) == UNSUPPORTED
    assert L.spw_spmm_ep_workspace_bytes(by(h), M) == 0

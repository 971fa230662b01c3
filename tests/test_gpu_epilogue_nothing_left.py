"""Decode with an epilogue where the rule, the column set or the mask leaves nothing: the result is
act(bias) + residual in every row, on both paths and in every column-fetch mode."""
import pytest
import torch

import ref64
from gpu_util import needs_gpu
from test_gpu_epilogue import half, layer, ok
import spmm_tiled_column_b200 as spw

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(params=[0, 1, 2], ids=["whole-tiles", "column-fetch", "always"])
def fetch(request):
    prev = spw.spw_set_column_fetch(request.param)
    yield request.param
    spw.spw_set_column_fetch(prev)


def words(on):
    w = torch.nn.functional.pad(on.long(), (0, -on.numel() % 32)).view(-1, 32) << torch.arange(32, device="cuda")
    w = w.sum(1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


SHAPES = [(1, 1), (130, 70), (100, 8200), (64, 4096), (2000, 300)]


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("B", [1, 2, 5, 16])
def test_nothing_takes_part(fetch, N, K, B):
    full, _ = layer(N, K, 0.5, "left")
    none, _ = layer(N, K, 0.0, "left")
    x, bias, res = half(B, K, "lx", B), half(1, N, "lb")[0].contiguous(), half(B, N, "lr", B)
    zeros = half(B, K, "lx", B).zero_()  # (zeros_like would lose the 16-byte row stride)
    empty = words(torch.zeros(K, dtype=torch.bool, device="cuda"))
    a, bound = ref64.epilogue(torch.zeros(B, N, dtype=torch.float64, device="cuda"),
                              torch.zeros(B, N, dtype=torch.float64, device="cuda"), "silu", bias, res)
    for lin, xs, t, bits in ((none, x, 0.0, None), (none, x, 0.5, empty), (full, x, 0.0, empty),
                             (full, zeros, 0.0, None), (full, x, 100.0, None)):
        y = lin.spmv_ep(xs, t, bits, bias=bias, act="silu", residual=res)
        ok()
        ref64.assert_within(y, a, bound)
        assert not lin.spmv_ep(xs, t, bits).any()
    ok()


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("B", [1, 2, 5, 16])
def test_few_columns_take_part(fetch, N, K, B):
    lin, W = layer(N, K, 0.5, "few")
    x, res = half(B, K, "fx", B), half(B, N, "fr", B)
    for on in (torch.arange(K, device="cuda") == K - 1, torch.arange(K, device="cuda") % 97 == 0):
        xt = torch.where(on & ~(x.float().abs() < 0.2), x, torch.zeros_like(x))
        z, dz = ref64.product(xt, W)
        dz = dz + K * 2.0 ** -24 * (xt.double().abs() @ W.double().abs().T)
        y = lin.spmv_ep(x, 0.2, words(on), act="gelu", residual=res)
        ok()
        ref64.assert_within(y, *ref64.epilogue(z, dz, "gelu", None, res))

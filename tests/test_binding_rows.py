"""Rows handed to the library as a pointer and a leading dimension: views whose rows overlap (a
broadcast, a sliding window) are refused, on the host."""
import pytest
import torch

import spmm_tiled_column_b200 as spw


def half(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


def overlapping():
    row = half(64)
    return {
        "broadcast": row.expand(10, 64),              # 128 bytes that would be read as 1280
        "gradient of a sum over rows": half(1, 64).expand(10, 64),
        "sliding window": half(100).unfold(0, 64, 4),  # 10 rows, 4 elements apart
        "one short": half(10 * 64).as_strided((10, 64), (63, 1)),
    }


@pytest.mark.parametrize("which", list(overlapping()))
def test_overlapping_rows_are_refused(which):
    t = overlapping()[which]
    assert t.shape == (10, 64) and t.stride(1) == 1
    with pytest.raises(ValueError, match="overlap"):
        spw._mat(t, None, 64, "residual")
    with pytest.raises(ValueError, match="overlap"):
        spw._rows(t, "Y")


def test_single_rows_and_padded_rows_are_taken():
    for t, rows, ld in ((half(64), 1, 64), (half(1, 64).expand(1, 64), 1, 64), (half(64).as_strided((1, 64), (0, 1)), 1, 64),
                        (half(10, 72)[:, :64], 10, 72), (half(10, 64), 10, 64), (half(0, 64), 0, 64),
                        (half(20, 64)[::2], 10, 128)):
        v, m, got = spw._mat(t, None, 64, "x")
        assert (m, got, v.shape) == (rows, ld, (rows, 64))
        v, got = spw._rows(t, "x")
        assert got == ld and v.shape == (rows, 64)


def meta(rows, cols, ld):
    """A view without storage: sizes and strides alone."""
    return torch.empty(0, dtype=torch.float16, device="meta").as_strided((rows, cols), (ld, 1))


@pytest.mark.parametrize("rows,ld", [(2, 2 ** 31), (2, 2 ** 32 + 64), (2 ** 31, 64), (2 ** 32 + 5, 64)])
def test_sizes_past_31_bits_are_refused(rows, ld):
    # the library's M and ld are C ints, and ctypes keeps the low 32 bits of what it is given
    with pytest.raises(ValueError, match="2147483647"):
        spw._mat(meta(rows, 64, ld), None, 64, "X")
    with pytest.raises(ValueError, match="2147483647"):
        spw._rows(meta(rows, 64, ld), "Y")


def test_largest_sizes_and_a_single_row_of_any_stride():
    assert spw._mat(meta(2 ** 31 - 1, 64, 64), None, 64, "X")[1:] == (2 ** 31 - 1, 64)
    assert spw._mat(meta(2, 64, 2 ** 31 - 8), None, 64, "X")[2] == 2 ** 31 - 8
    assert spw._mat(meta(1, 64, 2 ** 33), None, 64, "X")[1:] == (1, 64)
    assert spw._rows(meta(1, 64, 2 ** 33), "Y")[1] == 64

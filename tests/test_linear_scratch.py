"""The scratch of red_linear_logprob_grad at many rows: no piece of the vocabulary without a limit."""
import pytest


@pytest.fixture(scope="module")
def itr():
    from int_tensor_reductions_gb300 import _build
    import int_tensor_reductions_gb300 as itr
    _build.build_lib()
    return itr


@pytest.mark.parametrize("rows", [129, 1000, 8192, 32768, 32769, 65536, 131072, 200000, 1 << 18, 1 << 20, 1 << 22, 1 << 24])
@pytest.mark.parametrize("vocab", [1, 300, 385, 4096, 65536, 131072, 1 << 20])
def test_scratch_of_many_rows(itr, rows, vocab):
    size = itr.lib().red_linear_work_bytes(rows, 64, vocab, 1)
    padded = (rows + 255) // 256 * 256
    piece = max((384 << 20) if rows <= 32768 else min(padded * 12288, 12 << 30), padded * 1024)
    # packed hidden states and sums of dh (in shares of the vocabulary, where rows are few), six words of each row
    tiles = padded // 256
    shares = max(1, 72 // tiles)
    assert 0 < size <= piece + padded * (64 * 2 + 64 * 4 * shares + 24) + 4096


def test_scratch_of_very_many_rows(itr):
    """8 GiB of g at 2^20 rows, and no more beyond."""
    size = itr.lib().red_linear_work_bytes
    for rows in (1 << 20, 1 << 21, 1 << 22, 1 << 24):
        assert size(rows, 8, 65536, 1) <= (8 << 30) + rows * 128

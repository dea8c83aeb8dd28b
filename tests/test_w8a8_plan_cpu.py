"""The int8 product's choice of parts along K, through the room it asks for (no GPU needed)."""
import pytest

import gemm_w4a16_amd as w

W8 = w.W4A16_FMT_W8_ROW_FP32


@pytest.mark.parametrize("M,N,K", [(1, 4096, 24576), (2, 4096, 24576), (2, 8192, 24576), (1, 4096, 32768), (16, 4096, 24576)])
def test_no_parts_where_weights_are_read_once(M, N, K):
    """Weights of more than 64 MiB that one row tile reads are copied past the Infinity Cache by the unsplit
    product, faster than parts are copied: at two rows of 4096 x 24576 the unsplit one takes 27.5 us and parts
    took 35.2, so no room for their sums is asked for."""
    assert w.w4a16_w8a8_workspace_bytes(W8, M, N, K) == M * K + 4 * M


@pytest.mark.parametrize("M,N,K", [(60, 4096, 24576), (64, 8192, 16384), (100, 4096, 14336), (512, 4096, 14336)])
def test_parts_where_they_gain(M, N, K):
    """More rows of as long a K: 60 rows of 4096 x 24576 take 26.7 us in parts and 32.9 without."""
    assert w.w4a16_w8a8_workspace_bytes(W8, M, N, K) >= M * K + 4 * M + 2 * 4 * M * N

"""Sizes at the end of 32 bits, by the library's host checks (no GPU): the products count rows and
columns in tiles of 256 with 32-bit numbers, so a size that rounds up past 2^31 - 1 is refused; it
used to come out as no tiles at all, and an output that nothing had written."""
import pytest

from bit_matmul_decomposition_b200 import abi, build

INVALID = 1
F = 0x10000     # aligned, never dereferenced: validation rejects before any launch
MOST = (1 << 31) - 256
PAST = [MOST + 1, (1 << 31) - 1]
PAST16 = [MOST + 16, (1 << 31) - 16]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load()


def test_the_largest_sizes_are_taken(lib):
    assert (MOST + 255) % (1 << 32) < 1 << 31 and MOST % 256 == 0
    for size in (lib.i8_block_linear_workspace_size, lib.i8_block_linear_backward_workspace_size):
        assert size(MOST, 1, 16) > 0 and size(1, MOST, 16) > 0 and size(1, 1, MOST) > 0
    for size in (lib.i8_experts_workspace_size, lib.i8_experts_backward_workspace_size):
        assert size(MOST, 16, 16, 4, 1) > 0 and size(MOST // 2, 16, 16, 4, 2) > 0 and size(1, MOST, 16, 4, 1) > 0


@pytest.mark.parametrize("past", PAST)
def test_rows_and_outputs_past_the_last_tile(lib, past):
    big = 1 << 62
    for size in (lib.i8_block_linear_workspace_size, lib.i8_block_linear_backward_workspace_size):
        assert size(past, 1, 16) == 0 and size(1, past, 16) == 0
    for t, n in ((past, 1), (1, past)):
        assert lib.i8_block_linear_forward(F, 1, t, 16, F, F, None, n, F, F, big, None) == INVALID
        assert lib.i8_block_linear_backward(F, F, 1, t, n, 16, F, F, F, F, F, F, big, None) == INVALID
    for size in (lib.i8_experts_workspace_size, lib.i8_experts_backward_workspace_size):
        assert size(past, 16, 16, 4, 1) == 0 and size(1 << 30, 16, 16, 4, 2) == 0
    assert lib.i8_experts_forward(F, 1, past, 16, F, F, 1, F, F, F, F, 4, 16, F, None, F, big, None) == INVALID
    assert lib.i8_experts_backward(F, 1, past, 16, F, F, 1, F, F, F, F, 4, 16, F, F, F, F, big, None) == INVALID


@pytest.mark.parametrize("past", PAST16)
def test_features_past_the_last_tile(lib, past):
    big = 1 << 62
    for size in (lib.i8_block_linear_workspace_size, lib.i8_block_linear_backward_workspace_size):
        assert size(1, 1, past) == 0
    assert lib.i8_block_linear_forward(F, 1, 1, past, F, F, None, 1, F, F, big, None) == INVALID
    assert lib.i8_block_linear_backward(F, F, 1, 1, 1, past, F, F, F, F, F, F, big, None) == INVALID
    for size in (lib.i8_experts_workspace_size, lib.i8_experts_backward_workspace_size):
        assert size(1, past, 16, 4, 1) == 0 and size(1, 16, past, 4, 1) == 0

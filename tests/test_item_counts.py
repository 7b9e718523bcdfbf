"""Work items are counted in an int that the narrow kernels' CTAs step past the end of the list by a grid: calls whose items
come within a grid of the largest int are refused on the host (no GPU needed)."""
import pytest

import test_bf16_arguments as bf16
import test_fp8_arguments as fp8

UNSUPPORTED = bf16.UNSUPPORTED


@pytest.mark.parametrize("naive", [bf16._naive, fp8._naive])
@pytest.mark.parametrize("below", [1, 100])
def test_items_near_the_largest_int(naive, below):
    # pairs by two tiles of 128 columns: 2^31 - 2 * below items
    assert naive(M=(1 << 30) - below, topk=1, E=1, N=129, ldy=136) == UNSUPPORTED

"""Sizes whose products pass 64 bits are refused on the host (no GPU needed)."""
import ctypes

import pytest

import shape_driven_tile_gb300 as sdt
from test_paged_args import A, SHAPE, cache


@pytest.mark.parametrize("tokens", [(1 << 60) + 1, 1 << 62, (1 << 63) - 1, 1 << 32, ((1 << 31) - 1) // 16])
def test_append_of_more_tokens_than_it_counts(tokens):
    """16 pieces a token: the products wrap to 16, 0 and -16, or pass 2^31."""
    c = cache()
    assert sdt.lib().paged_append(tokens, A, 128, 64, A, 128, 64, 1, A, ctypes.byref(c), None) == SHAPE

"""Host checks of the paged attention's sizes at the ends of their types (CPU only)."""

import pytest

from deepseek_v4_top_gb300 import dsa

FAKE = 1 << 20     # a 16-byte-aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from deepseek_v4_top_gb300 import build
    build.build()
    return dsa.load()


@pytest.mark.parametrize("B,T,H", [((1 << 31) - 1, (1 << 31) - 1, 64), ((1 << 31) - 1, 1 << 30, 64), (1 << 30, 4, 1), (1 << 28, 1, 8)])
def test_sizes_whose_product_is_too_large(lib, B, T, H):
    """The product of the first two passes 64 bits: the rows are refused before they are multiplied by the heads."""
    assert lib.dsa_paged_attn(FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0.1, FAKE, FAKE, 1 << 30, B, T, H, 8, 64, 16, 1,
                              None) == dsa.DSA_ERR_INVALID_ARG
    assert lib.dsa_paged_sparse_attn(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0.1, FAKE, FAKE, 1 << 30, B, T, H, 8, 64, 16,
                                     4, 1, None) == dsa.DSA_ERR_INVALID_ARG

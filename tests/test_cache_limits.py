"""Sizes at the edge of what the cache's calls take. Needs no GPU."""
import pytest

from mask_aware_exact_gb300 import flashmask as fm


@pytest.fixture(scope="module", autouse=True)
def lib():
    from mask_aware_exact_gb300 import build
    build.build()
    return fm.load()


def test_pages_of_all_segments():
    # B * Hk * row tiles * max_pages is counted in 32 bits, and rounded up to whole
    # runs of up to 256 CTAs: 2^31 - 8 pages would pass 2^31
    size = fm.flashmask_cache_workspace_bytes
    assert 18705 * 8 * 14351 == 2 ** 31 - 8
    assert size(18705, 8, 8, 1, 64, 14351) == 0
    assert size(18705, 8, 8, 1, 64, 14350) > 0
    # 32 rows are two tiles: half as many pages
    assert size(18705, 16 * 8, 8, 2, 64, 7176) == 0
    assert size(18705, 16 * 8, 8, 2, 64, 7175) > 0

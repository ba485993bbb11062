"""Calls of the paged 8-bit context cache that need no GPU."""
import pytest

import speculative_block_draft_gb300 as pkg


@pytest.fixture(scope="module")
def lib():
    pkg.build()
    return pkg.lib()


def test_wait_hooks_refuse_no_cache(lib):
    assert lib.dflash_cache_set_wait_limit(None, 1000) == pkg.DFLASH_EINVAL
    assert lib.dflash_cache_debug_stall(None, 0) == pkg.DFLASH_EINVAL

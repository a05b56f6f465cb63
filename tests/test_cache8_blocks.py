"""Numbers of blocks past a page's are refused, those too whose product with 16 passes 32 bits (no GPU needed)."""

import pytest

from io_aware_exact_04_gb300 import _lib
from tests.test_cache8_abi import A, UNSUPPORTED


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("more", [1 << 28, 3 << 28, 7 << 28, 1 << 27, (1 << 31) - 256])
def test_too_many_blocks(built, page, more):
    lib = _lib.load("libfa.so")
    pool = _lib.Pool(A, 1 << 20, 1, 8, 2, page, 64, A, A, 4, 4)
    for extra in (0, 1, page // 16):
        scales = _lib.PoolScales(A, 0, more + extra)
        assert lib.fa_cache_update_8bit(pool, scales, A, A, A, A, 1 << 30, None) == UNSUPPORTED
        assert lib.fa_cache_compact_8bit(pool, scales, A, A, 1 << 30, None) == UNSUPPORTED

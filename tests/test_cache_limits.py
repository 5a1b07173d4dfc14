"""Sizes at which the 32-bit positions of the paged cache operators would run
out are refused before any launch (no GPU)."""
import ctypes

import pytest

import sparse_attention_20_b200 as dsa
from sparse_attention_20_b200 import build as dsa_build

FAKE = ctypes.c_void_p(0x10000)          # aligned, never dereferenced: checks fail first


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa.load_library()


@pytest.mark.parametrize("mass", [FAKE, None])
@pytest.mark.parametrize("max_pages,page_size,keep", [
    ((1 << 24) + 1, 64, 100),            # 2^30 + 64 positions
    (33554431, 64, 100),                 # the last table below 2^31
    (4, 64, (1 << 30) + 1),
    (4, 64, 2 ** 31 - 1),
])
def test_compaction_refuses_positions_beyond_2_30(lib, max_pages, page_size, keep, mass):
    before = dsa.launch_count()
    rc = lib.dsa_cache_compact_paged(FAKE, 1152, FAKE, 128, 8, page_size, FAKE, 2, max_pages, FAKE, keep, FAKE, mass,
                                     None)
    assert rc == -2 and b"supported" in lib.dsa_last_error() and dsa.launch_count() == before

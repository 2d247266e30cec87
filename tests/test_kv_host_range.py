"""Limits of the key/value cache calls, checked on the host before any CUDA call."""
import pytest

from tests.test_kv_host import append, attention, cache, moe  # noqa: F401


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_positions_do_not_wrap_around(moe, page_size):  # noqa: F811
    """The kernels look pages up ahead of a sequence's end: up to 32 tiles of 64 keys and a
    step in the one for few rows, 64 groups of 16 keys and a block in the one for many.  A
    length next to 2^31 would turn such a position negative, and the lookup, which only
    compares it with the length, would read in front of the page table."""
    longest = ((1 << 31) - (1 << 16)) // page_size
    ahead = max(32 * 64 + 64, (64 + 8) * 16 + 128)
    assert longest * page_size + ahead < 1 << 31
    for pages in (longest + 1, ((1 << 31) - 1) // page_size):
        assert append(moe, cache(moe, page_size=page_size, max_pages=pages)) == -2
        assert attention(moe, cache(moe, page_size=page_size, max_pages=pages))[0] == -2

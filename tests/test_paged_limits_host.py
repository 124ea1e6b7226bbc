"""The longest sequence that a page table may describe, whose 32-bit places the kernels go beyond, and the widest window (no GPU needed)."""
import ctypes

import pytest

from tests import attention_launches as L
from tests.test_attention_host import append_args, attention_args, calls, fb, layer  # noqa: F401

MOST = 2 ** 31 - 2 ** 16
AHEAD = 8 * 32 + 31 * 8 * 32 + 64  # keys that a look-up, a load or a count of tiles goes beyond the last one: see below


def test_places_beyond_the_last_key_fit_32_bits():
    """32 tiles' pages of eight waves are looked up at once, 64 keys taken at a time, lengths rounded up to 64."""
    assert MOST + AHEAD < 2 ** 31


@pytest.mark.parametrize("page", [16, 64, 1024, 65536])
def test_longer_tables_are_refused(fb, page):  # noqa: F811
    most = MOST // page
    for pages, status in ((most, fb.OK), (most + 1, 2), (2 ** 31 // page - 1, fb.OK if page == 65536 else 2)):
        b = fb.PagedBatch(**L.batch(page_size=page, table_pages=pages, table_ld=pages))
        assert fb.raw_status("fluxbin_paged_attention_workspace_size", ctypes.byref(b), ctypes.byref(ctypes.c_size_t())) == status
        if status:
            assert fb.raw_status("fluxbin_paged_attention", *attention_args(fb, batch=b)) == status
            assert fb.raw_status("fluxbin_rope_append", *append_args(fb, batch=b)) == status


@pytest.mark.parametrize("window", [-1, 1 << 31, 1 << 32])
def test_windows_that_attention_would_refuse_or_misread(calls, window):  # noqa: F811
    """Refused before anything is appended: 2^32 would have come through as 0, no window."""
    with pytest.raises(ValueError, match="window"):
        layer(window=window)
    assert not calls
    assert layer(window=(1 << 31) - 1).window == 2 ** 31 - 1

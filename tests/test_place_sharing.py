"""Memory that the moves inside the cache share: keys and values of one tensor
(no GPU: every call here returns before any CUDA work)."""

import pytest

from tests.test_place_checks import _compact, lib  # noqa: F401
from tests.test_token_checks import _cache

FAR = 1 << 30                                                # bytes from k to v, past either


def _layout(**kw):
    a = dict(k=4096, v=4096 + FAR, pages=10, heads=2, page_size=16, head_dim=64, k_page=2048, k_head=1024, k_row=64, v_page=2048,
             v_head=1024, v_row=64)
    a.update(kw)
    return _cache(**a)


# Rows that meet, each in its own way: the moves of one would overwrite what the other has still to read.
@pytest.mark.parametrize("kw", [
    dict(v=4096 + 16),                                       # a row's channels, 8 further on
    dict(v=4096 + 2 * 64),                                   # the next row
    dict(v=4096 + 2 * (1024 - 56)),                          # the end of a head and the start of the next
    dict(v=4096 + 2 * 2048 * 9 + 2 * 2040),                  # the last channels of the last page
    dict(v=4096, v_head=64, v_row=128),                      # the same pages, laid out otherwise
    dict(v=4096 + 2 * 64 * 16, v_page=1024, v_head=10240),   # pages of one head beside each other
    dict(k_page=4096, v_page=4096, v=4096 + 2 * 2048 - 16),  # nearly a half of each page of its own
    dict(pages=2 ** 30, k_page=2 ** 39, v_page=2 ** 39, v=4096 + 2 * 2 ** 59 + 16),  # past 64 bits in the sums
    dict(pages=1, heads=1, page_size=1, v=4096 + 2 * 56),    # a single row
])
def test_rows_that_meet_are_refused(lib, kw):  # noqa: F811
    assert _compact(lib, c=_layout(**kw)) == 1, kw
    assert b"memory in common" in lib.wan_vae_last_error()

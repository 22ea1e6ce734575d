"""Memory that the moves inside the cache share: keys and values of one tensor,
pages of several sequences (no GPU: every call here returns before any CUDA work)."""

import pytest
import torch

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


# ---------------------------------------------------------- the host's check of a compaction
def _i(v):
    return torch.tensor(v, dtype=torch.int32)


def _check(pages, lengths, first, keeps, size=16, n_pages=40):
    import video_vae_decoding_gb300 as wv
    cu = [sum(len(k) for k in keeps[:b]) for b in range(len(keeps) + 1)]
    wv.kv_check(_i(pages), _i(lengths), size, n_pages, _i(cu), first=_i(first), keep=_i(sum(map(list, keeps), [])))


SHARED = [[0, 1, 2, 3, 4], [0, 1, 2, 20, 21], [0, 1, 2, 30, 31]]    # a past of 48 keys in pages common to three sequences


def test_check_of_compactions_behind_common_pages(lib):  # noqa: F811
    _check(SHARED, [60, 70, 70], [60, 50, 48], [[], [51, 55, 69], range(52, 70)])
    _check(SHARED, [60, 70, 70], [60, 40, 48], [[], [*range(40, 48), 48, 60], []])   # what stays in its place is not written
    _check([[0, 1, 2, 3, 4]], [70], [4], [range(30, 70)])                # alone in the table
    _check([[-1, 7, -1, 3, 4]], [70], [20], [range(50, 60)])             # pages that no key moves from or to
    _check(SHARED, [0, 0, 0], [0, 0, 0], [[], [], []])
    _check([[0, 1], [2, 1]], [20, 18], [18, 18], [[19], []], size=12)    # row 6 of page 1: the second has six rows of it


def test_check_of_compactions_inside_common_pages(lib):  # noqa: F811
    import video_vae_decoding_gb300 as wv
    for lengths, first, keeps, names in (
            ([60, 70, 70], [60, 47, 70], [[], [50], []], "sequence 0: key 47 .* place 47 of sequence 1"),
            ([48, 70, 70], [48, 6, 70], [[], range(31, 70), []], "sequence 0: key 6 .* of sequence 1"),
            ([0, 70, 70], [0, 6, 6], [[], range(31, 70), range(31, 70)], "sequence 2: place 6 shares its row with place 6 of sequence 1"),
            ([10, 70, 40], [10, 20, 40], [[], [69], []], "sequence 2: key 20 .* of sequence 1")):
        with pytest.raises(wv.WanError, match=names):
            _check(SHARED, lengths, first, keeps)
    with pytest.raises(wv.WanError, match="sequence 0: key 36 .* place 4 of sequence 0"):   # a page twice in one row
        _check([[0, 1, 0, 3, 4]], [70], [4], [[50]])


def test_check_of_compactions_that_cannot_be(lib):  # noqa: F811
    import video_vae_decoding_gb300 as wv
    for pages, lengths, first, keeps, names in (
            ([[0, 1]], [30], [4], [[3]], "key 3 of 30 cannot move to place 4"), ([[0, 1]], [30], [4], [[9, 9]], "key 9"),
            ([[0, 1]], [30], [4], [[9, 30]], "key 30"), ([[0, 1]], [30], [31], [[]], "31 first keys of 30"),
            ([[0, 1]], [30], [-1], [[]], "first keys"), ([[0, 1]], [33], [4], [[5]], "length 33"),
            ([[0, 40]], [30], [4], [[17]], "page 1 is number 40"), ([[-1, 1]], [30], [4], [[17]], "page 0 is number -1")):
        with pytest.raises(wv.WanError, match=names):
            _check(pages, lengths, first, keeps)
    table, one = _i([[0, 1]]), _i([1])
    for kw in (dict(first=one), dict(keep=one), dict(first=one, keep=one), dict(cu_tokens=_i([0, 1]), first=one, keep=one, append=True),
               dict(cu_tokens=_i([0, 1]), first=one, keep=one, tokens=1), dict(cu_tokens=_i([0, 1]), first=_i([1, 2]), keep=one),
               dict(cu_tokens=_i([0, 1]), first=one, keep=one.long()), dict(cu_tokens=_i([0, 1, 1]), first=one, keep=one),
               dict(cu_tokens=_i([0, 1]), first=one, keep=_i([1, 2, 3])[::2])):
        with pytest.raises(ValueError):
            wv.kv_check(table, one, 16, 9, **kw)
    with pytest.raises(wv.WanError, match="range is none"):
        wv.kv_check(table, _i([30]), 16, 9, _i([0, 2]), first=one, keep=one)

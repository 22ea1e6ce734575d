"""Moves inside the cache where keys and values, or sequences, share memory."""

import pytest
import torch

from tests import place_reference as place
from tests import token_reference as ref
from tests.gpu_util import lib_ready
from tests.test_gpu_places import HALVES, _i32, _keeps, _randn, _status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wv():
    return lib_ready()


def _compact(wv, kc, vc, pages, first, keeps):
    status = _status()
    cu = [sum(len(k) for k in keeps[:b]) for b in range(len(keeps) + 1)]
    got = wv.kv_compact(kc, vc, pages, _i32(first), _i32(sum(keeps, [])), _i32(cu), status=status)
    wv.kv_status(status)
    return got.tolist()


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("kind", ["path", "rolled", "all", "choice"])
@pytest.mark.parametrize("case", [([40, 0, 17], 2, 128, 16), ([900, 333], 3, 80, 24), ([3000], 1, 256, 390), ([700] * 9, 1, 72, 7),
                                  ([60] * 200, 1, 64, 16), ([300, 500] * 3, 4, 128, 32)],
                         ids=lambda c: "b{}n{}h{}d{}p{}".format(len(c[0]), max(c[0]), *c[1:]))
def test_keys_that_are_their_own_values_move_once(wv, case, kind, dtype):
    """k and v one tensor: what a second move in place would make of the rows is not what was asked for."""
    lens, hk, D, size = case
    pages, _, n = ref.tables(lens, size)
    c = _randn(n, hk, size, D, dtype=dtype, seed=1)
    first, keeps = _keeps(kind, lens)
    want, _, lengths = place.compact(c, c, pages, first, keeps)
    assert _compact(wv, c, c, pages, first, keeps) == lengths
    assert torch.equal(c, want)


@pytest.mark.parametrize("layout", ["pages", "rows", "turned"])
def test_keys_and_values_interleaved(wv, layout):
    """Caches in one allocation whose rows have no memory in common."""
    lens, hk, size, D = [333, 40, 500], 2, 16, 64
    pages, _, n = ref.tables(lens, size)
    if layout == "pages":
        both = _randn(n, 2, hk, size, D, dtype=torch.bfloat16, seed=1)
        kc, vc = both[:, 0], both[:, 1]
    elif layout == "rows":
        both = _randn(n, hk, size, 2, D, dtype=torch.bfloat16, seed=1)
        kc, vc = both[..., 0, :], both[..., 1, :]
    else:                                                    # each page's values by rows, its keys by heads
        both = _randn(n, 2, hk * size * D, dtype=torch.bfloat16, seed=1)
        kc, vc = both[:, 0].view(n, hk, size, D), both[:, 1].view(n, size, hk, D).transpose(1, 2)
    first, keeps = _keeps("choice", lens)
    want = place.compact(kc.clone(), vc.clone(), pages, first, keeps)
    assert _compact(wv, kc, vc, pages, first, keeps) == want[2]
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_keys_and_values_that_overlap_are_refused(wv):
    both = _randn(9, 1, 16, 72, dtype=torch.bfloat16)
    before = both.clone()
    pages = _i32([[0, 1, 2]])
    for kc, vc in (both[..., :64], both[..., 8:]), (both[:8], both[1:]):
        with pytest.raises(wv.WanError, match="memory in common"):
            wv.kv_compact(kc, vc, pages, _i32([2]), _i32([5, 9]), _i32([0, 2]))
    assert torch.equal(both, before)


def _host_check(wv, pages, lengths, size, n, first, keeps):
    cpu = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    cu = [sum(len(k) for k in keeps[:b]) for b in range(len(keeps) + 1)]
    wv.kv_check(pages.cpu(), cpu(lengths), size, n, cpu(cu), first=cpu(first), keep=cpu(sum(keeps, [])))


@pytest.mark.parametrize("share", [True, False], ids=["share", "copy"])
def test_fork_then_compact(wv, share):
    """Futures of one past: behind its common pages each keeps what it likes, and the past and the others stay; inside them
    only a future that was copied whole may roll on."""
    size, hk, D, past = 16, 2, 64, 70
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    table[0, :5] = torch.arange(5)
    fresh = torch.arange(10, 20, dtype=torch.int32, device="cuda").view(2, 5)
    kc, vc = (_randn(40, hk, size, D, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    lengths = _i32([past, 0, 0])
    wv.kv_fork(kc, vc, table, lengths, _i32([0, 0]), _i32([1, 2]), fresh[:, :1].contiguous() if share else fresh, share)
    table[1, 5:], table[2, 5:] = _i32([20, 21, 22]), _i32([30, 31, 32])
    lens = [past, 100, 110]                                  # both went on
    first, keeps = [past, 66, 70], [[], [68, 75, *range(80, 99)], list(range(90, 110))]
    _host_check(wv, table, lens, size, 40, first, keeps)
    before = [ref.keys_of(c, table[b], lens[b], h) for c in (kc, vc) for b in range(3) for h in range(hk)]
    want = place.compact(kc, vc, table, first, keeps)
    assert _compact(wv, kc, vc, table, first, keeps) == want[2]
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    kept = [list(range(f)) + k for f, k in zip(first, keeps)]
    after = [ref.keys_of(c, table[b], len(kept[b]), h) for c in (kc, vc) for b in range(3) for h in range(hk)]
    for i, (x, y) in enumerate(zip(before, after)):
        assert torch.equal(x[kept[i // hk % 3]], y)
    # the first future rolls on behind 6 first keys
    lens, first, keeps = want[2], [past, 6, want[2][2]], [[], list(range(50, want[2][1])), []]
    if share:
        with pytest.raises(wv.WanError, match="sequence 0: key 6 .* sequence 1"):
            _host_check(wv, table, lens, size, 40, first, keeps)
        return
    _host_check(wv, table, lens, size, 40, first, keeps)
    assert _compact(wv, kc, vc, table, first, keeps) == [past, 6 + len(keeps[1]), lens[2]]
    rolled = [*range(6), *keeps[1]]
    for i, y in enumerate(after):
        c, b, h = (kc, vc)[i // (3 * hk)], i // hk % 3, i % hk
        assert torch.equal(ref.keys_of(c, table[b], len(rolled) if b == 1 else lens[b], h), y[rolled] if b == 1 else y)

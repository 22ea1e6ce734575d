"""Attention by place (a window with first keys, a tree of drafts) and the moves
inside the cache (forks, compaction) on the GPU, against plain forms, and runs of
them together."""

import math

import pytest
import torch

from tests import place_reference as place
from tests import token_reference as ref
from tests.gpu_util import lib_ready

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def wv():
    return lib_ready()


def _randn(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _case(lens, new, hk, g, D, size, dtype, sees=None, room=0, seed=0):
    """A cache whose rows that nobody sees hold NaN, and whose pages that nobody sees have numbers that are none."""
    pages, lengths, n_pages = ref.tables(lens, size, seed=seed)
    more = max(0, -(-room // size) - pages.shape[1])
    pages = torch.cat([pages, torch.full((len(lens), more), -7, dtype=torch.int32, device="cuda")], 1)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    kc, vc = (_randn(n_pages, hk, size, D, dtype=dtype, seed=seed + i) for i in (1, 2))
    if sees is not None:
        held = torch.zeros(n_pages, size, dtype=torch.bool, device="cuda")
        for b, s in enumerate(sees):
            live = s.any(0) if s.shape[0] else torch.zeros(s.shape[1], dtype=torch.bool)
            at = live.nonzero()[:, 0].cuda()
            held[pages[b][at // size].long(), at % size] = True
            used = set((at // size).tolist())
            for j in range(pages.shape[1]):
                if j not in used:
                    pages[b, j] = -1 if j % 2 else n_pages + j
        hidden = ~held[:, None, :, None].expand_as(kc)
        kc[hidden], vc[hidden] = math.nan, math.nan
    q = _randn(cu[-1], hk * g, D, dtype=dtype, seed=seed + 3, scale=1.5)
    return q, kc, vc, pages, lengths, _i32(cu)


def _check(call, q, kc, vc, pages, lengths, cu, sees):
    """Two rows behind the last sequence stay as they are; the same bits come twice."""
    status = _status()
    wide, T = torch.cat([q, torch.ones_like(q[:1]).expand(2, -1, -1)]), q.shape[0]
    out = torch.full_like(wide, 7.0)
    got, lse = call(wide, out=out, return_lse=True, status=status)
    wv_status = status.item()
    assert wv_status == 0, wv_status
    assert got is out and bool((out[T:] == 7.0).all())
    ref.check_attention(got[:T], lse[:T], place.attention(q, kc, vc, pages, lengths, cu, sees))
    again = call(wide, out=torch.full_like(wide, 7.0), return_lse=True, status=None)
    assert torch.equal(again[0], got) and torch.equal(again[1][:T], lse[:T])


# ------------------------------------------------------------------- window
# lens, new (None: one each), kv heads, group, head dim, page size, window, sinks, frame
WINDOW = [
    ([1], None, 1, 1, 64, 16, 1, 0, 1), ([1, 0, 2, 15, 16, 17], None, 2, 1, 128, 16, 5, 2, 1),
    ([300, 64, 65, 1000], None, 1, 4, 128, 64, 100, 4, 1), ([1000], None, 16, 1, 128, 16, 300, 16, 1),
    ([5, 700, 33], None, 4, 5, 80, 24, 33, 17, 1), ([257, 31], None, 2, 16, 64, 1, 40, 3, 1),
    ([90, 391], None, 1, 17, 96, 7, 50, 60, 1), ([300, 1, 299], None, 3, 8, 256, 100, 128, 33, 1),
    ([5000, 12], None, 2, 8, 128, 256, 1, 1, 1), ([2000], None, 1, 40, 8, 390, 64, 400, 1),
    ([881, 1761], None, 2, 2, 128, 880, 1, 440, 440), ([333], None, 1, 2, 64, 16, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1),
    ([170] * 90, None, 1, 2, 72, 32, 48, 8, 3),
    ([5], [5], 1, 1, 64, 16, 2, 1, 1), ([40, 0, 3], [7, 0, 3], 2, 3, 128, 16, 4, 1, 2),
    ([200, 130], [130, 1], 2, 1, 128, 64, 30, 4, 1), ([700, 64, 300], [300, 64, 5], 1, 4, 64, 32, 60, 16, 1),
    ([900], [440], 3, 1, 128, 220, 1, 110, 110), ([1513, 1000], [257, 512], 2, 5, 80, 24, 200, 7, 1),
    ([400, 77], [129, 77], 1, 2, 256, 100, 3, 50, 20), ([350], [350], 2, 2, 96, 7, 9, 100, 1),
    ([3000], [128], 1, 8, 128, 128, 128, 128, 1), ([260, 130], [260, 130], 1, 1, 16, 1, 33, 0, 1),
    ([4400], [880], 2, 1, 128, 880, 2, 880, 880), ([1500], [150], 1, 48, 64, 16, 70, 20, 1),
    ([3000, 20], [2, 20], 4, 2, 128, 256, 10, 700, 100), ([2600], [300], 2, 1, 64, 390, 90, 200, 1),
    ([4000, 700], [200, 150], 1, 1, 256, 256, 500, 300, 1), ([1513], [400], 1, 2, 192, 24, 64, 1000, 7),
    ([900], [300], 1, 16, 144, 8, 40, 5, 1), ([1290], [400], 2, 2, 128, 16, 2, 130, 129),
    ([600], [200], 1, 2, 64, 8, 100, 37, 1), ([600, 250], [100, 200], 2, 2, 128, 128, 50, 130, 1), ([3000], [300], 1, 1, 128, 16, 1000, 16, 1),
    ([900], [250], 1, 4, 256, 32, 5, 70, 33), ([700], [260], 1, 1, 64, 40, 90, 41, 1),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "t{}n{}h{}g{}d{}p{}w{}s{}f{}".format(sum(c[1] or [len(c[0])]), max(c[0]), *c[2:]))
@pytest.mark.parametrize("room", [0, 40_000], ids=["tight", "roomy"])
def test_window(wv, case, dtype, room):
    lens, new, hk, g, D, size, window, sinks, frame = case
    step = new is None
    new = [1] * len(lens) if step else new
    sees = [place.window_sees(n, min(n, m), window, sinks, frame) if n else torch.zeros(m, 0, dtype=torch.bool)
            for n, m in zip(lens, new)]
    q, kc, vc, pages, lengths, cu = _case(lens, new, hk, g, D, size, dtype, sees, room)
    told = 0 in [n for n, m in zip(lens, new) if m > n]      # a new token of a sequence without a key has no place

    def call(x, status=None, **kw):
        got = wv.kv_window_attention(x, kc, vc, pages, lengths, window, sinks, frame, None if step else cu, status=status, **kw)
        if told and status is not None:
            with pytest.raises(wv.WanError, match="length or token range"):
                wv.kv_status(status)
        return got
    _check(call, q, kc, vc, pages, lengths, cu, sees)


# --------------------------------------------------------------------- tree
def _tree(n, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1] * n
    if kind == "comb":                                       # a chain with a leaf at each link
        return [-1] + [(i - 1) // 2 * 2 for i in range(1, n)]
    return [-1 if i == 0 or torch.rand((), generator=g) < 0.05 else int(torch.randint(max(0, i // 3 - 2), i, (), generator=g))
            for i in range(n)]


# lens, drafts, kv heads, group, head dim, page size, kind of tree
TREE = [
    ([1], [1], 1, 1, 64, 16, "random"), ([40, 0, 3], [7, 0, 3], 2, 3, 128, 16, "random"), ([2026], [26], 16, 1, 128, 16, "random"),
    ([26, 27, 300], [26, 26, 26], 2, 1, 128, 64, "star"), ([700, 64, 300], [47, 64, 5], 4, 5, 80, 24, "random"),
    ([333], [130], 1, 1, 64, 7, "random"), ([200, 333], [100, 33], 1, 1, 128, 16, "comb"), ([150], [90], 1, 1, 96, 32, "chain"),
    ([2000], [15], 1, 2, 256, 100, "random"), ([80], [70], 1, 2, 256, 16, "roots"),
    ([500, 64, 65], [64, 64, 64], 2, 4, 128, 64, "random"), ([1000, 129], [64, 64], 1, 8, 64, 16, "comb"),
    ([400, 1300], [129, 200], 1, 2, 128, 128, "random"), ([300], [300], 1, 1, 128, 24, "chain"), ([900], [257], 2, 1, 64, 390, "random"),
    ([1000], [64], 1, 16, 256, 64, "random"), ([500, 300], [33, 1], 1, 40, 80, 8, "star"), ([2000], [280], 1, 1, 256, 256, "comb"),
    ([130] * 20, [64] * 20, 2, 2, 128, 16, "random"), ([1100], [1024], 1, 1, 64, 64, "random"),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("case", TREE, ids=lambda c: "t{}n{}h{}g{}d{}p{}{}".format(sum(c[1]), max(c[0]), *c[2:]))
@pytest.mark.parametrize("room", [0, 40_000], ids=["tight", "roomy"])
def test_tree(wv, case, dtype, room):
    lens, new, hk, g, D, size, kind = case
    trees = [_tree(m, kind, i) for i, m in enumerate(new)]
    sees = [place.tree_sees(n, t) for n, t in zip(lens, trees)]
    q, kc, vc, pages, lengths, cu = _case(lens, new, hk, g, D, size, dtype, sees, room)
    parents = _i32(sum(trees, []) + [-1, 5])                 # of the rows behind the last sequence: not looked at
    _check(lambda x, **kw: wv.kv_tree_attention(x, kc, vc, pages, lengths, parents, cu, **kw), q, kc, vc, pages, lengths, cu, sees)


def test_tree_of_one_draft_each(wv):
    """Without token ranges: a token a sequence, which sees everything."""
    q, kc, vc, pages, lengths, cu = _case([3, 500, 64], [1, 1, 1], 2, 2, 64, 16, torch.bfloat16)
    got = wv.kv_tree_attention(q, kc, vc, pages, lengths, _i32([-1, -1, -1]))
    ref.check_attention(got, None, ref.attention(q, kc, vc, pages, lengths))


@pytest.mark.parametrize("drafts", [9, 150], ids=["few", "many"])
def test_tree_with_parents_that_are_none(wv, drafts):
    """A parent that does not come before its child counts as none, and is told; no walk leaves the tree."""
    n = drafts + 60
    tree = _tree(drafts, "random")
    q, kc, vc, pages, lengths, cu = _case([n], [drafts], 1, 2, 64, 16, torch.bfloat16, room=40_000)
    for i, p in (2, 2), (3, 4), (5, 10 ** 9), (7, -2), (8, -2 ** 31):
        bad = list(tree)
        bad[i] = p
        status = _status()
        got = wv.kv_tree_attention(q, kc, vc, pages, lengths, _i32(bad), cu, status=status)
        with pytest.raises(wv.WanError, match="parent"):
            wv.kv_status(status)
        sees = [place.tree_sees(n, [p if 0 <= p < j else -1 for j, p in enumerate(bad)])]
        ref.check_attention(got, None, place.attention(q, kc, vc, pages, lengths, cu, sees))


# ------------------------------------------------------------ both of them
def _calls(wv, kind, kc, vc, pages, lengths, cu, lens, new, window=40, sinks=5, frame=1):
    """The operator on these tables, and what its rows see."""
    if kind == "window":
        sees = [place.window_sees(n, m, window, sinks, frame) for n, m in zip(lens, new)]
        return lambda q, **kw: wv.kv_window_attention(q, kc, vc, pages, lengths, window, sinks, frame, cu, **kw), sees
    trees = [_tree(m, "random", i) for i, m in enumerate(new)]
    parents = _i32(sum(trees, []))
    return (lambda q, **kw: wv.kv_tree_attention(q, kc, vc, pages, lengths, parents, cu, **kw),
            [place.tree_sees(n, t) for n, t in zip(lens, trees)])


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("new", [[1, 1], [3, 2], [150, 200]], ids=str)
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(wv, kind, new, scale):
    lens = [333, 200]
    q, kc, vc, pages, lengths, cu = _case(lens, new, 2, 2, 64, 16, torch.bfloat16, room=40_000)
    call, sees = _calls(wv, kind, kc, vc, pages, lengths, cu, lens, new)
    got, lse = call(q, scale=scale, return_lse=True)
    ref.check_attention(got, lse, place.attention(q, kc, vc, pages, lengths, cu, sees, scale=scale))


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [6, 200], ids=["few", "many"])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_odd_values_reach_the_rows_that_see_them_alone(wv, new, dtype, D, kind):
    n = 420
    q, kc, vc, pages, lengths, cu = _case([n], [new], 2, 3, D, 16, dtype, room=40_000)
    call, sees = _calls(wv, kind, kc, vc, pages, lengths, cu, [n], [new], window=60, sinks=20)
    spot = lambda i: (int(pages[0, i // 16]), i % 16)  # noqa: E731
    for i, h, c, value in ((n - 2, 0, 3, math.inf), (n - 3, 0, 4, math.nan), (n - 2, 1, D - 1, -math.inf), (n - 5, 1, 0, math.inf),
                           (n - 3, 1, 0, -math.inf), (n - 65, 0, 5, math.inf), (19, 0, 6, math.nan), (n - 70, 1, 7, math.nan)):
        p, r = spot(i)
        vc[p, h, r, c] = value
    p, r = spot(n - 1)
    kc[p, 0, r, 5] = math.nan                                 # only the last row sees this key
    got, lse = call(q, return_lse=True)
    out, err, z, zerr = place.attention(q, kc, vc, pages, lengths, cu, sees)
    assert bool(torch.isnan(got[-1, :3]).all()) and bool(torch.isnan(out[-1, :3]).all())
    ref.check_attention(got[:-1], lse[:-1], (out[:-1], err[:-1], z[:-1], zerr[:-1]))
    ref.check_attention(got[-1:, 3:], lse[-1:, 3:], (out[-1:, 3:], err[-1:, 3:], z[-1:, 3:], zerr[-1:, 3:]))


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("new", [[1, 1, 1], [2, 9, 1], [140, 70, 200]], ids=["step", "few", "many"])
def test_strides_places_and_streams(wv, new, kind):
    lens = [400, 256, 300]
    q, kc, vc, pages, lengths, cu = _case(lens, new, 2, 2, 64, 16, torch.float16, room=40_000)
    call, sees = _calls(wv, kind, kc, vc, pages, lengths, cu, lens, new)
    want = place.attention(q, kc, vc, pages, lengths, cu, sees)
    T = q.shape[0]
    turned = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc)]
    for caches in turned, (turned[0], vc):
        other, _ = _calls(wv, kind, *caches, pages, lengths, cu, lens, new)
        ref.check_attention(other(q), None, want, "rows first")
    packed = torch.zeros(T, 4 + 4, 64, dtype=torch.float16, device="cuda")
    packed[:, 2:6] = q
    out = torch.zeros(T, 9, 64, dtype=torch.float16, device="cuda")[:, 3:7]
    assert call(packed[:, 2:6], out=out) is out
    ref.check_attention(out, None, want, "views")
    flat = torch.zeros(T * 256 + 3, dtype=torch.float16, device="cuda")[3:].view(T, 4, 64)   # off 16-byte boundaries
    flat.copy_(q)
    assert call(flat, out=flat) is flat
    ref.check_attention(flat, None, want, "in place")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(q, stream=side)
    side.synchronize()
    ref.check_attention(got, None, want, "stream")


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("new", [[2, 1, 3, 5], [70, 30, 200, 100]], ids=["few", "many"])
def test_what_is_not_there_is_left_out(wv, new, kind):
    lens, size = [100, 40, 300, 200], 16
    q, kc, vc, pages, lengths, cu = _case(lens, new, 1, 2, 64, size, torch.bfloat16, room=40_000)
    call, sees = _calls(wv, kind, kc, vc, pages, lengths, cu, lens, new, window=50, sinks=10)
    good = place.attention(q, kc, vc, pages, lengths, cu, sees)
    status = _status()
    # a page that is none: its keys are hidden
    old = pages[0, 5].item()
    pages[0, 5] = kc.shape[0]
    got = call(q, status=status)
    with pytest.raises(wv.WanError, match="outside the cache"):
        wv.kv_status(status)
    pages[0, 5] = old
    less = [s.clone() for s in sees]
    less[0][:, 80:96] = False
    ref.check_attention(got, None, place.attention(q, kc, vc, pages, lengths, cu, less))
    # a sequence without a key, one of fewer keys than new tokens, one longer than its table: zeros, and the word tells
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    rows = slice(int(cu[1]), int(cu[2]))
    keep[rows] = False
    for n in 0, new[1] - 1, pages.shape[1] * size + 1, -1:
        lengths[1] = n
        got, lse = call(q, status=status, return_lse=True)
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        assert not got[rows].any() and bool(torch.isinf(lse[rows]).all())
        ref.assert_rounded(got[keep], good[0][keep], good[1][keep])
    lengths[1] = lens[1]


@pytest.mark.parametrize("drafts", [1024, 1025])
def test_most_drafts_of_a_tree(wv, drafts):
    """One more than a tree may have: zeros and a code; the other sequence as ever."""
    lens, new = [1300, 90], [drafts, 70]
    q, kc, vc, pages, lengths, cu = _case(lens, new, 1, 1, 64, 64, torch.bfloat16)
    trees = [_tree(m, "chain") for m in new]
    status = _status()
    got, lse = wv.kv_tree_attention(q, kc, vc, pages, lengths, _i32(sum(trees, [])), cu, status=status, return_lse=True)
    want = place.attention(q, kc, vc, pages, lengths, cu, [place.tree_sees(n, t) for n, t in zip(lens, trees)])
    if drafts > 1024:
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        assert not got[:drafts].any() and bool(torch.isinf(lse[:drafts]).all())
        ref.check_attention(got[drafts:], lse[drafts:], tuple(t[drafts:] for t in want))
    else:
        wv.kv_status(status)
        ref.check_attention(got, lse, want)


@pytest.mark.parametrize("new", [[2, 5], [150, 90]], ids=["few", "many"])
def test_places_past_32_bits(wv, new):
    """Pages more than 2^31 elements apart: attention, forks and compaction reach them all."""
    lens, size, D, hk = [200, 90], 64, 64, 1
    far = 2 ** 31 + 64                                        # elements from page to page
    base = torch.zeros(6 * far + hk * size * D, dtype=torch.bfloat16, device="cuda")
    kc, vc = (base[i * hk * size * D:].as_strided((6, hk, size, D), (far, size * D, D, 1)) for i in (0, 1))
    pages = _i32([[5, 0, 3, 1] + [-1] * 700, [4, 2, 0, 0] + [-1] * 700])   # room for more: many rows go by their own kernel
    lengths = _i32(lens)
    fill = [(_randn(6, hk, size, D, dtype=torch.bfloat16, seed=i)) for i in (1, 2)]
    kc.copy_(fill[0]), vc.copy_(fill[1])
    cu = _i32([0, new[0], sum(new)])
    q = _randn(sum(new), 2, D, dtype=torch.bfloat16, seed=3)
    for kind in "window", "tree":
        call, sees = _calls(wv, kind, kc, vc, pages, lengths, cu, lens, [min(a, b) for a, b in zip(new, lens)])
        ref.check_attention(call(q), None, place.attention(q, *fill, pages, lengths, cu, sees))
    tables = _i32([[5, 0, 3, 1], [-1] * 4]), _i32([120, 0])
    want = place.fork(*fill, *tables, [0], [1], _i32([[2, 4]]), False)
    wv.kv_fork(kc, vc, *tables, _i32([0]), _i32([1]), _i32([[2, 4]]), False)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and torch.equal(tables[0], want[2])
    keep = list(range(10, 200, 3))
    want = place.compact(want[0], want[1], pages, [5], [keep])
    assert wv.kv_compact(kc, vc, pages[:1], _i32([5]), _i32(keep), _i32([0, len(keep)])).tolist() == want[2]
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_window_and_ranges_agree(wv):
    """A window without first keys is a range: the same bits from the kernel for few rows, and no other keys from the one
    for many."""
    for lens, new in ([700, 300], [1, 1]), ([700, 300], [4, 9]), ([1700, 900], [300, 200]):
        q, kc, vc, pages, lengths, cu = _case(lens, new, 2, 2, 128, 16, torch.bfloat16, room=40_000)
        at = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).int()
        ranges = torch.stack([(at - 99).clamp(min=0), at + 1], 1).cuda()
        a, la = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges, return_lse=True)
        b, lb = wv.kv_window_attention(q, kc, vc, pages, lengths, 100, cu_tokens=cu, return_lse=True)
        want = ref.attention(q, kc, vc, pages, lengths, cu, ranges)
        ref.check_attention(a, la, want)
        ref.check_attention(b, lb, want)


@pytest.mark.parametrize("kind", ["window", "tree"])
@pytest.mark.parametrize("drafts", [3, 80], ids=["few", "many"])
def test_steps_in_graphs(wv, kind, drafts):
    """Two graphs of a step (append, attention), replayed on two streams with other lengths, trees and inputs in place."""
    hq, hk, D, size, B = 8, 2, 128, 16, 3
    pages, lengths, n_pages = ref.tables([600] * B, size)
    cu = _i32([i * drafts for i in range(B + 1)])
    T = B * drafts
    state = [dict(x=_randn(T, hq + 2 * hk, D, dtype=torch.bfloat16, seed=3 + i), kc=_randn(n_pages, hk, size, D, dtype=torch.bfloat16, seed=i),
                  vc=_randn(n_pages, hk, size, D, dtype=torch.bfloat16, seed=9 + i), parents=_i32(_tree(drafts, "random", i) * B),
                  lengths=_i32([200, 100, 300])) for i in range(2)]

    def step(s):
        x = s["x"]
        wv.kv_append(x[:, hq:hq + hk], x[:, hq + hk:], s["kc"], s["vc"], pages, s["lengths"], cu)
        if kind == "window":
            return wv.kv_window_attention(x[:, :hq], s["kc"], s["vc"], pages, s["lengths"], 70, 9, cu_tokens=cu)
        return wv.kv_tree_attention(x[:, :hq], s["kc"], s["vc"], pages, s["lengths"], s["parents"], cu)

    side = torch.cuda.Stream()
    graphs, outs = [], []
    for s in state:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(s))
        graphs.append(graph)
    for lens in [80, 600, 81], [599, 90, 333]:
        trees = [_tree(drafts, k, 5) for k in ("random", "comb", "star")]
        for i, s in enumerate(state):
            s["lengths"].copy_(torch.tensor(lens))
            s["parents"].copy_(torch.tensor(sum(trees, [])))
            s["x"].copy_(_randn(T, hq + 2 * hk, D, dtype=torch.bfloat16, seed=sum(lens) + i))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, o in zip(state, outs):
            got = o.clone()
            assert torch.equal(got, step(s))
            sees = [place.window_sees(n, drafts, 70, 9, 1) if kind == "window" else place.tree_sees(n, t)
                    for n, t in zip(lens, trees)]
            ref.check_attention(got, None, place.attention(s["x"][:, :hq], s["kc"], s["vc"], pages, s["lengths"], cu, sees))


# --------------------------------------------------------------------- fork
# lens of the sources (and of sequences that are none), sources, targets (rows of the table behind them), kv heads, D, size
FORK = [
    ([1], [0], 1, 8, 16), ([16], [0], 1, 64, 16), ([17, 33], [0, 1], 2, 128, 16), ([100, 0, 64, 65], [0, 0, 1, 2, 3, 3, 0], 3, 80, 24),
    ([880 * 3 + 5], [0, 0, 0], 4, 128, 880), ([7, 9], [1] * 40, 1, 256, 1), ([300, 20, 500], [2, 2, 0, 1, 1], 2, 96, 390),
    ([129], [0] * 5, 12, 72, 64), ([50, 60], [0, 1] * 20, 1, 16, 7), ([20_000, 3], [0, 1, 0], 2, 128, 64),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("share", [True, False], ids=["share", "copy"])
@pytest.mark.parametrize("case", FORK, ids=lambda c: "n{}f{}h{}d{}p{}".format(max(c[0]), len(c[1]), *c[2:]))
def test_fork(wv, case, share, dtype):
    lens, sources, hk, D, size = case
    N, S = len(sources), len(lens)
    own, _, used = ref.tables(lens, size)
    need = [max(1, -(-lens[s] // size)) for s in sources]
    n_pages = used + (N if share else sum(need)) + 2
    spare = (torch.randperm(n_pages - used, generator=torch.Generator().manual_seed(1)) + used).int()
    fresh = torch.full((N, 1 if share else max(need)), -3, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        m = 1 if share else m
        fresh[i, :m] = spare[at:at + m]
        at += m
    pages = torch.full((S + N + 1, own.shape[1] + 1), -9, dtype=torch.int32, device="cuda")
    pages[:S, :own.shape[1]] = own
    lengths = _i32(lens + [5] * (N + 1))
    targets = (torch.randperm(N, generator=torch.Generator().manual_seed(2)) + S).tolist()
    kc, vc = (_randn(n_pages, hk, size, D, dtype=dtype, seed=i) for i in (1, 2))
    want = place.fork(kc, vc, pages, lengths, sources, targets, fresh, share)
    status = _status()
    args = kc, vc, pages, lengths, _i32(sources), _i32(targets), fresh.cuda(), share
    versions = [t._version for t in args[:4]]
    assert wv.kv_fork(*args, status=status) is None
    wv.kv_status(status)
    for got, w in zip(args, want):
        assert torch.equal(got, w)
    assert all(t._version > v for t, v in zip(args[:4], versions))
    wv.kv_fork(*args, status=status)                         # the same forks again change nothing
    wv.kv_status(status)
    for got, w in zip(args, want):
        assert torch.equal(got, w)


def test_fork_strides(wv):
    """Caches laid out [pages, rows, heads, channels], tables that are columns of wider ones."""
    lens, size = [70, 33], 16
    pages, lengths, used = ref.tables(lens + [0, 0], size)
    wide = torch.zeros(4, 9, dtype=torch.int32, device="cuda")
    wide[:, :pages.shape[1]] = pages
    table = wide[:, :6]
    fresh = torch.arange(used, used + 12, dtype=torch.int32, device="cuda").view(2, 6)
    kc, vc = (_randn(used + 12, size, 2, 64, dtype=torch.bfloat16, seed=i).transpose(1, 2) for i in (1, 2))
    for share in True, False:
        want = place.fork(kc, vc, table, lengths, [1, 0], [2, 3], fresh, share)
        wv.kv_fork(kc, vc, table, lengths, _i32([1, 0]), _i32([2, 3]), fresh[:, :5] if share else fresh, share)
        for got, w in zip((kc, vc, table, lengths), want):
            assert torch.equal(got, w)


def test_forks_that_cannot_be(wv):
    """Left out, told, and the others are done: nothing is written for them."""
    size = 16
    pages, lengths, used = ref.tables([40, 17, 64, 1, 2, 3], size)
    fresh = torch.arange(used, used + 3, dtype=torch.int32, device="cuda")[:, None]
    kc, vc = (_randn(used + 3, 1, size, 8, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    status = _status()
    for sources, targets, done in (([0, 6, 1], [3, 4, 5], [0, 2]), ([0, -1, 1], [3, 4, 5], [0, 2]), ([0, 1, 2], [3, 6, -2], [0]),
                                   ([0, 3, 1], [3, 4, 5], [1, 2]), ([0, 1, 2], [3, 3, 4], [0, 2]), ([0, 1, 2], [0, 3, 4], [1, 2])):
        keep = kc.clone(), vc.clone(), pages.clone(), lengths.clone()
        state = [t.clone() for t in keep]
        wv.kv_fork(*state, _i32(sources), _i32(targets), fresh, status=status)
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        want = place.fork(*keep, [sources[i] for i in done], [targets[i] for i in done], fresh[done], True)
        for got, w in zip(state, want):
            assert torch.equal(got, w)
    for n in -1, pages.shape[1] * size + 1:                  # lengths that are none
        state = [t.clone() for t in (kc, vc, pages, lengths)]
        state[3][0] = n
        want = place.fork(*state, [1], [4], fresh[1:2], True)
        wv.kv_fork(*state, _i32([0, 1]), _i32([3, 4]), fresh[:2], status=status)
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        for got, w in zip(state, want):
            assert torch.equal(got, w)
    # too few fresh pages
    state = [t.clone() for t in (kc, vc, pages, lengths)]
    wv.kv_fork(*state, _i32([0, 3]), _i32([4, 5]), fresh[:2], False, status)
    with pytest.raises(wv.WanError, match="length or token range"):
        wv.kv_status(status)
    want = place.fork(kc, vc, pages, lengths, [3], [5], fresh[1:2], False)
    for got, w in zip(state, want):
        assert torch.equal(got, w)
    # pages outside the cache: what they would hold is not copied
    for bad in -1, kc.shape[0]:
        state = [t.clone() for t in (kc, vc, pages, lengths)]
        wv.kv_fork(*state, _i32([0, 1]), _i32([4, 5]), _i32([[bad], [used]]), status=status)
        with pytest.raises(wv.WanError, match="outside the cache"):
            wv.kv_status(status)
        want = place.fork(kc, vc, pages, lengths, [1], [5], _i32([[used]]), True)
        assert torch.equal(state[0], want[0]) and torch.equal(state[1], want[1])
        assert state[2][4, :3].tolist() == pages[0, :2].tolist() + [bad] and state[3].tolist() == [40, 17, 64, 1, 40, 17]
    wv.kv_fork(kc, vc, pages, lengths, _i32([]), _i32([]), fresh[:0])       # none


# ------------------------------------------------------------------ compact
def _keeps(kind, lens, seed=0):
    g = torch.Generator().manual_seed(seed)
    first, keeps = [], []
    for n in lens:
        if kind == "path":
            f = max(0, n - 30)
            k = [f + int(i) for i in (torch.rand(n - f, generator=g) < 0.3).nonzero()[:, 0]]
        elif kind == "last":
            f = min(4, n)
            k = list(range(max(f, n - max(0, (n - f) * 2 // 3)), n))
        elif kind == "rolled":                               # no key's old place is a new one
            f = min(4, n)
            k = list(range(n - (n - f) // 2, n))
        elif kind == "all":
            f, k = n // 2, list(range(n // 2, n))
        else:
            f = min(n, 3)
            k = [f + int(i) for i in (torch.rand(n - f, generator=g) < 0.6).nonzero()[:, 0]]
        first.append(f)
        keeps.append(k)
    return first, keeps


COMPACT = [
    ([5], 1, 8, 16), ([40, 0, 17, 1], 2, 128, 16), ([900, 333], 3, 80, 24), ([5000], 2, 128, 64), ([2000, 30], 1, 256, 390),
    ([700] * 9, 1, 72, 7), ([130], 12, 64, 1), ([2640], 4, 96, 880), ([60] * 200, 1, 64, 16), ([4000], 1, 136, 128),
    ([300] * 12, 4, 128, 16), ([300, 500] * 3, 4, 128, 32),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("kind", ["path", "last", "rolled", "all", "choice"])
@pytest.mark.parametrize("case", COMPACT, ids=lambda c: "b{}n{}h{}d{}p{}".format(len(c[0]), max(c[0]), *c[1:]))
def test_compact(wv, case, kind, dtype):
    lens, hk, D, size = case
    pages, _, n_pages = ref.tables(lens, size)
    kc, vc = (_randn(n_pages, hk, size, D, dtype=dtype, seed=i) for i in (1, 2))
    first, keeps = _keeps(kind, lens)
    cu = [sum(len(k) for k in keeps[:b]) for b in range(len(keeps) + 1)]
    wk, wv_, wn = place.compact(kc, vc, pages, first, keeps)
    status = _status()
    versions = kc._version, vc._version
    got = wv.kv_compact(kc, vc, pages, _i32(first), _i32(sum(keeps, [])), _i32(cu), status=status)
    wv.kv_status(status)
    assert torch.equal(kc, wk) and torch.equal(vc, wv_) and got.tolist() == wn and got.dtype == torch.int32
    assert kc._version > versions[0] and vc._version > versions[1]


def test_compact_strides(wv):
    lens, size = [70, 133, 5], 16
    pages, _, n = ref.tables(lens, size)
    wide = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :pages.shape[1]] = pages
    kc = _randn(n, size, 2, 64, dtype=torch.bfloat16, seed=1).transpose(1, 2)
    vc = _randn(n, 2, size, 64, dtype=torch.bfloat16, seed=2)
    first, keeps = _keeps("choice", lens)
    cu = [sum(len(k) for k in keeps[:b]) for b in range(4)]
    want = place.compact(kc, vc, pages, first, keeps)
    lengths = torch.full((3,), 99, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert wv.kv_compact(kc, vc, wide[:, :12], _i32(first), _i32(sum(keeps, [])), _i32(cu), lengths, stream=side) is lengths
    side.synchronize()
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and lengths.tolist() == want[2]
    assert lengths._version > 0


def test_compact_leaves_out_what_cannot_be(wv):
    size = 16
    pages, _, n = ref.tables([60, 60, 60], size)
    kc, vc = (_randn(n, 1, size, 8, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    status = _status()
    cu = [0, 2, 5, 7]
    keep = [10, 20, 5, 6, 9, 1, 2]
    # one that moves back, past the table, below any place, twice, out of order: it alone is left out
    for at, value in (0, 3), (1, 64), (1, -1), (4, 2 ** 31 - 1), (5, -2 ** 31), (1, 10), (4, 6), (6, 1):
        bad = list(keep)
        bad[at] = value
        k, v = kc.clone(), vc.clone()
        got = wv.kv_compact(k, v, pages, _i32([4, 4, 0]), _i32(bad), _i32(cu), status=status)
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        same = list(keep)                                    # a key that moves to its own place stands for one left out
        b = max(i for i in range(3) if cu[i] <= at)
        same[at] = [4, 4, 0][b] + at - cu[b]
        want = place.compact(kc, vc, pages, [4, 4, 0], [same[0:2], same[2:5], same[5:7]])
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and got.tolist() == [6, 7, 2]
    for first, ranges, lens in (([-1, 4, 0], cu, [0, 7, 2]), ([4, 65, 0], cu, [6, 0, 2]), ([4, 62, 0], cu, [6, 62, 2]),
                                ([4, 4, 0], [0, 2, 1, 7], [6, 4, 0]), ([4, 4, 0], [0, 2, 5, 8], [6, 7, 0])):
        k, v = kc.clone(), vc.clone()
        got = wv.kv_compact(k, v, pages, _i32(first), _i32(keep), _i32(ranges), status=status)
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        keeps = [keep[0:2], keep[2:5], keep[5:7]]
        for b in range(3):
            if lens[b] != first[b] + (cu[b + 1] - cu[b]):
                keeps[b] = []
        if ranges == [0, 2, 1, 7]:
            keeps[2], lens = keep[1:7], [6, 4, 6]            # rows behind a range that is none may be anybody's
            continue
        want = place.compact(kc, vc, pages, [max(0, f) for f in first], keeps)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and got.tolist() == lens
    # pages outside the cache
    for slot in 0, 1:                                        # of the place moved to, and of the key moved
        table = pages.clone()
        table[0, slot] = n
        k, v = kc.clone(), vc.clone()
        wv.kv_compact(k, v, table, _i32([4, 4, 0]), _i32([20, 21] + keep[2:]), _i32(cu), status=status)
        with pytest.raises(wv.WanError, match="outside the cache"):
            wv.kv_status(status)
        want = place.compact(kc, vc, pages, [4, 4, 0], [[], keep[2:5], keep[5:7]])
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert wv.kv_compact(kc, vc, pages, _i32([1, 2, 3]), _i32([]), _i32([0, 0, 0, 0])).tolist() == [1, 2, 3]


# ------------------------------------------------------- a run of them together
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_drafting_gives_what_one_token_at_a_time_gives(wv, dtype):
    """A past is forked; each future drafts a tree, attends to it, keeps a path, drops what is behind its window, and
    drafts on.  Against plain attention of the accepted tokens alone."""
    hq, hk, D, size, window, sinks = 4, 2, 64, 16, 90, 6
    pages = torch.full((3, 12), -1, dtype=torch.int32, device="cuda")
    pages[0] = torch.arange(12)
    kc, vc = (torch.full((40, hk, size, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    lengths = _i32([0, 0, 0])
    status = _status()
    past = 70
    x = _randn(past, hq + 2 * hk, D, dtype=dtype, seed=1)
    lengths[0] = past
    wv.kv_append(x[:, hq:hq + hk], x[:, hq + hk:], kc, vc, pages[:1], lengths[:1], _i32([0, past]), status=status)
    wv.kv_fork(kc, vc, pages, lengths, _i32([0, 0]), _i32([1, 2]), _i32([[20], [30]]), status=status)
    pages[1, 5:], pages[2, 5:] = torch.arange(21, 28), torch.arange(31, 38)
    table = pages[1:]
    seqs = [[(x[i, hq:hq + hk], x[i, hq + hk:]) for i in range(past)] for _ in range(2)]    # keys and values that are kept
    for turn in range(5):
        drafts = [7, 12]
        trees = [_tree(m, "random", 10 * turn + i) for i, m in enumerate(drafts)]
        y = _randn(sum(drafts), hq + 2 * hk, D, dtype=dtype, seed=50 + turn)
        cu = _i32([0, 7, 19])
        now = _i32([len(s) + m for s, m in zip(seqs, drafts)])
        wv.kv_append(y[:, hq:hq + hk], y[:, hq + hk:], kc, vc, table, now, cu, status=status)
        got = wv.kv_tree_attention(y[:, :hq], kc, vc, table, now, _i32(sum(trees, [])), cu, status=status)
        keeps = []
        for b in range(2):
            base, row0 = len(seqs[b]), (0, 7)[b]
            path, node = [], drafts[b] - 1
            while node >= 0:
                path.insert(0, node)
                node = trees[b][node]
            for i, node in enumerate(path):                  # what each accepted draft got, from the kept tokens alone
                kv = seqs[b] + [(y[row0 + j, hq:hq + hk], y[row0 + j, hq + hk:]) for j in path[:i + 1]]
                k, v = (torch.stack([t[c] for t in kv], 1)[None] for c in (0, 1))
                want = ref.attention(y[row0 + node:row0 + node + 1, :hq], k, v, _i32([[0]]), _i32([len(kv)]))
                ref.assert_rounded(got[row0 + node:row0 + node + 1], want[0], want[1], (turn, b, i))
            keeps.append([base + j for j in path])
            seqs[b] += [(y[row0 + j, hq:hq + hk], y[row0 + j, hq + hk:]) for j in path]
        ck = _i32([0, len(keeps[0]), len(keeps[0]) + len(keeps[1])])
        base = _i32([len(s) - len(k) for s, k in zip(seqs, keeps)])
        lens = wv.kv_compact(kc, vc, table, base, _i32(sum(keeps, [])), ck, status=status)
        assert lens.tolist() == [len(s) for s in seqs]
        # one token more, over the first keys and the window, then the cache rolls on
        z = _randn(2, hq + 2 * hk, D, dtype=dtype, seed=80 + turn)
        lens = lens + 1
        wv.kv_append(z[:, hq:hq + hk], z[:, hq + hk:], kc, vc, table, lens, status=status)
        got = wv.kv_window_attention(z[:, :hq], kc, vc, table, lens, window, sinks, status=status)
        for b in range(2):
            seqs[b].append((z[b, hq:hq + hk], z[b, hq + hk:]))
            n = len(seqs[b])
            seqs[b] = [s for i, s in enumerate(seqs[b]) if i < sinks or i >= n - window]
            k, v = (torch.stack([t[c] for t in seqs[b]], 1)[None] for c in (0, 1))
            want = ref.attention(z[b:b + 1, :hq], k, v, _i32([[0]]), _i32([len(seqs[b])]))
            ref.assert_rounded(got[b:b + 1], want[0], want[1], (turn, b))
        kept = [range(max(sinks, n - window), n) for n in lens.tolist()]
        keep = [i for k in kept for i in k]
        rolled = wv.kv_compact(kc, vc, table, _i32([sinks, sinks]), _i32(keep), _i32([0, len(kept[0]), len(keep)]), status=status)
        assert rolled.tolist() == [len(s) for s in seqs]
    wv.kv_status(status)


class _Strange(torch.Tensor):
    """A subclass: such tensors are marshalled in Python, plain ones in C++."""


def test_both_ways_in_give_the_same(wv):
    lens, new = [40, 64], [3, 2]
    q, kc, vc, pages, lengths, cu = _case(lens, new, 2, 4, 128, 16, torch.bfloat16)
    strange = lambda t: t.as_subclass(_Strange)  # noqa: E731
    parents = _i32([-1, 0, 0, -1, 0])
    for call in (lambda x, **kw: wv.kv_window_attention(x, kc, vc, pages, lengths, 20, 3, 2, cu, **kw),
                 lambda x, **kw: wv.kv_tree_attention(x, kc, vc, pages, lengths, parents, cu, **kw)):
        for kw in {}, dict(scale=0.5), dict(return_lse=True), dict(status=_status()):
            a, b = call(q, **kw), call(strange(q), **kw)
            for s, t in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
                assert torch.equal(s, t.as_subclass(torch.Tensor))
    fork = _i32([0]), _i32([1]), _i32([[4]])
    one, two = ([t.clone() for t in (kc, vc, pages, lengths)] for _ in range(2))
    wv.kv_fork(*one, *fork)
    wv.kv_fork(strange(two[0]), *two[1:], *fork)
    keep = _i32([3, 1]), _i32([5, 9, 30]), _i32([0, 2, 3])
    a = wv.kv_compact(*one[:3], *keep)
    b = wv.kv_compact(strange(two[0]), *two[1:3], *keep)
    assert a.tolist() == b.tolist() == [5, 2]
    assert all(torch.equal(s, t.as_subclass(torch.Tensor)) for s, t in zip(one, two))

"""A stream that runs on: forks, trees, compaction and windows in turn, with windows that are passed."""

import math

import pytest
import torch

from tests import token_reference as ref
from tests.gpu_util import lib_ready
from tests.test_gpu_places import HALVES, _i32, _randn, _status, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wv():
    return lib_ready()


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("share", [True, False], ids=["share", "copy"])
def test_futures_run_on_past_their_windows(wv, share, dtype):
    """A past is forked; each future drafts a tree, keeps a path of it, and goes on by a token that sees first keys and a
    window.  Copied whole, it then drops what is behind the window (keys move inside all its pages); with common pages it
    keeps its keys, and only drafts are compacted, behind them.  Against plain attention of the tokens that are seen, and
    the past is as it was."""
    hq, hk, D, size, window, sinks, past = 4, 2, 64, 16, 40, 6, 70
    pages = torch.full((3, 14), -1, dtype=torch.int32, device="cuda")
    pages[0, :5] = torch.arange(5)
    kc, vc = (torch.full((60, hk, size, D), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    lengths, status = _i32([past, 0, 0]), _status()
    x = _randn(past, hq + 2 * hk, D, dtype=dtype, seed=1)
    wv.kv_append(x[:, hq:hq + hk], x[:, hq + hk:], kc, vc, pages[:1], lengths[:1], _i32([0, past]), status=status)
    fresh = torch.arange(10, 20, dtype=torch.int32, device="cuda").view(2, 5)
    wv.kv_fork(kc, vc, pages, lengths, _i32([0, 0]), _i32([1, 2]), fresh[:, :1].contiguous() if share else fresh, share, status)
    pages[1, 5:], pages[2, 5:] = torch.arange(20, 29), torch.arange(40, 49)
    table = pages[1:]
    held = [ref.keys_of(c, pages[0], past, h) for c in (kc, vc) for h in range(hk)]
    token = lambda t, i: (t[i, hq:hq + hk], t[i, hq + hk:])  # noqa: E731
    seqs = [[token(x, i) for i in range(past)] for _ in range(2)]

    def plain(q, kv):
        k, v = (torch.stack([t[c] for t in kv], 1)[None] for c in (0, 1))
        return ref.attention(q, k, v, _i32([[0]]), _i32([len(kv)]))

    if not share:                                            # the past itself is behind the window already
        keep = list(range(past - window, past)) * 2
        wv.kv_compact(kc, vc, table, _i32([sinks] * 2), _i32(keep), _i32([0, window, 2 * window]), status=status)
        seqs = [s[:sinks] + s[past - window:] for s in seqs]
    for turn in range(4):
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
            for i, node in enumerate(path):
                want = plain(y[row0 + node:row0 + node + 1, :hq], seqs[b] + [token(y, row0 + j) for j in path[:i + 1]])
                ref.assert_rounded(got[row0 + node:row0 + node + 1], want[0], want[1], (turn, b, i))
            keeps.append([base + j for j in path])
            seqs[b] += [token(y, row0 + j) for j in path]
        base = _i32([len(s) - len(k) for s, k in zip(seqs, keeps)])
        lens = wv.kv_compact(kc, vc, table, base, _i32(sum(keeps, [])), _i32([0, len(keeps[0]), sum(map(len, keeps))]), status=status)
        assert lens.tolist() == [len(s) for s in seqs]
        z = _randn(2, hq + 2 * hk, D, dtype=dtype, seed=80 + turn)
        lens = lens + 1
        wv.kv_append(z[:, hq:hq + hk], z[:, hq + hk:], kc, vc, table, lens, status=status)
        got = wv.kv_window_attention(z[:, :hq], kc, vc, table, lens, window, sinks, status=status)
        keep, cu_keep = [], [0]
        for b in range(2):
            seqs[b].append(token(z, b))
            n = len(seqs[b])
            assert n > sinks + window                        # the window is passed: some keys are hidden
            seen = [*range(sinks), *range(n - window, n)]
            want = plain(z[b:b + 1, :hq], [seqs[b][i] for i in seen])
            ref.assert_rounded(got[b:b + 1], want[0], want[1], (turn, b))
            if not share:
                seqs[b] = [seqs[b][i] for i in seen]
                keep += seen[sinks:]
                cu_keep.append(len(keep))
        if not share:
            rolled = wv.kv_compact(kc, vc, table, _i32([sinks] * 2), _i32(keep), _i32(cu_keep), status=status)
            assert rolled.tolist() == [sinks + window] * 2
    wv.kv_status(status)
    for got, was in zip([ref.keys_of(c, pages[0], past, h) for c in (kc, vc) for h in range(hk)], held):
        assert torch.equal(got, was)


def test_compaction_of_ranges_that_overlap(wv):
    """Where one sequence's range is none, it moves nothing; the other two move theirs."""
    size = 16
    pages, _, n = ref.tables([60, 60, 60], size)
    kc, vc = (_randn(n, 1, size, 8, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    keep = [10, 20, 21, 26, 29, 31, 32]
    was = kc.clone(), vc.clone()
    status = _status()
    got = wv.kv_compact(kc, vc, pages, _i32([4, 4, 0]), _i32(keep), _i32([0, 2, 1, 7]), status=status)
    with pytest.raises(wv.WanError, match="length or token range"):
        wv.kv_status(status)
    assert got.tolist()[:2] == [6, 4]
    for c, old in zip((kc, vc), was):
        for b, f, k in (0, 4, keep[:2]), (1, 4, []):
            now, before = ref.keys_of(c, pages[b], 60, 0), ref.keys_of(old, pages[b], 60, 0)
            before[f:f + len(k)] = before[k]
            assert torch.equal(now, before)


@pytest.mark.parametrize("new", [[1, 1, 1], [5, 1, 2]], ids=["step", "few"])
def test_a_window_of_everything_is_a_call_without_ranges(wv, new):
    """The operators agree to the bit where one warp takes all of a row tile; where the line is cut otherwise, sums come in
    another order."""
    lens, size = [16, 9, 12], 16
    pages, lengths, n = ref.tables(lens, size)
    kc, vc = (_randn(n, 2, size, 128, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    cu = _i32([0, new[0], new[0] + new[1], sum(new)])
    q = _randn(sum(new), 4, 128, dtype=torch.bfloat16, seed=3)
    at = torch.cat([torch.arange(a - m, a) for a, m in zip(lens, new)])
    ranges = torch.stack([torch.zeros_like(at), at + 1], 1).int().cuda()
    a, la = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges, return_lse=True)
    b, lb = wv.kv_window_attention(q, kc, vc, pages, lengths, 1000, cu_tokens=cu, return_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)

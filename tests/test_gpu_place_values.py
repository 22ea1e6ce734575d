"""Infinities and NaN among the values of attention of many rows: they reach the
rows that see them, in pages of any length, and cost next to nothing where no
row does."""

import math

import pytest
import torch

from tests import place_reference as place
from tests import token_reference as ref
from tests.gpu_util import lib_ready
from tests.test_gpu_places import HALVES, _case, _i32, _randn, _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wv():
    return lib_ready()


def _causal(lens, new):
    at = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)])
    return torch.stack([torch.zeros_like(at), at + 1], 1).int().cuda()


def _call(wv, kind, q, kc, vc, pages, lengths, cu, lens, new, window=300, sinks=140):
    """A call of the operator, and the plain form's answer to the tensors as they are then."""
    if kind == "ranges":
        r = _causal(lens, new)
        return (lambda **kw: wv.kv_attention(q, kc, vc, pages, lengths, cu, r, **kw),
                lambda: ref.attention(q, kc, vc, pages, lengths, cu, r))
    if kind == "window":
        sees = [place.window_sees(n, m, window, sinks, 1) for n, m in zip(lens, new)]
        return (lambda **kw: wv.kv_window_attention(q, kc, vc, pages, lengths, window, sinks, 1, cu, **kw),
                lambda: place.attention(q, kc, vc, pages, lengths, cu, sees))
    trees = [_tree(m, "random", i) for i, m in enumerate(new)]
    sees = [place.tree_sees(n, t) for n, t in zip(lens, trees)]
    return (lambda **kw: wv.kv_tree_attention(q, kc, vc, pages, lengths, _i32(sum(trees, [])), cu, **kw),
            lambda: place.attention(q, kc, vc, pages, lengths, cu, sees))


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("kind", ["window", "tree", "ranges"])
@pytest.mark.parametrize("D", [64, 72, 128, 256])
@pytest.mark.parametrize("size", [16, 24, 64, 128, 256, 390])
@pytest.mark.parametrize("heads", [(2, 1), (1, 3)], ids=["one", "group"])
def test_odd_values_of_pages_of_any_length(wv, heads, size, D, kind, dtype):
    """Of first keys, of keys on either edge of a window and of drafts; NaN where no row looks, behind the end too."""
    lens, new, (hk, g) = [1500, 700], [200, 33], heads
    q, kc, vc, pages, lengths, cu = _case(lens, new, hk, g, D, size, dtype, room=40_000)
    call, want = _call(wv, kind, q, kc, vc, pages, lengths, cu, lens, new)

    def spot(b, i, c, value):
        vc[int(pages[b, i // size]), (b + i) % hk, i % size, c] = value

    # only a window leaves keys that no row sees: its own begin at place 1001 (b 0) and 368 (b 1)
    spots = [(0, 139, 0, math.inf), (0, 5, 1, math.nan), (0, 1003, 2, -math.inf), (0, 1080, D - 1, math.inf), (0, 1301, 9, math.nan),
             (0, 1390, 3, -math.inf), (0, 1499, 4, math.inf), (0, 1498, 4, math.inf), (1, 130, 7, math.inf), (1, 375, 8, -math.inf),
             (1, 690, 5, math.nan)]
    if kind == "window":
        spots += [(0, 141, 0, math.nan), (0, 600, 0, math.nan), (0, 1000, 10, math.nan), (1, 367, 0, math.inf)]
    for s in spots:
        spot(*s)
    for b, n in enumerate(lens):
        if n % size:
            vc[int(pages[b, n // size]), :, n % size:] = math.nan
            kc[int(pages[b, n // size]), :, n % size:] = math.nan
    got, lse = call(return_lse=True)
    ref.check_attention(got, lse, want())


@pytest.mark.parametrize("kind", ["window", "tree", "ranges"])
def test_all_values_odd(wv, kind):
    """Every value of the last keys is a NaN or an infinity: rows that see none of them stay as they are."""
    lens, new, size = [900], [180], 64
    q, kc, vc, pages, lengths, cu = _case(lens, new, 1, 2, 128, size, torch.bfloat16, room=40_000)
    call, want = _call(wv, kind, q, kc, vc, pages, lengths, cu, lens, new, window=100, sinks=5)
    for i in range(800, 900):
        vc[int(pages[0, i // size]), 0, i % size] = math.nan if i % 3 else math.inf
    got, lse = call(return_lse=True)
    ref.check_attention(got, lse, want())


def _time(call):
    for _ in range(3):
        call()
    took = []
    for _ in range(7):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(4):
            call()
        b.record()
        b.synchronize()
        took.append(a.elapsed_time(b))
    return sorted(took)[3]


@pytest.mark.parametrize("kind", ["window", "tree", "ranges"])
@pytest.mark.parametrize("size", [64, 256])
def test_what_stands_behind_the_end_costs_little(wv, size, kind):
    """A cache of memory as it came holds NaN behind its sequences; walks for values that no row sees took twenty times
    the call."""
    lens, new = [2000 + 531 * i for i in range(8)], [64 if kind == "tree" else 400] * 8
    q, kc, vc, pages, lengths, cu = _case(lens, new, 4, 2, 128, size, torch.bfloat16)
    call, _ = _call(wv, kind, q, kc, vc, pages, lengths, cu, lens, new, window=700, sinks=20)
    clean, before = _time(call), call()
    for b, n in enumerate(lens):
        if n % size:
            vc[int(pages[b, n // size]), :, n % size:] = math.nan
    assert torch.equal(call(), before)
    assert _time(call) < 3 * clean


def test_odd_values_of_a_deep_tree_cost_little(wv):
    """A chain of 1024 drafts with an infinity in its first and last one: the walks to what a row sees are made once for
    64 keys."""
    lens, new, D = [1524], [1024], 128
    q, kc, vc, pages, lengths, cu = _case(lens, new, 2, 1, D, 64, torch.bfloat16)
    parents = _i32(_tree(1024, "chain"))

    def call():
        return wv.kv_tree_attention(q, kc, vc, pages, lengths, parents, cu)
    clean = _time(call)
    for i in 500, 1523:
        vc[int(pages[0, i // 64]), 0, i % 64, 3] = math.inf
    want = place.attention(q, kc, vc, pages, lengths, cu, [place.tree_sees(1524, _tree(1024, "chain"))])
    ref.check_attention(call(), None, want)
    assert _time(call) < 6 * clean


def test_rows_behind_the_last_sequence_stay(wv):
    """Rows behind the last sequence stay as they are where odd values are given back."""
    lens, new = [500], [150]
    q, kc, vc, pages, lengths, cu = _case(lens, new, 1, 2, 64, 16, torch.float16, room=40_000)
    vc[int(pages[0, 25]), 0, 3, 4] = math.inf
    wide = torch.cat([q, _randn(3, 2, 64, dtype=torch.float16, seed=9)])
    out = torch.full_like(wide, 5.0)
    wv.kv_window_attention(wide, kc, vc, pages, lengths, 70, 9, cu_tokens=cu, out=out)
    assert bool((out[150:] == 5.0).all())
    ref.check_attention(out[:150], None, place.attention(q, kc, vc, pages, lengths, cu, [place.window_sees(500, 150, 70, 9, 1)]))


@pytest.mark.parametrize("new", [1, 64], ids=["few", "many"])
def test_windows_of_more_than_2_31_keys(wv, new):
    """Two frames of 1.5e9 keys hold a sequence of 1.6e9 (two pages, which the table repeats: the first half of the places
    has ones as values, the second zeros); frames that end past 2^31 leave the narrow windows as they are."""
    size, ones, n = 1 << 20, 762, 1_600_000_000
    kc = torch.zeros(2, 1, size, 8, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    vc[0] = 1.0
    pages = torch.ones(1, -(-n // size), dtype=torch.int32, device="cuda")
    pages[0, :ones] = 0
    q, lengths, cu = _randn(new, 1, 8, dtype=torch.bfloat16), _i32([n]), _i32([0, new])
    for window, frame, sinks, lo in ((2, 1_500_000_000, 0, 0), (3, 1_000_000_000, 5, 0), (2 ** 31 - 1, 2 ** 31 - 1, 0, 0),
                                     (1, 1_500_000_000, 0, 1_500_000_000), (1, 1_500_000_000, 1000, 1_500_000_000)):
        out, lse = wv.kv_window_attention(q, kc, vc, pages, lengths, window, sinks, frame, cu, return_lse=True)
        seen = n - lo + (min(sinks, lo) if lo else 0)
        want = torch.full((new, 1, 8), (ones * size if lo == 0 else sinks) / seen, dtype=torch.float64, device="cuda")
        # counts of up to 1.6e9 ones, summed in 32 bits: 2^-23 for each chained sum of a part's blocks and of the parts (a part
        # of 1 / 152 or less has under 2^24 keys, whose count is exact)
        ref.assert_rounded(out, want, want * 152 * 2.0 ** -23)
        assert bool(((lse.double() - math.log(seen)).abs() < 1e-4).all())

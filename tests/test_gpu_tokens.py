"""The token operators on the GPU against plain 64-bit forms: rotary positions
and their gradient, the append to a paged cache, attention over it, and the
steps of a streaming model made of them."""

import ctypes
import math
import time

import pytest
import torch

from tests import token_reference as ref
from tests.gpu_util import lib_ready

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def wv():
    return lib_ready()


def _randn(*shape, dtype=torch.float32, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _positions(T, axes, seed=0, lo=0, hi=50, dtype=torch.int32, batch=None):
    g = torch.Generator().manual_seed(seed)
    shape = (T, axes) if batch is None else (batch, T, axes)
    return torch.randint(lo, hi, shape, generator=g).to(dtype).cuda()


# ------------------------------------------------------------------- rotary
# (shape, sections): video and text forms, channels left over, single tokens,
# odd pair counts (narrow accesses), the widest head
ROTARY = [
    ((1, 1, 128), (22, 21, 21)), ((4, 1, 16, 128), (22, 21, 21)), ((2, 33, 5, 80), (8, 16, 16)), ((77, 3, 64), (32,)),
    ((5, 2, 96), (40,)), ((9, 9, 256), (44, 42, 42)), ((3, 7, 30), (7, 4, 4)), ((2, 1, 2), (1,)), ((31, 40, 12), (3, 1)),
    ((600, 12, 40), (5, 5, 5, 5)),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("interleaved", [True, False], ids=["pairs", "halves"])
@pytest.mark.parametrize("shape,sections", ROTARY, ids=lambda v: "x".join(map(str, v)))
def test_rotary(wv, shape, sections, interleaved, dtype):
    x = _randn(*shape, dtype=dtype, seed=1)
    pos = _positions(shape[-3], len(sections), seed=2)
    for fn, sign in (wv.rotary, 1.0), (wv.rotary_grad, -1.0):
        got = fn(x, pos, sections, interleaved=interleaved)
        want, err = ref.rotary(x, pos, sections, interleaved=interleaved, sign=sign)
        ref.assert_rounded(got, want, err)
        assert torch.equal(got[..., 2 * sum(sections):], x[..., 2 * sum(sections):])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64], ids=str)
def test_rotary_far_and_negative_positions(wv, kind):
    x = _randn(64, 2, 64)
    for lo, hi in (-50, 50), (999_000, 1_000_001), (2 ** 31 - 1000, 2 ** 31 - 1), (-2 ** 31, -2 ** 31 + 1000):
        pos = _positions(64, 2, lo=lo, hi=hi, dtype=kind)
        want, err = ref.rotary(x, pos, (20, 12))
        ref.assert_rounded(wv.rotary(x, pos, (20, 12)), want, err, (lo, hi))


def test_rotary_own_frequencies(wv):
    freq = [0.0, -0.25, 7.5, 1e-9, math.pi, 2 * math.pi, 123.456, 1.0]
    x, pos = _randn(40, 3, 16), _positions(40, 2, hi=900)
    for inter in True, False:
        want, err = ref.rotary(x, pos, (5, 3), freq=freq, interleaved=inter)
        # a frequency is kept to 2^-53 of itself and its turns to 2^-53 of theirs
        err = err + 900 * 124 * 2.0 ** -51 * x.abs().amax().double()
        ref.assert_rounded(wv.rotary(x, pos, wv.Rotation((5, 3), freq=freq, interleaved=inter)), want, err)


@pytest.mark.parametrize("interleaved", [True, False], ids=["pairs", "halves"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_rotary_strides_and_places(wv, dtype, interleaved):
    sections = (8, 4, 4)
    pos = _positions(21, 3, batch=2)
    packed = _randn(2, 21, 3 * 6, 40, dtype=dtype)          # q, k and v of a packed projection
    q = packed[:, :, 3:9]
    want, err = ref.rotary(q, pos, sections, interleaved=interleaved)
    ref.assert_rounded(wv.rotary(q, pos, sections, interleaved=interleaved), want, err, "view")
    heads_first = q.transpose(1, 2).contiguous().transpose(1, 2)
    ref.assert_rounded(wv.rotary(heads_first, pos, sections, interleaved=interleaved), want, err, "heads first")
    for off in 1, 2, 4:                                       # elements off a 16-byte boundary
        flat = torch.empty(q.numel() + off, dtype=dtype, device="cuda")
        moved = flat[off:].view(q.shape)
        moved.copy_(q)
        ref.assert_rounded(wv.rotary(moved, pos, sections, interleaved=interleaved), want, err, off)
        ref.assert_rounded(wv.rotary(q, pos, sections, interleaved=interleaved, out=moved), want, err, off)
    one = _randn(2, 21, 1, 40, dtype=dtype).expand(2, 21, 6, 40)  # a broadcast input
    w1, e1 = ref.rotary(one, pos, sections, interleaved=interleaved)
    ref.assert_rounded(wv.rotary(one, pos, sections, interleaved=interleaved), w1, e1, "broadcast")
    before = packed.clone()
    assert wv.rotary(q, pos, sections, interleaved=interleaved, out=q).data_ptr() == q.data_ptr()
    ref.assert_rounded(q, want, err, "in place")
    assert torch.equal(packed[:, :, :3], before[:, :, :3]) and torch.equal(packed[:, :, 9:], before[:, :, 9:])
    with pytest.raises(wv.WanError, match="broadcast"):
        wv.rotary(q, pos, sections, out=one)


def test_rotary_leaves_odd_values_where_they_are(wv):
    x = _randn(6, 4, 32)
    x[1, 2, 30], x[2, 1, 31], x[3, 0, 4] = math.inf, math.nan, math.inf
    for inter in True, False:
        got = wv.rotary(x, _positions(6, 1, lo=1), (14,), interleaved=inter)
        odd = ~torch.isfinite(got)
        rows = torch.zeros_like(odd)
        rows[1, 2, 30] = rows[2, 1, 31] = rows[3, 0, 4] = True
        rows[3, 0, 5 if inter else 18] = True               # the pair's other channel
        assert torch.equal(odd, rows)


def test_rotary_empty(wv):
    for shape in (0, 4, 32), (2, 0, 4, 32), (0, 5, 4, 32):
        x = torch.empty(shape, device="cuda")
        assert wv.rotary(x, torch.empty(shape[-3], 1, dtype=torch.int32, device="cuda"), (16,)).shape == x.shape


def test_rotary_gradient(wv):
    """The gradient against the formula's (64-bit autograd), against
    differences, and as the backward pass of an autograd function."""
    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, pos):
            ctx.save_for_backward(pos)
            return wv.rotary(x, pos, (6, 5, 5), interleaved=False)

        @staticmethod
        def backward(ctx, dy):
            return wv.rotary_grad(dy, ctx.saved_tensors[0], (6, 5, 5), interleaved=False), None

    pos, w = _positions(13, 3), _randn(13, 3, 36, seed=5)
    base = _randn(13, 1, 36, seed=4)
    x = base.clone().requires_grad_()
    loss = (Turn.apply(x.expand(13, 3, 36), pos) * w).sum()    # one row for three heads: their gradients add up
    loss.backward()
    xd = base.double().requires_grad_()
    (ref.rotary(xd.expand(13, 3, 36), pos, (6, 5, 5), interleaved=False)[0] * w).sum().backward()
    _, err = ref.rotary(w, pos, (6, 5, 5), interleaved=False, sign=-1.0)
    tol = err.sum(1, keepdim=True) + 5 * 2.0 ** -24 * w.double().abs().sum(1, keepdim=True) * math.sqrt(2)
    assert bool(((x.grad.double() - xd.grad).abs() <= tol).all())
    # differences along a direction: the map is linear, so a step of one shows no curvature
    d = _randn(13, 1, 36, seed=6)
    up = (wv.rotary((base + d).expand(13, 3, 36), pos, (6, 5, 5), interleaved=False).double() * w).sum()
    down = (wv.rotary((base - d).expand(13, 3, 36), pos, (6, 5, 5), interleaved=False).double() * w).sum()
    scale = (w.double().abs().sum() * (base.abs() + d.abs()).amax() * 2).item()
    assert abs((up - down).item() / 2 - (x.grad.double() * d).sum().item()) <= 2.0 ** -20 * scale


# ------------------------------------------------------------------- append
def _append_reference(k, v, kc, vc, pages, lens, cu, pos, sections, interleaved, q):
    """Caches and q in 64 bits, their bounds, and the rows that were written."""
    kr, ke = (k.double(), torch.zeros_like(k, dtype=torch.float64)) if sections is None else ref.rotary(
        k, pos, sections, interleaved=interleaved)
    want_k, want_v = kc.double(), vc.double()
    err = torch.zeros_like(want_k)
    size = kc.shape[2]
    written = torch.zeros(kc.shape[0], size, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        new = cu[b + 1] - cu[b]
        at = torch.arange(n - new, n, device="cuda")
        p, r = pages[b][at // size].long(), at % size
        want_k[p, :, r], err[p, :, r] = kr[cu[b]:cu[b + 1]], ke[cu[b]:cu[b + 1]]
        want_v[p, :, r] = v[cu[b]:cu[b + 1]].double()
        written[p, r] = True
    return want_k, err, want_v, written


# lens (with the new tokens), new tokens, page size, kv heads, q heads, head dim, sections
APPEND = [
    ([1], [1], 16, 1, 1, 8, (4,)),
    ([100, 17, 16, 1], [1, 1, 1, 1], 16, 8, 32, 128, (64,)),
    ([880 * 3], [1760], 880, 4, 4, 128, (22, 21, 21)),
    ([70, 33, 1, 5], [70, 0, 1, 3], 24, 2, 0, 96, (40,)),
    ([9, 300], [9, 299], 1, 3, 6, 80, (13, 13, 13)),
    ([65, 64], [2, 64], 64, 1, 16, 256, None),
    ([500, 500], [333, 1], 100, 2, 10, 72, (36,)),
    ([50], [7], 390, 12, 12, 64, (9, 9, 9)),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("interleaved", [True, False], ids=["pairs", "halves"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: "n{}p{}h{}q{}d{}".format(sum(c[1]), *c[2:6]))
def test_append(wv, case, interleaved, dtype):
    lens, new, size, hk, hq, D, sections = case
    pages, lengths, n_pages = ref.tables(lens, size)
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    T = cu[-1] + 2                                             # two rows behind the last sequence
    k, v = _randn(T, hk, D, dtype=dtype, seed=1), _randn(T, hk, D, dtype=dtype, seed=2)
    q = _randn(T, hq, D, dtype=dtype, seed=3) if hq else None
    kc, vc = _randn(n_pages, hk, size, D, dtype=dtype, seed=4), _randn(n_pages, hk, size, D, dtype=dtype, seed=5)
    pos = None if sections is None else _positions(T, len(sections), hi=3000)
    want_k, err, want_v, written = _append_reference(k, v, kc, vc, pages, lens, cu, pos, sections, interleaved, q)
    k0 = kc.clone()
    q_out = None if q is None else torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    step = all(n == 1 for n in new)
    got = wv.kv_append(k, v, kc, vc, pages, lengths, None if step else torch.tensor(cu, dtype=torch.int32).cuda(), pos,
                       sections, interleaved=interleaved, q=q, q_out=q_out, status=status)
    wv.kv_status(status)
    hidden = ~written[:, None, :, None].expand_as(kc)
    assert torch.equal(kc[hidden], k0[hidden])                 # nothing else was touched
    ref.assert_rounded(kc, want_k, err)
    assert torch.equal(vc.double(), want_v)
    if q is not None:
        assert got is q_out
        wq, eq = (q.double(), torch.zeros(1, device="cuda")) if sections is None else ref.rotary(
            q, pos, sections, interleaved=interleaved)
        ref.assert_rounded(got[:cu[-1]], wq[:cu[-1]], eq[:cu[-1]] if sections is not None else eq.double())
        assert bool((got[cu[-1]:] == 7.0).all())
    else:
        assert got is None


def test_append_strides_and_in_place_q(wv):
    """A cache laid out [pages, rows, heads, channels], k, v and q as views of
    one packed projection, and q turned in place."""
    lens, new = [40, 21, 19], [3, 5, 2]
    pages, lengths, n_pages = ref.tables(lens, 16)
    cu = [0, 3, 8, 10]
    packed = _randn(10, 4 + 2 + 2, 64, dtype=torch.bfloat16)
    kc, vc = (_randn(n_pages, 16, 2, 64, dtype=torch.bfloat16, seed=i).transpose(1, 2) for i in (1, 2))
    pos = _positions(10, 3, dtype=torch.int64)
    q, k, v = packed[:, :4], packed[:, 4:6], packed[:, 6:]
    want_k, err, want_v, _ = _append_reference(k, v, kc, vc, pages, lens, cu, pos, (10, 11, 11), True, q)
    wq, eq = ref.rotary(q, pos, (10, 11, 11))
    wide = torch.zeros(3, 9, dtype=torch.int32, device="cuda")     # a table with room for more pages
    wide[:, :pages.shape[1]] = pages
    got = wv.kv_append(k, v, kc, vc, wide[:, :5], lengths, torch.tensor(cu, dtype=torch.int32).cuda(), pos, (10, 11, 11),
                       q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr()
    ref.assert_rounded(kc, want_k, err)
    assert torch.equal(vc.double(), want_v)
    ref.assert_rounded(q, wq, eq)


def test_append_leaves_out_what_is_not_there(wv):
    """Page numbers outside the cache, lengths beyond the table and more new
    tokens than keys: nothing is written for them, the others are, and the
    status word says so."""
    D, size = 64, 16
    kc, vc = (torch.zeros(4, 1, size, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.ones(4, 1, D, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1], [1, 4], [2, -1], [3, 0]], dtype=torch.int32).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    for lens, cu, rows, message in (
            (i32(1, 17, 17, 1), None, [(0, 0), (3, 0)], "outside the cache"),
            (i32(33, 16, 0, 2), None, [(1, 15), (3, 1)], "length or token range"),
            (i32(1, 1, 1, 2 ** 31 - 1), None, [(0, 0), (1, 0), (2, 0)], "length or token range"),
            (i32(1, 1, 1, 1), i32(0, 1, 3, 3, 4), [(0, 0), (1, 0), (3, 0)], "length or token range"),
            (i32(1, 1, 1, 1), i32(0, 1, 2, 3, 9), [(0, 0), (1, 0), (2, 0)], "length or token range")):
        kc.zero_(), vc.zero_()
        q = wv.kv_append(k, k, kc, vc, table, lens, cu, q=k, status=status)
        assert q.shape == k.shape
        with pytest.raises(wv.WanError, match=message):
            wv.kv_status(status)
        wv.kv_status(status)                                    # cleared
        want = torch.zeros_like(kc)
        for p, r in rows:
            want[p, 0, r] = 1
        assert torch.equal(kc, want) and torch.equal(vc, want)


# ---------------------------------------------------------------- attention
def _attention_case(wv, lens, hk, g, D, size, dtype, new=None, ranges=None, seed=0, scale=None, fill=None, spare=3, room=40_000):
    pages, lengths, n_pages = ref.tables(lens, size, seed=seed, spare=spare)
    # tables with room for more keys than any sequence has (calls of many tokens take another way where there is little)
    more = max(0, -(-room // size) - pages.shape[1])
    pages = torch.cat([pages, torch.full((len(lens), more), -1, dtype=torch.int32, device="cuda")], 1)
    new = [1] * len(lens) if new is None else new
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    T = int(cu[-1])
    kc, vc = _randn(n_pages, hk, size, D, dtype=dtype, seed=seed + 1), _randn(n_pages, hk, size, D, dtype=dtype, seed=seed + 2)
    if fill is not None:  # whatever no sequence holds
        held = torch.zeros(n_pages, size, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            at = torch.arange(n, device="cuda")
            held[pages[b][at // size].long(), at % size] = True
        hidden = ~held[:, None, :, None].expand_as(kc)
        kc[hidden] = fill
        vc[hidden] = fill
    q = _randn(T, hk * g, D, dtype=dtype, seed=seed + 3, scale=1.5)
    return q, kc, vc, pages, lengths, cu.cuda()


# lens, kv heads, group, head dim, page size
DECODE = [
    ([1], 1, 1, 64, 16), ([1, 0, 2, 15, 16, 17], 2, 1, 128, 16), ([63, 64, 65, 127, 128, 129], 1, 4, 128, 64),
    ([1000], 16, 1, 128, 16), ([5, 700, 33], 4, 5, 80, 24), ([257, 31], 2, 16, 64, 1), ([90, 91], 1, 17, 96, 7),
    ([300, 1, 299], 3, 8, 256, 100), ([5000, 12], 8, 8, 128, 256), ([2000], 1, 40, 8, 390), ([880 * 3 + 1], 2, 2, 128, 880),
    ([70] * 200, 1, 2, 72, 32),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "b{}n{}h{}g{}d{}p{}".format(len(c[0]), max(c[0]), *c[1:]))
def test_attention_of_one_token(wv, case, dtype):
    lens, hk, g, D, size = case
    q, kc, vc, pages, lengths, _ = _attention_case(wv, lens, hk, g, D, size, dtype, fill=math.nan)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = wv.kv_attention(q, kc, vc, pages, lengths, return_lse=True, status=status)
    wv.kv_status(status)
    ref.check_attention(got, lse, ref.attention(q, kc, vc, pages, lengths))
    assert torch.equal(wv.kv_attention(q, kc, vc, pages, lengths), got)   # and the same bits again


# lens, new tokens, kv heads, group, head dim, page size, mask
CHUNK = [
    ([5], [5], 1, 1, 64, 16, "causal"), ([40, 0, 3], [7, 0, 3], 2, 3, 128, 16, None), ([200, 130], [130, 1], 2, 1, 128, 64, "causal"),
    ([700, 64, 300], [300, 64, 5], 1, 4, 64, 32, "causal"), ([900], [440], 3, 1, 128, 220, "frames"),
    ([513, 1000], [257, 512], 2, 5, 80, 24, "causal"), ([400, 77], [129, 77], 1, 2, 256, 100, "frames"),
    ([350], [350], 2, 2, 96, 7, "documents"), ([300], [128], 1, 8, 128, 128, "window"), ([260, 130], [260, 130], 1, 1, 16, 1, "holes"),
    ([2000], [880], 2, 1, 128, 880, None), ([150], [150], 1, 48, 64, 16, "causal"), ([3000, 20], [2, 20], 4, 2, 128, 256, "frames"),
]


def _ranges(kind, lens, new):
    if kind is None:
        return None
    got = []
    for n, m in zip(lens, new):
        for p in range(n - m, n):
            got.append({"causal": (0, p + 1), "frames": (0, (p // 110 + 1) * 110), "documents": (p // 60 * 60, p + 1),
                        "window": (p - 70, p + 1),
                        "holes": [(0, 0), (5, 5), (9, 2), (n, n + 5), (-3, 1), (n - 1, 10 ** 9), (0, n), (p, p + 1)][p % 8]}[kind])
    return torch.tensor(got, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("case", CHUNK, ids=lambda c: "t{}n{}h{}g{}d{}p{}{}".format(sum(c[1]), max(c[0]), *c[2:6], c[6] or ""))
@pytest.mark.parametrize("room", [0, 40_000], ids=["tight", "roomy"])
def test_attention_of_many_tokens(wv, case, dtype, room):
    lens, new, hk, g, D, size, mask = case
    q, kc, vc, pages, lengths, cu = _attention_case(wv, lens, hk, g, D, size, dtype, new=new, fill=math.nan, room=room)
    ranges = _ranges(mask, lens, new)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # two rows behind the last sequence stay as they are
    wide, out = torch.cat([q, q[:2]]), torch.full((q.shape[0] + 2, *q.shape[1:]), 7.0, dtype=dtype, device="cuda")
    rr = None if ranges is None else torch.cat([ranges, ranges[:2]])
    got, lse = wv.kv_attention(wide, kc, vc, pages, lengths, cu, rr, out=out, return_lse=True, status=status)
    wv.kv_status(status)
    T = q.shape[0]
    assert got is out and bool((out[T:] == 7.0).all())
    ref.check_attention(got[:T], lse[:T], ref.attention(q, kc, vc, pages, lengths, cu, ranges))
    again = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges)
    assert torch.equal(again, got[:T])


# heads of more than 128 channels (one half of a tile's rows), pages in part and in parts, pieces that meet in a tile
WIDE = [
    ([64], [64], 1, 1, 256, 16, "causal"), ([700, 33], [300, 33], 2, 2, 256, 64, "causal"), ([900], [440], 3, 1, 136, 220, "frames"),
    ([513, 1000], [257, 512], 2, 5, 192, 24, "causal"), ([350], [350], 2, 2, 200, 390, "documents"),
    ([300], [128], 1, 8, 256, 128, "window"), ([260, 130], [260, 130], 1, 1, 144, 8, "holes"), ([4000], [200], 1, 1, 256, 256, None),
    ([0, 150], [70, 150], 1, 16, 256, 16, "holes"),
]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("case", WIDE, ids=lambda c: "t{}n{}h{}g{}d{}p{}{}".format(sum(c[1]), max(c[0]), *c[2:6], c[6] or ""))
def test_attention_of_wide_heads(wv, case, dtype):
    test_attention_of_many_tokens(wv, case, dtype, 40_000)


@pytest.mark.parametrize("new", [[1, 1], [3, 2], [150, 200]], ids=str)
@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attention_scales(wv, new, scale):
    q, kc, vc, pages, lengths, cu = _attention_case(wv, [333, 200], 2, 2, 64, 16, torch.bfloat16, new=new)
    got, lse = wv.kv_attention(q, kc, vc, pages, lengths, cu, scale=scale, return_lse=True)
    ref.check_attention(got, lse, ref.attention(q, kc, vc, pages, lengths, cu, scale=scale))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [6, 200], ids=["few", "many"])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_attention_keeps_odd_values_from_rows_that_do_not_see_them(wv, new, dtype, D):
    """Infinities and NaNs in keys and values: each row's own where it sees
    them, none where its range leaves them out, inside one tile of keys."""
    n = 260
    q, kc, vc, pages, lengths, cu = _attention_case(wv, [n], 2, 3, D, 16, dtype, new=[new])
    ranges = _ranges("causal", [n], [new])
    place = lambda i: (int(pages[0, i // 16]), i % 16)  # noqa: E731
    for i, h, c, value in ((n - 2, 0, 3, math.inf), (n - 3, 0, 4, math.nan), (n - 2, 1, D - 1, -math.inf), (n - 4, 1, 0, math.inf),
                           (n - 3, 1, 0, -math.inf)):
        p, r = place(i)
        vc[p, h, r, c] = value
    p, r = place(n - 1)
    kc[p, 0, r, 5] = math.nan                                    # only the last row sees this key
    got, lse = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges, return_lse=True)
    out, err, z, zerr = ref.attention(q, kc, vc, pages, lengths, cu, ranges)
    assert bool(torch.isnan(got[-1, :3]).all()) and bool(torch.isnan(out[-1, :3]).all())
    ref.check_attention(got[:-1], lse[:-1], (out[:-1], err[:-1], z[:-1], zerr[:-1]))
    ref.check_attention(got[-1:, 3:], lse[-1:, 3:], (out[-1:, 3:], err[-1:, 3:], z[-1:, 3:], zerr[-1:, 3:]))


@pytest.mark.parametrize("new", [[1, 1, 1], [2, 9, 1], [140, 70, 300]], ids=["step", "few", "many"])
def test_attention_strides_and_streams(wv, new):
    lens = [400, 256, 300]
    q, kc, vc, pages, lengths, cu = _attention_case(wv, lens, 2, 2, 64, 16, torch.float16, new=new)
    want = ref.attention(q, kc, vc, pages, lengths, cu)
    T = q.shape[0]
    rows_first = lambda c: c.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    ref.check_attention(wv.kv_attention(q, rows_first(kc), vc, pages, lengths, cu), None, want, "rows first")
    packed = torch.zeros(T, 4 + 4, 64, dtype=torch.float16, device="cuda")
    packed[:, 2:6] = q
    out = torch.zeros(T, 9, 64, dtype=torch.float16, device="cuda")
    wv.kv_attention(packed[:, 2:6], kc, vc, pages, lengths, cu, out=out[:, 3:7])
    ref.check_attention(out[:, 3:7], None, want, "packed")
    assert not out[:, :3].any() and not out[:, 7:].any()
    odd = torch.zeros(T * 4 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(T, 4, 64)
    odd.copy_(q)
    wv.kv_attention(odd, kc, vc, pages, lengths, cu, out=odd)      # off a 16-byte boundary, and onto itself
    ref.check_attention(odd, None, want, "odd address")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = wv.kv_attention(q, kc, vc, pages, lengths, cu, stream=s)
    b = wv.kv_attention(q, kc, vc, pages, lengths, cu)            # both at once: a workspace each
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    ref.check_attention(a, None, want, "stream")


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [1, 4, 2, 1], [70, 1, 200, 100]], ids=["step", "few", "many"])
def test_attention_leaves_out_what_is_not_there(wv, new):
    """Bad page numbers hide their keys, a bad length or token range its
    sequence; the status word tells."""
    lens, size = [100, 40, 300, 200], 16
    q, kc, vc, pages, lengths, cu = _attention_case(wv, lens, 1, 2, 64, size, torch.bfloat16, new=new)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = pages.clone()
    bad[0, 2], bad[2, 18] = kc.shape[0], -5
    got = wv.kv_attention(q, kc, vc, bad, lengths, cu, status=status)
    with pytest.raises(wv.WanError, match="outside the cache"):
        wv.kv_status(status)
    # a key that nobody sees is a key that scores -inf
    k2, v2 = kc.clone(), vc.clone()
    fixed = pages.clone()
    spare = torch.full((1, *kc.shape[1:]), 0.0, dtype=kc.dtype, device="cuda")
    k2, v2 = torch.cat([k2, spare]), torch.cat([v2, spare])
    out, err, z, zerr = ref.attention(q, kc, vc, pages, lengths, cu)
    i = 0
    for b, hole in (0, 2), (2, 18):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        keep = torch.tensor([k for k in range(lens[b]) if k // size != hole], device="cuda")
        short = torch.arange(len(keep), device="cuda")
        # the same sequence without the hole, in pages of its own
        n = -(-len(keep) // size)
        kk = torch.zeros(n, 1, size, 64, dtype=kc.dtype, device="cuda")
        vv = torch.zeros_like(kk)
        src = pages[b][keep // size].long()
        kk[short // size, :, short % size] = kc[src, :, keep % size]
        vv[short // size, :, short % size] = vc[src, :, keep % size]
        one = ref.attention(q[rows], kk, vv, torch.arange(n, dtype=torch.int32, device="cuda")[None],
                            torch.tensor([len(keep)]), torch.tensor([0, new[b]]))
        out[rows], err[rows] = one[0], one[1]
        i += 1
    ref.assert_rounded(got, out, err)
    # a length beyond the table: its rows see nothing
    long = lengths.clone()
    long[1] = pages.shape[1] * size + 1
    got, lse = wv.kv_attention(q, kc, vc, pages, long, cu, status=status, return_lse=True)
    with pytest.raises(wv.WanError, match="length or token range"):
        wv.kv_status(status)
    rows = slice(int(cu[1]), int(cu[2]))
    assert not got[rows].any() and bool(torch.isinf(lse[rows]).all())
    keep = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
    keep[rows] = False
    good = ref.attention(q, kc, vc, pages, lengths, cu)
    ref.assert_rounded(got[keep], good[0][keep], good[1][keep])
    if max(new) > 1:  # a token range that is none
        broken = cu.clone()
        broken[2] = broken[1] - 1
        out = torch.full_like(q, 7.0)
        wv.kv_attention(q, kc, vc, pages, lengths, broken, out=out, status=status)
        with pytest.raises(wv.WanError, match="length or token range"):
            wv.kv_status(status)
        ref.assert_rounded(out[:new[0]], good[0][:new[0]], good[1][:new[0]])


def test_attention_far_into_a_cache(wv):
    """Offsets past 2^32 elements of the cache."""
    size, hk, D = 256, 8, 128
    n_pages = (1 << 32) // (size * hk * D) + 5
    kc = torch.empty(n_pages, hk, size, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    used = torch.tensor([n_pages - 1, 0, n_pages - 2, n_pages // 2 + 1], dtype=torch.int32)
    for p in used.tolist():
        kc[p], vc[p] = _randn(hk, size, D, dtype=torch.bfloat16, seed=p), _randn(hk, size, D, dtype=torch.bfloat16, seed=p + 1)
    pages, lengths = used.view(1, 4).cuda(), torch.tensor([1000], dtype=torch.int32).cuda()
    k, v = _randn(3, hk, D, dtype=torch.bfloat16, seed=1), _randn(3, hk, D, dtype=torch.bfloat16, seed=2)
    wv.kv_append(k, v, kc, vc, pages, lengths, torch.tensor([0, 3], dtype=torch.int32).cuda())
    at = torch.arange(997, 1000)
    assert torch.equal(kc[used[3].item(), :, at % size].transpose(0, 1), k) or torch.equal(kc[used[3].item(), :, at % size], k)
    for T in 1, 200:
        q = _randn(T, hk * 2, D, dtype=torch.bfloat16, seed=3)
        cu = torch.tensor([0, T], dtype=torch.int32).cuda()
        got, lse = wv.kv_attention(q, kc, vc, pages, lengths, cu, return_lse=True)
        ref.check_attention(got, lse, ref.attention(q, kc, vc, pages, lengths, cu))


# --------------------------------------------------------- the steps together
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_streaming_steps(wv, dtype):
    """Latent frames, then single tokens, of two clips of different lengths:
    append and attend step by step, frame-causal, against attention over the
    whole clips at once; the whole step replayed from a graph with lengths,
    pages and inputs changed in place gives the same."""
    hq, hk, D, frame, size = 6, 2, 64, 60, 24
    sections = (12, 10, 10)
    frames = [3, 2]
    lens = [f * frame + 4 for f in frames]
    g = torch.Generator(device="cuda").manual_seed(9)
    total = [(torch.randn(n, hq + 2 * hk, D, generator=g, device="cuda")).to(dtype) for n in lens]
    places = [torch.stack([torch.arange(n) // frame, torch.arange(n) % frame // 10, torch.arange(n) % 10], -1).int().cuda()
              for n in lens]
    pages, _, n_pages = ref.tables(lens, size)
    kc = torch.full((n_pages, hk, size, D), math.nan, dtype=dtype, device="cuda")
    vc = torch.full_like(kc, math.nan)
    steps = [[(0, 60), (0, 60)], [(60, 120), (60, 120)], [(120, 180), (120, 121)]]
    steps += [[(180 + i, 181 + i), (121 + i, 122 + i)] for i in range(3)]
    got = [[], []]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in steps:
        x = torch.cat([total[b][s:e] for b, (s, e) in enumerate(step)])
        pos = torch.cat([places[b][s:e] for b, (s, e) in enumerate(step)])
        new = [e - s for s, e in step]
        cu = None if new == [1, 1] else torch.tensor([0, new[0], sum(new)], dtype=torch.int32).cuda()
        lengths = torch.tensor([e for _, e in step], dtype=torch.int32).cuda()
        q = wv.kv_append(x[:, hq:hq + hk], x[:, hq + hk:], kc, vc, pages, lengths, cu, pos, sections, q=x[:, :hq],
                         status=status)
        o = wv.kv_attention(q, kc, vc, pages, lengths, cu, status=status)
        for b in range(2):
            got[b].append(o[:new[0]] if b == 0 else o[new[0]:])
    wv.kv_status(status)
    for b in range(2):
        o = torch.cat(got[b])
        n = o.shape[0]
        seen = torch.empty(n, dtype=torch.int64)
        for step in steps:
            s, e = step[b]
            seen[s:e] = e
        turn = lambda t: wv.rotary(t.contiguous(), places[b][:n], sections)  # noqa: E731
        q, k, v = turn(total[b][:n, :hq]), turn(total[b][:n, hq:hq + hk]), total[b][:n, hq + hk:]
        cache = lambda t: t.transpose(0, 1)[None]  # noqa: E731  one page, a row a key
        ranges = torch.stack([torch.zeros_like(seen), seen], -1).int().cuda()
        want = ref.attention(q, cache(k), cache(v), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([n]),
                             torch.tensor([0, n]), ranges)
        ref.assert_rounded(o, want[0], want[1], b)


def test_steps_in_graphs(wv):
    """Two graphs captured from the same step, replayed with other lengths,
    pages and inputs in place, one after the other and on two streams."""
    hq, hk, D, size, B = 8, 2, 128, 16, 3
    lens0, lens1 = [40, 7, 90], [200, 65, 1]
    pages, lengths, n_pages = ref.tables([300] * B, size)
    lengths.copy_(torch.tensor(lens0))
    kc, vc = _randn(n_pages, hk, size, D, dtype=torch.bfloat16, seed=1), _randn(n_pages, hk, size, D, dtype=torch.bfloat16, seed=2)
    state = [dict(x=_randn(B, hq + 2 * hk, D, dtype=torch.bfloat16, seed=3 + i), pos=_positions(B, 1, seed=i),
                  kc=kc.clone(), vc=vc.clone(), lengths=lengths.clone()) for i in range(2)]

    def step(s):
        q = wv.kv_append(s["x"][:, hq:hq + hk], s["x"][:, hq + hk:], s["kc"], s["vc"], pages, s["lengths"], None, s["pos"],
                         (D // 2,), interleaved=False, q=s["x"][:, :hq])
        return wv.kv_attention(q, s["kc"], s["vc"], pages, s["lengths"])

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
    for lens in lens1, lens0, [1, 2, 3]:
        for i, s in enumerate(state):
            s["lengths"].copy_(torch.tensor(lens))
            s["x"].copy_(_randn(B, hq + 2 * hk, D, dtype=torch.bfloat16, seed=sum(lens) + i))
            s["pos"].copy_(torch.tensor(lens)[:, None] + i)
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        torch.cuda.synchronize()
        for s, o in zip(state, outs):
            got = o.clone()
            assert torch.equal(got, step(s))
            q = wv.rotary(s["x"][:, :hq], s["pos"], (D // 2,), interleaved=False)
            ref.check_attention(got, None, ref.attention(q, s["kc"], s["vc"], pages, s["lengths"]))


class _Strange(torch.Tensor):
    """A subclass: such tensors are marshalled in Python, plain ones in C++."""


def test_both_ways_in_give_the_same(wv):
    rot = wv.Rotation((22, 21, 21))
    kc = torch.zeros(9, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pages = torch.arange(8, dtype=torch.int32).reshape(2, 4).cuda()
    lens = torch.tensor([40, 64], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 3, 5], dtype=torch.int32).cuda()
    q, k, v = (_randn(5, h, 128, dtype=torch.bfloat16, seed=h) for h in (8, 2, 2))
    pos = _positions(5, 3)
    ranges = torch.tensor([[0, 39], [1, 40], [7, 7], [0, 60], [5, 64]], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    results = []
    for wrap in (lambda t: t), (lambda t: t.as_subclass(_Strange)):
        kc.zero_(), vc.zero_()
        q_, k_ = wrap(q), wrap(k)
        turned = wv.rotary(q_, pos, rot)
        back = wv.rotary_grad(q_, pos, (22, 21, 21))
        wv.kv_append(k_, v, kc, vc, pages, lens, cu, pos, rot)
        new = wv.kv_append(k_, v, kc, vc, pages, lens, cu, pos, rot, q=q_, status=status)
        caches = kc.clone(), vc.clone()
        out, lse = wv.kv_attention(wrap(new), kc, vc, pages, lens, cu, ranges, return_lse=True, status=status)
        one = wv.kv_attention(wrap(new[:2]), kc, vc, pages, lens, scale=0.3)
        results.append([t.as_subclass(torch.Tensor) for t in (turned, back, new, *caches, out, lse, one)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    wv.kv_status(status)


@pytest.mark.parametrize("way", ["plain", "subclass"])
def test_refusals_are_the_same_on_both_ways(wv, way):
    wrap = (lambda t: t) if way == "plain" else (lambda t: t.as_subclass(_Strange))
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    pages = torch.arange(4, dtype=torch.int32).reshape(2, 2).cuda()
    lens = torch.tensor([3, 5], dtype=torch.int32).cuda()
    q = _randn(2, 4, 64, dtype=torch.bfloat16)
    grad = wrap(q.clone()).requires_grad_()
    with pytest.raises(ValueError, match="autograd"):
        wv.kv_attention(grad, kc, kc, pages, lens)
    with torch.no_grad():
        wv.kv_attention(grad, kc, kc, pages, lens)
    with pytest.raises(ValueError, match="not on cpu|is on cpu"):
        wv.kv_attention(wrap(q), kc, kc, pages.cpu(), lens)
    with pytest.raises(ValueError, match="lengths is torch.int64"):
        wv.kv_attention(wrap(q), kc, kc, pages, lens.long())
    with pytest.raises(ValueError, match="contiguous"):
        wv.kv_attention(wrap(q), kc, kc, pages, torch.zeros(4, dtype=torch.int32, device="cuda")[::2])
    with pytest.raises(ValueError, match="rows for"):
        wv.kv_attention(wrap(q), kc, kc, pages, lens[:1])
    with pytest.raises((ValueError, wv.WanError)):
        wv.kv_attention(wrap(q[:, :3]), kc, kc, pages, lens)
    with pytest.raises(ValueError, match="positions need sections"):
        wv.kv_append(wrap(q[:, :2]), q[:, :2], kc, kc.clone(), pages, lens, positions=_positions(2, 1))
    with pytest.raises(ValueError, match="positions must be"):
        wv.rotary(wrap(q), _positions(2, 2), (32,))
    with pytest.raises((ValueError, wv.WanError)):
        wv.rotary(wrap(q), _positions(2, 1), (33,))
    with pytest.raises(ValueError, match="out is"):
        wv.rotary(wrap(q), _positions(2, 1), (32,), out=torch.empty(2, 4, 64, device="cuda"))


def test_attention_of_many_short_sequences(wv):
    """More row tiles than the card has SMs, some sequences without a key or a token."""
    g = torch.Generator().manual_seed(5)
    lens = [int(n) for n in torch.randint(0, 300, (130,), generator=g)]
    lens[3] = lens[77] = 0
    new = [min(n, int(m)) for n, m in zip(lens, torch.randint(0, 40, (130,), generator=g))]
    for D, dtype in (64, torch.bfloat16), (128, torch.float16), (256, torch.bfloat16):
        q, kc, vc, pages, lengths, cu = _attention_case(wv, lens, 2, 8, D, 16, dtype, new=new, fill=math.nan)
        ranges = _ranges("causal", lens, new)
        got, lse = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges, return_lse=True)
        ref.check_attention(got, lse, ref.attention(q, kc, vc, pages, lengths, cu, ranges))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_in_graphs(wv, D):
    """A step of many tokens, captured, replayed with other lengths, token ranges and masks in place, on two streams."""
    hq, hk, size, B, T = 8, 2, 16, 2, 120
    pages, lengths, n_pages = ref.tables([900] * B, size)
    pages = torch.cat([pages, torch.full((B, 2000), -1, dtype=torch.int32, device="cuda")], 1)
    state = []
    for i in range(2):
        state.append(dict(
            q=_randn(T, hq, D, dtype=torch.bfloat16, seed=i), k=_randn(T, hk, D, dtype=torch.bfloat16, seed=2 + i),
            v=_randn(T, hk, D, dtype=torch.bfloat16, seed=4 + i), kc=_randn(n_pages, hk, size, D, dtype=torch.bfloat16, seed=6 + i),
            vc=_randn(n_pages, hk, size, D, dtype=torch.bfloat16, seed=8 + i), cu=torch.tensor([0, 60, T], dtype=torch.int32).cuda(),
            lengths=torch.tensor([600, 300], dtype=torch.int32).cuda(), pos=_positions(T, 1, seed=i),
            ranges=torch.tensor([[0, 900]] * T, dtype=torch.int32).cuda()))

    def step(s):
        q = wv.kv_append(s["k"], s["v"], s["kc"], s["vc"], pages, s["lengths"], s["cu"], s["pos"], (D // 2,), q=s["q"])
        return wv.kv_attention(q, s["kc"], s["vc"], pages, s["lengths"], s["cu"], s["ranges"])

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
    for lens, cut in ([600, 300], 60), ([119, 900], 119), ([30, 90], 30):
        new = [cut, T - cut]
        for s in state:
            s["lengths"].copy_(torch.tensor(lens))
            s["cu"].copy_(torch.tensor([0, cut, T]))
            s["ranges"].copy_(_ranges("causal", lens, new))
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        torch.cuda.synchronize()
        for s, o in zip(state, outs):
            got = o.clone()
            assert torch.equal(got, step(s))
            q = wv.rotary(s["q"], s["pos"], (D // 2,))
            ref.check_attention(got, None, ref.attention(q, s["kc"], s["vc"], pages, s["lengths"], s["cu"], s["ranges"]))


@pytest.mark.parametrize("heads", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_attention_odd_values_of_a_block_that_half_a_tile_sees(wv, dtype, D, heads):
    """A window that moves inside a tile of 256 rows: its first 128 rows see a whole block of keys, the others only
    its later part.  Infinities there reach the rows that see them, however small (2^-43) their weights, the same in
    every call: none is taken away while a product reads it."""
    n, T = 512, 256
    q, kc, vc, pages, lengths, cu = _attention_case(wv, [n], heads, 1, D, 16, dtype, new=[T])
    q.fill_(1.0)
    kc.zero_()
    place = lambda i: (int(pages[0, i // 16]), slice(None), i % 16)  # noqa: E731
    for i, c, value in (100, 3, math.inf), (100, D - 1, -math.inf), (101, 5, math.nan), (10, 7, math.inf), (300, 3, math.inf):
        vc[place(i)][..., c] = value
    kc[place(100)] = -30.0 / D                                  # a score of -30 at a scale of one, all others 0
    ranges = torch.tensor([[0, n]] * 128 + [[40, n]] * 128, dtype=torch.int32).cuda()
    got, lse = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges, scale=1.0, return_lse=True)
    want = ref.attention(q, kc, vc, pages, lengths, cu, ranges, scale=1.0)
    assert bool(torch.isinf(want[0][:128, :, 7]).all()) and bool(torch.isfinite(want[0][128:, :, 7]).all())
    ref.check_attention(got, lse, want)
    for _ in range(20):
        again = wv.kv_attention(q, kc, vc, pages, lengths, cu, ranges, scale=1.0)
        assert torch.equal(again.nan_to_num(0.5, 1.5, 2.5), got.nan_to_num(0.5, 1.5, 2.5))


@pytest.mark.parametrize("D", [64, 128, 200])
def test_attention_bounded_wait_expires_and_is_reported(wv, D):
    """A block of keys that is never loaded (no fault: the wait for it runs out after a second): the code is reported,
    the rows are NaN with or without a status word, soon enough, and the context stays usable."""
    code = ctypes.c_int32(0)
    start = time.monotonic()
    status = wv.load().wan_selftest_kv_attention_timeout(D, ctypes.byref(code), None)
    message = wv.load().wan_vae_last_error()
    # two calls of one second each (some waits follow others): the limit is one in time, not only in tries
    assert time.monotonic() - start < 10
    assert status == 9 and code.value in (1, 2, 3), (status, code.value, message)
    assert b"bounded wait" in message
    q, kc, vc, pages, lengths, cu = _attention_case(wv, [300, 500], 2, 2, D, 64, torch.bfloat16, new=[100, 290])
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = wv.kv_attention(q, kc, vc, pages, lengths, cu, return_lse=True, status=word)
    wv.kv_status(word)
    ref.check_attention(got, lse, ref.attention(q, kc, vc, pages, lengths, cu))


@pytest.mark.parametrize("way", ["plain", "subclass"])
def test_dual_tensors_are_refused_on_both_ways(wv, way):
    wrap = (lambda t: t) if way == "plain" else (lambda t: t.as_subclass(_Strange))
    fwd = torch.autograd.forward_ad
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    pages = torch.arange(4, dtype=torch.int32).reshape(2, 2).cuda()
    lens = torch.tensor([3, 5], dtype=torch.int32).cuda()
    q = wrap(_randn(2, 2, 64, dtype=torch.bfloat16))
    with fwd.dual_level():
        dual = fwd.make_dual(q, torch.ones_like(q))
        for call in (lambda: wv.rotary(dual, _positions(2, 1), (32,)), lambda: wv.kv_append(dual, q, kc, kc.clone(), pages, lens),
                     lambda: wv.kv_append(q, q, kc, kc.clone(), pages, lens, q=dual), lambda: wv.kv_attention(dual, kc, kc, pages, lens)):
            with pytest.raises(ValueError, match="autograd"):
                call()
        wv.kv_attention(q, kc, kc, pages, lens)


@pytest.mark.parametrize("way", ["plain", "subclass"])
def test_tensors_written_in_place_are_known_to_autograd(wv, way):
    """A tensor that a call writes to counts a version on, so autograd's check finds what it saved changed; new results
    and refused calls count none."""
    wrap = (lambda t: t) if way == "plain" else (lambda t: t.as_subclass(_Strange))
    kc, vc = (torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = torch.arange(4, dtype=torch.int32).reshape(2, 2).cuda()
    lens = torch.tensor([3, 5], dtype=torch.int32).cuda()
    q = wrap(_randn(2, 2, 64, dtype=torch.bfloat16))
    pos, out = _positions(2, 1), torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    versions = lambda: [t._version for t in (q, kc, vc, out, pos, pages)]  # noqa: E731
    for call, written in ((lambda: wv.rotary(q, pos, (32,), out=out), [0, 0, 0, 1, 0, 0]),
                          (lambda: wv.rotary_grad(q, pos, (32,), out=q), [1, 0, 0, 0, 0, 0]),
                          (lambda: wv.kv_append(q, q, kc, vc, pages, lens), [0, 1, 1, 0, 0, 0]),
                          (lambda: wv.kv_append(q, q, kc, vc, pages, lens, q=q), [0, 1, 1, 0, 0, 0]),
                          (lambda: wv.kv_append(q, q, kc, vc, pages, lens, q=q, q_out=out), [0, 1, 1, 1, 0, 0]),
                          (lambda: wv.kv_attention(q, kc, vc, pages, lens, out=out), [0, 0, 0, 1, 0, 0]),
                          (lambda: wv.kv_attention(q, kc, vc, pages, lens), [0, 0, 0, 0, 0, 0])):
        before = versions()
        call()
        assert [b - a for a, b in zip(before, versions())] == written
    before = versions()
    with pytest.raises((ValueError, wv.WanError)):
        wv.rotary(q, pos, (33,), out=out)
    assert versions() == before
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = (x * out).sum()                                         # saves out
    wv.rotary(q, pos, (32,), out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():                                # tensors made here have no counter
        buffer = torch.empty_like(out)
    assert wv.rotary(q, pos, (32,), out=wrap(buffer)) is not None


def test_ordinary_calls_are_marshalled_in_cpp(wv):
    from video_vae_decoding_gb300 import _tokens, tokens
    wv.rotary(_randn(2, 4, 64), _positions(2, 1), (32,))
    assert tokens._short is _tokens


@pytest.mark.parametrize("group", [1, 8, 9, 16])
@pytest.mark.parametrize("lens", [[64], [40, 64, 17, 1], [130, 100]], ids=str)
def test_weights_of_few_rows_lose_nothing(wv, lens, group):
    """The few-row kernel's weights enter the product with v in two parts, in float16 as in bfloat16: the bound is that
    of 32-bit weights (the form for float32 queries), twice over for the parts' 2^-21, and what the least float16 value
    and its half add for each key, 1.5 * 2^-36 of the largest weight."""
    q, kc, vc, pages, lengths, cu = _attention_case(wv, lens, 4, group, 64, 16, torch.float16)
    q = (q / 8).half()                                          # scores of about one: many weights count
    got, lse = wv.kv_attention(q, kc, vc, pages, lengths, return_lse=True)
    out, err, z, zerr = ref.attention(q.float(), kc, vc, pages, lengths)
    floor = max(lens) * 1.5 * 2.0 ** -36 * vc.abs().max().double()
    ref.check_attention(got, lse, (out, 2 * err + floor, z, zerr))


def test_inputs_outlive_a_call_on_another_stream(wv):
    """Tensors of the current stream handed to a call on another one and dropped at once: their memory goes to nobody
    else before that stream has read them."""
    s = torch.cuda.Stream()
    kc, vc = (_randn(8, 2, 16, 64, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    pages = torch.arange(8, dtype=torch.int32).reshape(1, 8).cuda()
    lens, cu = torch.tensor([100], dtype=torch.int32).cuda(), torch.tensor([0, 40], dtype=torch.int32).cuda()
    keep = [_randn(40, 2, 64, dtype=torch.bfloat16, seed=i) for i in (3, 4, 5)]
    pos = _positions(40, 1)
    want_rot = wv.rotary(keep[0], pos, (32,))
    want_out = wv.kv_attention(keep[0], kc, vc, pages, lens, cu)
    k2, v2 = kc.clone(), vc.clone()
    want_q = wv.kv_append(keep[1], keep[2], k2, v2, pages, lens, cu, pos, (32,), q=keep[0])

    def overwritten(call):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)                        # 10 ms: s starts after all below is done
        got = call()
        junk = [torch.full((40, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(64)]
        junk += [torch.full((40, 1), 9, dtype=torch.int32, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        del junk
        return got
    copy = lambda i: keep[i].clone()  # noqa: E731  in memory that only the call holds
    assert torch.equal(overwritten(lambda: wv.rotary(copy(0), pos.clone(), (32,), stream=s)), want_rot)
    assert torch.equal(overwritten(lambda: wv.kv_attention(copy(0), kc, vc, pages.clone(), lens.clone(), cu.clone(), stream=s)), want_out)
    assert torch.equal(overwritten(lambda: wv.kv_append(copy(1), copy(2), kc, vc, pages, lens.clone(), cu.clone(), pos.clone(), (32,),
                                                        q=copy(0), stream=s)), want_q)
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_refusals_on_another_stream_keep_their_words(wv):
    s = torch.cuda.Stream()
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    pages = torch.arange(4, dtype=torch.int32).reshape(2, 2).cuda()
    lens = torch.tensor([3, 5], dtype=torch.int32).cuda()
    q = _randn(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q is on cpu"):
        wv.kv_append(q, q, kc, kc.clone(), pages, lens, q=q.cpu(), stream=s)
    with pytest.raises(ValueError, match="out is on cpu"):
        wv.kv_attention(q, kc, kc, pages, lens, out=q.cpu(), stream=s)
    with pytest.raises(ValueError, match="out is on cpu"):
        wv.rotary(q, _positions(2, 1), (32,), out=q.cpu(), stream=s)
    with pytest.raises(ValueError, match="on cuda|CUDA|cpu"):
        wv.kv_attention(q.cpu(), kc, kc, pages, lens, stream=s)

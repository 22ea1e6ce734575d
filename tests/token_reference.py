"""Plain 64-bit forms of the token operators, and what the kernels may be off
by, for their tests."""

import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def frequencies(sections, theta=10000.0):
    freq = [theta ** (-i / n) for n in sections for i in range(n)]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return torch.tensor(freq, dtype=torch.float64), torch.tensor(axis)


def rotary(x, positions, sections, theta=10000.0, interleaved=True, sign=1.0, freq=None):
    """x [..., T, H, D] turned, in 64 bits; and a bound of a 32-bit computation's error."""
    f, axis = frequencies(sections, theta)
    if freq is not None:
        f = torch.tensor(freq, dtype=torch.float64)
    pos = positions.to(torch.float64).to(x.device)
    angle = (sign * pos[..., axis.to(x.device)] * f.to(x.device))[..., None, :]
    cos, sin = angle.cos(), angle.sin()
    n, y = f.numel(), x.double()
    out = y.clone()
    a, b = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if interleaved else (y[..., :n], y[..., n:2 * n])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    # The angle (a fraction of a half turn, rounded to 24 bits: pi 2^-25), the
    # library's sine and cosine (2 units of 2^-24) and the product and sum
    # (2^-24 each of terms up to |a| + |b|) are off by under 2^-21 (|a| + |b|);
    # the frequency, rounded to 2^-53 and to 2^-64 of a turn, turns a position p
    # by up to |p| 2^-51 more, here and in this function alike.
    off = (a.abs() + b.abs()) * (2.0 ** -21 + pos.abs().amax() * 2.0 ** -51)
    err = torch.zeros_like(out)
    if interleaved:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = ra, rb
        err[..., 0:2 * n:2], err[..., 1:2 * n:2] = off, off
    else:
        out[..., :n], out[..., n:2 * n] = ra, rb
        err[..., :n], err[..., n:2 * n] = off, off
    return out, err


def assert_rounded(got, ref, err, what=""):
    """got is ref, off by err, rounded once to its type."""
    fine = torch.isfinite(ref)
    if not fine.all():
        assert torch.equal(got[~fine].double().nan_to_num(0.5), ref[~fine].nan_to_num(0.5)), what
        got, ref, err = got[fine], ref[fine], err[fine]
    tol = err + HALF[got.dtype] * (ref.abs() + err) + TINY[got.dtype]
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), (got.double() - ref).abs().max().item(), bad.nonzero()[:3].tolist())


def keys_of(cache, row, n, head):
    """The first n rows of a sequence: [n, D] in 64 bits."""
    size = cache.shape[2]
    at = torch.arange(n, device=cache.device)
    return cache[row[at // size].long(), head, at % size].double()


def attention(q, k_cache, v_cache, pages, lengths, cu=None, ranges=None, scale=None):
    """out, lse in 64 bits, and bounds of the kernels' errors.

    A score, summed in 32 bits over D products (a tensor core's chained sums
    round or cut to 2^-23 of the running sum, D / 8 times at most), is off by
    ds = D / 8 * 2^-23 * scale * sum |q k|, and by two roundings of itself.  A
    weight exp(s - m) is then off by 2 ds relatively (its own score and the
    maximum), by 2^-21 for the exponential, and by half a step of its 16-bit
    type as it enters the product with v; in float16 one below 2^-24 is lost
    (2^-25 of the largest weight).  Each of the n / 8 chained sums of the
    product rounds to 2^-23 of sum p |v|.  The division by the sum doubles
    what the weights are off by."""
    T, H, D = q.shape
    Hk = k_cache.shape[1]
    g = H // Hk
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    lse_err = torch.zeros_like(lse)
    B = lengths.numel()
    cu = list(range(B + 1)) if cu is None else cu.tolist()
    for b in range(B):
        n = int(lengths[b])
        rows = slice(cu[b], cu[b + 1])
        if n == 0 or cu[b] == cu[b + 1]:
            continue
        at = torch.arange(n, device=q.device)[None, None]
        if ranges is None:
            seen = torch.ones(1, cu[b + 1] - cu[b], n, dtype=torch.bool, device=q.device)
        else:
            r = ranges[rows].long()
            seen = (at >= r[None, :, :1]) & (at < r[None, :, 1:])
        some = seen.any(-1)  # [1, t]
        for h in range(Hk):
            k, v = keys_of(k_cache, pages[b], n, h), keys_of(v_cache, pages[b], n, h)
            hs = slice(h * g, h * g + g)
            mine = q[rows, hs].double().transpose(0, 1)  # [g, t, D]
            s = mine @ k.T * scale
            ds = (D / 8 * 2.0 ** -23) * abs(scale) * (mine.abs() @ k.abs().T) + 2.0 ** -22 * s.abs()
            s = torch.where(seen, s, -math.inf)
            ds = torch.where(seen, ds, 0.0).amax(-1)
            z = torch.logsumexp(s, -1)
            p = torch.where(seen & some[..., None], (s - z[..., None]).exp(), 0.0)
            v0 = torch.where(seen.any(1)[0][:, None], v, 0.0)
            if torch.isfinite(v0).all():
                o = p @ v0
            else:  # what a row does not see must not reach it: 0 times an infinity is a NaN
                o = torch.stack([p[:, t][:, seen[0, t if ranges is not None else 0]] @
                                 v[seen[0, t if ranges is not None else 0]] for t in range(mine.shape[1])], 1)
                v0 = torch.nan_to_num(v0, 0.0, 0.0, 0.0)
            pv = p @ v0.abs()
            half = HALF[q.dtype]
            w = 2 * ds + 2.0 ** -21 + half
            e = (2 * w + (n / 8 + 8) * 2.0 ** -23)[..., None] * pv
            if q.dtype == torch.float16:
                e = e + n * 2.0 ** -25 * torch.nan_to_num(v0.abs(), 0.0, 0.0, 0.0).amax()
            out[rows, hs], err[rows, hs] = o.transpose(0, 1), e.transpose(0, 1)
            lse[rows, hs] = torch.where(some, z, -math.inf).T
            lse_err[rows, hs] = (ds + (n / 8 + 8) * 2.0 ** -23 + 2.0 ** -22 * z.abs().nan_to_num(0.0, 0.0, 0.0)).T
    return out, err, lse, lse_err


def check_attention(got, lse, ref, what=""):
    out, err, z, zerr = ref
    assert_rounded(got, out, err, what)
    if lse is not None:
        empty = torch.isinf(z)
        assert torch.equal(torch.isinf(lse) & (lse < 0), empty), what
        d = (lse.double() - z)[~empty].abs()
        assert bool((d <= zerr[~empty]).all()), (what, d.max().item())
        assert not got[empty].any(), what


def tables(lens, page_size, spare=3, seed=0, device="cuda"):
    """pages, lengths and the number of pages of a cache that holds them in a random order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page_size) for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g).int()
    pages = torch.zeros(len(lens), max(1, *need) if len(need) > 1 else max(1, need[0]), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    return pages.to(device), torch.tensor(lens, dtype=torch.int32, device=device), n_pages

"""Plain 64-bit forms of the operators that see, copy and move keys by their
place in a sequence, for their tests."""

import math

import torch

from tests.token_reference import HALF, keys_of


def window_sees(n, m, window, sinks, frame):
    """[m, n]: what the last m of n tokens see."""
    sees = torch.zeros(m, n, dtype=torch.bool)
    for i in range(m):
        f = (n - m + i) // frame
        sees[i, :sinks] = True
        sees[i, max(0, (f - window + 1) * frame):(f + 1) * frame] = True
        sees[i, (f + 1) * frame:] = False                # first keys that are later ones too
    return sees


def tree_sees(n, parents):
    m = len(parents)
    sees = torch.zeros(m, n, dtype=torch.bool)
    sees[:, :n - m] = True
    for i, p in enumerate(parents):
        if 0 <= p < i:
            sees[i] |= sees[p]
        sees[i, n - m + i] = True
    return sees


def attention(q, k_cache, v_cache, pages, lengths, cu, sees, scale=None):
    """out, lse and bounds of their errors (derived at token_reference.attention), sees[b] being [tokens, keys]."""
    T, H, D = q.shape
    Hk = k_cache.shape[1]
    g = H // Hk
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    lse_err = torch.zeros_like(lse)
    half = HALF[q.dtype]
    for b in range(len(sees)):
        rows, seen = slice(int(cu[b]), int(cu[b + 1])), sees[b].to(q.device)
        n = seen.shape[1]
        if not seen.any():
            continue
        live = seen.any(0)                                   # keys that some row sees: others are not looked at
        at = live.nonzero()[:, 0]
        some = seen.any(1)
        for h in range(Hk):
            size = k_cache.shape[2]
            page, off = pages[b][at // size].long(), at % size
            k, v = k_cache[page, h, off].double(), v_cache[page, h, off].double()
            hs = slice(h * g, h * g + g)
            mine = q[rows, hs].double().transpose(0, 1)     # [g, m, D]
            see = seen[:, live][None]
            s = mine @ k.T * scale
            ds = (D / 8 * 2.0 ** -23) * abs(scale) * (mine.abs() @ k.abs().T) + 2.0 ** -22 * s.abs()
            s = torch.where(see, s, -math.inf)
            ds = torch.where(see, ds, 0.0).amax(-1)
            z = torch.logsumexp(s, -1)
            p = torch.where(see & some[None, :, None], (s - z[..., None]).exp(), 0.0)
            if torch.isfinite(v).all():
                o = p @ v
            else:  # what a row does not see must not reach it: 0 times an infinity is a NaN
                o = torch.stack([p[:, t][:, see[0, t]] @ v[see[0, t]] for t in range(mine.shape[1])], 1)
            v0 = torch.nan_to_num(v.abs(), 0.0, 0.0, 0.0)
            pv = p.nan_to_num(0.0) @ v0
            w = 2 * ds + 2.0 ** -21 + half
            e = (2 * w + (n / 8 + 8) * 2.0 ** -23)[..., None] * pv
            if q.dtype == torch.float16:
                e = e + n * 2.0 ** -25 * v0.amax()
            out[rows, hs], err[rows, hs] = o.transpose(0, 1), e.transpose(0, 1)
            lse[rows, hs] = torch.where(some, z, -math.inf).T
            lse_err[rows, hs] = (ds + (n / 8 + 8) * 2.0 ** -23 + 2.0 ** -22 * z.abs().nan_to_num(0.0, 0.0, 0.0)).T
    return out, err, lse, lse_err


def fork(k_cache, v_cache, pages, lengths, sources, targets, fresh, share):
    """The caches (in their own type), pages and lengths after the forks; arguments unchanged."""
    size = k_cache.shape[2]
    k, v, pages, lengths = k_cache.clone(), v_cache.clone(), pages.clone(), lengths.clone()
    was, n_of = pages.tolist(), lengths.tolist()
    for s, t, f in zip(sources, targets, fresh.tolist()):
        n = n_of[s]
        whole = n // size if share else 0
        for j in range(-(-n // size)):
            to = was[s][j] if j < whole else f[j - whole]
            pages[t, j] = to
            if j >= whole:
                r = min(size, n - j * size)
                for new, old in (k, k_cache), (v, v_cache):
                    new[to, :, :r] = old[was[s][j], :, :r]
        lengths[t] = n
    return k, v, pages, lengths


def compact(k_cache, v_cache, pages, first, keeps):
    """The caches after the moves, and the lengths."""
    size = k_cache.shape[2]
    k, v = k_cache.clone(), v_cache.clone()
    for b, keep in enumerate(keeps):
        if not len(keep):
            continue
        a = torch.tensor(keep, device=k.device)
        z = first[b] + torch.arange(len(keep), device=k.device)
        pa, pz = pages[b][a // size].long(), pages[b][z // size].long()
        for new, old in (k, k_cache), (v, v_cache):
            new[pz, :, z % size] = old[pa, :, a % size]
    return k, v, [f + len(keep) for f, keep in zip(first, keeps)]


__all__ = ["window_sees", "tree_sees", "attention", "fork", "compact", "keys_of"]

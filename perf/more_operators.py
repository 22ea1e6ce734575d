"""Operators of a cache that outlives its clip: cases, plain forms and exact values.

A streaming video model runs on while its paged key-value cache may not grow: it
attends to the frames of a window and to its first ones; it drafts several
continuations at once, as a tree, and keeps the branch that it accepts; it tries
several futures of one past; and it drops what it needs no more.  Four operators,
each computed by elementary torch operations (the plain form) or, with ``own``
set, by this package's kernels:

window   softmax(q k^T * scale) v over the first keys and a window of the last
         ones, by keys or by whole frames, for one new token per sequence or many
tree     the same for a tree of drafted tokens: each sees all keys before the
         drafts, its ancestors and itself
fork     sequences become copies of others: whole pages shared, the last one
         copied, or all of them copied
compact  a sequence's kept keys and values move together in its pages
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of a few streams that run on: where the launch is what counts
        dict(name="window_step", op="window", dtype="bf16", batch=4, new_min=1, new_max=1, len_min=900, len_max=1500,
             q_heads=16, kv_heads=16, head_dim=128, page=16, window=500, sinks=4, frame=1),
        # a serving batch of long ragged sequences, four query heads on each key head
        dict(name="window_batch", op="window", dtype="bf16", batch=48, new_min=1, new_max=1, len_min=1000, len_max=20000,
             q_heads=32, kv_heads=8, head_dim=128, page=64, window=4096, sinks=128, frame=1),
        # one new latent frame of a 720p clip (880 tokens) that sees the first frame and the last nine
        dict(name="window_frame", op="window", dtype="bf16", batch=1, new_min=880, new_max=880, len_min=27280, len_max=27280,
             q_heads=16, kv_heads=16, head_dim=128, page=880, window=9, sinks=880, frame=880),
        # ragged prompts, each token seeing the last thousand keys or so and the first sixteen
        dict(name="window_prompts", op="window", dtype="fp16", batch=5, new_min=1, new_max=2500, len_min=2500, len_max=6000,
             q_heads=20, kv_heads=4, head_dim=64, page=32, window=1000, sinks=16, frame=1),
        # the drafts of one stream against two thousand keys
        dict(name="tree_one", op="tree", dtype="bf16", batch=1, new_min=26, new_max=26, len_min=2026, len_max=2026,
             q_heads=16, kv_heads=16, head_dim=128, page=16),
        # a serving batch, 64 drafts a sequence, four query heads on each key head
        dict(name="tree_batch", op="tree", dtype="bf16", batch=24, new_min=64, new_max=64, len_min=300, len_max=9000,
             q_heads=32, kv_heads=8, head_dim=128, page=64),
        # trees of all sizes, a group of five query heads, a head dim and a page that are no powers of two
        dict(name="tree_odd", op="tree", dtype="fp16", batch=9, new_min=1, new_max=47, len_min=50, len_max=3001,
             q_heads=20, kv_heads=4, head_dim=80, page=24),
        # four futures of each of six streams, the pasts' whole pages shared
        dict(name="fork_futures", op="fork", dtype="bf16", batch=6, copies=4, len_min=100, len_max=9000, kv_heads=8,
             head_dim=128, page=64, share=True),
        # three copies of a whole 720p clip's cache, one page a latent frame
        dict(name="fork_clip", op="fork", dtype="bf16", batch=1, copies=3, len_min=27280, len_max=27280, kv_heads=16,
             head_dim=128, page=880, share=False),
        # the accepted path of 64 drafts of each of 24 sequences
        dict(name="compact_drafts", op="compact", dtype="bf16", batch=24, len_min=300, len_max=9000, kv_heads=8, head_dim=128,
             page=64, first_min=64, first_max=64, kept_min=1, kept_max=6, how="drafts"),
        # a clip's cache rolls on: the first frame stays, the last thirteen of 31 move up to it
        dict(name="compact_roll", op="compact", dtype="bf16", batch=1, len_min=27280, len_max=27280, kv_heads=16,
             head_dim=128, page=880, first_min=880, first_max=880, kept_min=11440, kept_max=11440, how="last"),
        # ragged sequences keep the keys that were attended to most, wherever those are
        dict(name="compact_choice", op="compact", dtype="fp16", batch=13, len_min=4000, len_max=16001, kv_heads=8,
             head_dim=96, page=32, first_min=4, first_max=64, kept_min=500, kept_max=1900, how="choice"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "tree", "tree", "fork", "compact", "compact"])
    head_dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 12, 16])
    page = rng.choice([16, 16, 24, 32, 64, 64, 128, 256, 390, 880])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), kv_heads=kv_heads, head_dim=head_dim, page=page)
    row = kv_heads * head_dim
    if op == "fork":
        batch, copies = rng.choice([1, 1, 2, 3, 6, 12]), rng.choice([1, 2, 3, 4, 8])
        length = _log(rng, 1, min(40000, 150_000_000 // (row * batch * copies)))
        return dict(case, batch=batch, copies=copies, len_min=rng.randint(1, length), len_max=length,
                    share=rng.random() < 0.5)
    if op == "compact":
        how = rng.choice(["drafts", "last", "choice"])
        batch = rng.choice([1, 1, 2, 4, 9, 24])
        length = _log(rng, 12, min(40000, 56_000_000 // (row * batch)))
        least = rng.randint(max(12, length // 3), length)
        first = rng.randint(2, min(300, least - 1)) if how == "drafts" else rng.randint(0, min(900, least // 2))
        room = first if how == "drafts" else least - first
        most = min(12, room // 2) if how == "drafts" else room // 2
        kept = _log(rng, 1, max(1, most))
        return dict(case, batch=batch, len_min=least, len_max=length, first_min=first, first_max=first,
                    kept_min=rng.randint(0, kept), kept_max=kept, how=how)
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    while kv_heads * group > 64:
        group //= 2
    case["q_heads"] = heads = kv_heads * group
    # the most query-key pairs and cached keys: those of the largest listed case
    pairs = min(27280 * 16 * 880, 27280 * 880 * 2048 // head_dim)
    if op == "tree":
        batch = rng.choice([1, 1, 2, 5, 12, 24])
        new_max = _log(rng, 1, min(200, math.isqrt(pairs // (batch * heads))))
        length = new_max + _log(rng, 1, max(1, min(30000, pairs // (batch * heads * new_max), 56_000_000 // (row * batch))))
        return dict(case, batch=batch, new_min=rng.randint(1, new_max), new_max=new_max, len_min=new_max, len_max=length)
    frame = rng.choice([1, 1, rng.randint(2, 900)])
    if rng.random() < 0.5:
        batch = _log(rng, 1, 64)
        new_max = 1
    else:
        batch = rng.choice([1, 1, 2, 3, 5])
        new_max = _log(rng, 2, min(2500, math.isqrt(pairs // (batch * heads))))
    length = _log(rng, new_max, max(new_max, min(60000, pairs // (batch * heads * new_max), 100_000_000 // (row * batch))))
    window = _log(rng, 1, max(1, min(length, 20000) // frame))
    return dict(case, batch=batch, new_min=rng.randint(1, new_max), new_max=new_max, len_min=new_max, len_max=length,
                window=window, sinks=rng.choice([0, 1, 4, 16, frame, rng.randint(0, 2000)]), frame=frame)


# ------------------------------------------------------------------ sizes
def _between(case, what, n):
    """n sizes spread over [min, max], the largest among them: a case's own, whatever the seed."""
    lo, hi = case[what + "_min"], case[what + "_max"]
    g = torch.Generator().manual_seed(hi * 7 + lo + n)
    got = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    got[n // 2] = hi
    return got


def _lens(case):
    lens = _between(case, "len", case["batch"])
    if "new_max" in case:
        new = _between(case, "new", case["batch"])
        return [max(a, b) for a, b in zip(lens, new)], new
    return lens, None


def _firsts_and_kept(case, lens):
    """How many keys of each sequence stay where they are, and how many of the later ones are kept."""
    first, kept = _between(case, "first", case["batch"]), _between(case, "kept", case["batch"])
    if case["how"] == "drafts":  # `first` counts the drafts: what is ahead of them stays
        first = [n - f for n, f in zip(lens, first)]
    return first, [min(k, (n - f) // 2) for k, n, f in zip(kept, lens, first)]


def _seen(case, place, length):
    """The keys that a token at `place` sees: [0, a) and [b, c)."""
    after = (place // case["frame"] + 1) * case["frame"]
    b, c = max(0, after - case["window"] * case["frame"]), min(length, after)
    return min(case["sinks"], b), b, c


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    d = torch.device("cuda")
    g = torch.Generator(device=d).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    dtype, batch, page = DTYPES[case["dtype"]], case["batch"], case["page"]
    kv, hd, op = case["kv_heads"], case["head_dim"], case["op"]
    lens, new = _lens(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=d, dtype=torch.float32).to(dtype)

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=d)

    s = dict(case=case, lens=lens, new=new)
    copies = batch * case["copies"] if op == "fork" else 0
    per = -(-max(lens) // page)  # pages of the longest sequence
    need = [-(-n // page) for n in lens]
    past = [lens[i % batch] for i in range(copies)]
    spare = [(n % page > 0) if case["share"] else -(-n // page) for n in past] if copies else []
    n_pages = sum(need) + sum(spare) + 3  # and a few that belong to nobody
    order = torch.randperm(n_pages, generator=host).to(torch.int32)
    pages = torch.zeros(batch + copies, per, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    if copies:
        fresh = torch.zeros(copies, 1 if case["share"] else per, dtype=torch.int32)
        for i, n in enumerate(spare):
            fresh[i, :n] = order[at:at + n]
            at += n
        s.update(fresh=fresh.to(d), sources=i32([i % batch for i in range(copies)]), targets=i32(list(range(batch, batch + copies))),
                 past=past)
    s.update(pages=pages.to(d), lengths=i32(lens + [0] * copies), most_keys=max(lens),
             k_cache=normal(n_pages, kv, page, hd), v_cache=normal(n_pages, kv, page, hd))
    if op == "compact":
        first, kept = _firsts_and_kept(case, lens)
        keep = []
        for n, f, k in zip(lens, first, kept):
            if case["how"] == "last":
                keep.append(torch.arange(n - k, n))
            else:  # later than the places that they move to, as most of a tree's paths and of a long cache's keys are
                keep.append((f + k + torch.randperm(n - f - k, generator=host)[:k]).sort()[0])
        s.update(first=i32(first), keep=torch.cat(keep).to(torch.int32).to(d),
                 cu=i32([0] + [sum(kept[:b + 1]) for b in range(batch)]))
    if op in ("window", "tree"):
        total = sum(new)
        # scores of a trained model spread wider than those of independent normal vectors
        s["q"] = (torch.randn(total, case["q_heads"], hd, generator=g, device=d) * 1.5).to(dtype)
        s.update(cu=i32([0] + [sum(new[:b + 1]) for b in range(batch)]), most_new=max(new))
    if op == "tree":
        parents = []
        for n in new:  # about three children each, some drafts without a parent
            i = torch.arange(n)
            up = (i - 1) // 3 + torch.randint(-2, 3, (n,), generator=host)
            up = torch.minimum(up.clamp(min=0), i - 1)
            parents.append(torch.where(torch.rand(n, generator=host) < 0.03, -1, up))
        s["parents"] = torch.cat(parents).to(torch.int32).to(d)
    return s


# ------------------------------------------------------------ plain forms
def _rows(cu, total):
    """The sequence of each row, and the row's place among its sequence's."""
    row = torch.arange(total, device=cu.device)
    seq = torch.bucketize(row, cu[1:].long(), right=True)
    return seq, row - cu.long()[seq]


def _gathered(cache, pages, keys):
    """The first `keys` entries of every sequence: [batch, keys, kv_heads, head_dim] in 32 bits."""
    page = cache.shape[2]
    at = torch.arange(keys, device=cache.device)
    return cache[pages[:, at // page].long(), :, (at % page)[None]].float()


def _window_hidden(s, seq, place):
    """[rows, keys]: what each token does not see."""
    case = s["case"]
    n = s["lengths"].long()[seq]
    p = n - (s["cu"][1:] - s["cu"][:-1]).long()[seq] + place
    after = (p // case["frame"] + 1) * case["frame"]
    first = (after - case["window"] * case["frame"]).clamp(min=0)[:, None]
    at = torch.arange(s["most_keys"], device=p.device)[None]
    return ((at >= case["sinks"]) & (at < first)) | (at >= after[:, None]) | (at >= n[:, None])


def _tree_hidden(s, seq, place):
    n = s["lengths"].long()[seq]
    base = n - (s["cu"][1:] - s["cu"][:-1]).long()[seq]
    at = torch.arange(s["most_keys"], device=n.device)[None]
    hidden = at >= base[:, None]
    row = torch.arange(seq.numel(), device=n.device)
    begin = s["cu"].long()[seq]
    node = place.clone()  # an ancestor of each token, up to the root
    for _ in range(s["most_new"]):
        live = node >= 0
        spot = (base + node).clamp(min=0)
        hidden[row, spot] = hidden[row, spot] & ~live
        node = torch.where(live, s["parents"].long()[begin + node.clamp(min=0)], -1)
    return hidden


def _attend(s, hidden_of):
    """q's tokens, padded to the most of a sequence, against all keys, padded to the longest sequence."""
    q, cu, batch = s["q"], s["cu"], s["case"]["batch"]
    total, heads, hd = q.shape
    kv = s["k_cache"].shape[1]
    k, v = _gathered(s["k_cache"], s["pages"], s["most_keys"]), _gathered(s["v_cache"], s["pages"], s["most_keys"])
    seq, place = _rows(cu, total)
    qp = torch.zeros(batch, s["most_new"], heads, hd, device=q.device)
    qp[seq, place] = q.float()
    hidden = torch.ones(batch, s["most_new"], s["most_keys"], dtype=torch.bool, device=q.device)
    hidden[seq, place] = hidden_of(s, seq, place)
    qg = qp.view(batch, s["most_new"], kv, heads // kv, hd).permute(0, 2, 3, 1, 4).reshape(batch, kv, -1, hd)
    scores = qg @ k.permute(0, 2, 3, 1)
    scores = scores.view(batch, kv, heads // kv, s["most_new"], -1) * (1.0 / math.sqrt(hd))
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    total_p = p.sum(-1, keepdim=True)
    o = p.view(batch, kv, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3)
    o = o.view(batch, kv, heads // kv, s["most_new"], hd) / total_p.clamp(min=1e-38)
    lse = (top + total_p.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, s["most_new"], heads, hd)[seq, place]
    lse = lse.permute(0, 3, 1, 2).reshape(batch, s["most_new"], heads)[seq, place]
    return {"out": o.to(q.dtype), "lse": lse}


def _fork(s):
    page, share = s["case"]["page"], s["case"]["share"]
    pages, fresh, sources, targets = s["pages"], s["fresh"], s["sources"].long(), s["targets"].long()
    begin = [n // page * page if share else 0 for n in s["past"]]  # the first key that is copied
    i = torch.cat([torch.full((n - b,), j, device=pages.device) for j, (n, b) in enumerate(zip(s["past"], begin))])
    at = torch.cat([torch.arange(b, n, device=pages.device) for n, b in zip(s["past"], begin)])
    first = torch.tensor(begin, device=pages.device)
    have = pages.long()[sources[i], at // page]
    to = fresh.long()[i, (at - first[i]) // page]
    for cache in s["k_cache"], s["v_cache"]:
        cache[to, :, at % page] = cache[have, :, at % page]
    slot = torch.arange(pages.shape[1], device=pages.device)[None]
    whole = first[:, None] // page
    held = torch.tensor([-(-n // page) for n in s["past"]], device=pages.device)[:, None]
    mine = torch.gather(fresh, 1, (slot - whole).clamp(0, fresh.shape[1] - 1).expand(fresh.shape[0], -1))
    was = pages[targets]
    pages[targets] = torch.where(slot < whole, pages[sources], torch.where(slot < held, mine, was))
    s["lengths"][targets] = s["lengths"][sources]
    return {k: s[k] for k in ("k_cache", "v_cache", "pages", "lengths")}


def _compact(s):
    page, cu, first, keep = s["case"]["page"], s["cu"], s["first"].long(), s["keep"].long()
    seq, place = _rows(cu, keep.numel())
    to = first[seq] + place
    pages = s["pages"].long()
    for cache in s["k_cache"], s["v_cache"]:
        cache[pages[seq, to // page], :, to % page] = cache[pages[seq, keep // page], :, keep % page]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": s["first"] + cu[1:] - cu[:-1]}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import video_vae_decoding_gb300 as wv

        cache = s["k_cache"], s["v_cache"], s["pages"]
        if op == "window":
            o, lse = wv.kv_window_attention(s["q"], *cache, s["lengths"], case["window"], sinks=case["sinks"],
                                            frame=case["frame"], cu_tokens=None if case["new_max"] == 1 else s["cu"],
                                            return_lse=True)
            return {"out": o, "lse": lse}
        if op == "tree":
            o, lse = wv.kv_tree_attention(s["q"], *cache, s["lengths"], s["parents"], cu_tokens=s["cu"], return_lse=True)
            return {"out": o, "lse": lse}
        if op == "fork":
            wv.kv_fork(*cache, s["lengths"], s["sources"], s["targets"], s["fresh"], share=case["share"])
            return {k: s[k] for k in ("k_cache", "v_cache", "pages", "lengths")}
        lengths = wv.kv_compact(*cache, s["first"], s["keep"], s["cu"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lengths": lengths}
    if op in ("window", "tree"):
        return _attend(s, _window_hidden if op == "window" else _tree_hidden)
    return _fork(s) if op == "fork" else _compact(s)


# ------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that a pass cannot do without, of the case's own sizes."""
    lens, new = _lens(case)
    page, row = case["page"], case["kv_heads"] * case["head_dim"] * 2 * 2  # bytes of a key and its value
    if case["op"] == "fork":
        # each key that is copied is read once, however many copies are made of it
        copied = [n % page if case["share"] else n for n in lens]
        tables = sum(-(-n // page) for n in lens) * 4 * (1 + case["copies"])
        return {"bytes": sum(copied) * row * (1 + case["copies"]) + tables, "flops": 0}
    if case["op"] == "compact":
        kept = sum(_firsts_and_kept(case, lens)[1])
        return {"bytes": 2 * kept * row + 4 * kept, "flops": 0}
    read = pairs = 0
    for n, m in zip(lens, new):
        if case["op"] == "tree":
            read += n
            pairs += m * (n - m) + min(m * 6, m * (m + 1) // 2)  # a draft and its ancestors: a few
            continue
        seen = [_seen(case, p, n) for p in range(n - m, n)]
        pairs += sum(a + c - b for a, b, c in seen)
        lo, hi = min(b for _, b, _ in seen), max(c for _, _, c in seen)
        read += min(max(a for a, _, _ in seen), lo) + hi - lo
    rows = sum(new) * case["q_heads"]
    return {"bytes": read * row + rows * (2 * case["head_dim"] * 2 + 4), "flops": 4 * pairs * case["q_heads"] * case["head_dim"]}


# ------------------------------------------------------------------ exact
def _exact_moves(s):
    """fork and compact by sequences, in Python's own integers; the values move as they are."""
    case, page = s["case"], s["case"]["page"]
    pages, lengths = s["pages"].tolist(), s["lengths"].tolist()
    old = s["k_cache"].double(), s["v_cache"].double()
    new = old[0].clone(), old[1].clone()

    def move(a, b):  # (page, row) of each key: from, to
        if a:
            (ap, ar), (bp, br) = (torch.tensor(list(zip(*x)), device=old[0].device) for x in (a, b))
            for o, n in zip(old, new):
                n[bp, :, br] = o[ap, :, ar]

    if case["op"] == "compact":
        first, keep, cu = s["first"].tolist(), s["keep"].tolist(), s["cu"].tolist()
        for b, table in enumerate(pages):
            kept = keep[cu[b]:cu[b + 1]]
            move([(table[k // page], k % page) for k in kept],
                 [(table[(first[b] + j) // page], (first[b] + j) % page) for j in range(len(kept))])
            lengths[b] = first[b] + len(kept)
        return {"k_cache": new[0], "v_cache": new[1], "lengths": torch.tensor(lengths, dtype=torch.int32)}
    for p, t, fresh in zip(s["sources"].tolist(), s["targets"].tolist(), s["fresh"].tolist()):
        n = lengths[p]
        whole = n // page if case["share"] else 0
        for j in range(-(-n // page)):
            pages[t][j] = pages[p][j] if j < whole else fresh[j - whole]
        lengths[t] = n
        keys = range(whole * page, n)
        move([(pages[p][k // page], k % page) for k in keys], [(pages[t][k // page], k % page) for k in keys])
    return {"k_cache": new[0], "v_cache": new[1], "pages": torch.tensor(pages, dtype=torch.int32),
            "lengths": torch.tensor(lengths, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return _exact_moves(s)
    cu, lens, new, page = s["cu"].tolist(), s["lens"], s["new"], case["page"]
    q, group = s["q"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b in range(case["batch"]):
        n, m = lens[b], new[b]
        sees = torch.zeros(m, n, dtype=torch.bool)
        if case["op"] == "window":
            for i in range(m):
                first, lo, hi = _seen(case, n - m + i, n)
                sees[i, :first] = True
                sees[i, lo:hi] = True
        else:
            sees[:, :n - m] = True
            up = s["parents"][cu[b]:cu[b + 1]].tolist()
            for i in range(m):  # a parent comes before its children: what it sees is known
                if up[i] >= 0:
                    sees[i] = sees[up[i]]
                sees[i, n - m + i] = True
        sees = sees.to(q.device)
        held = s["pages"][b, :-(-n // page)].long()
        for h in range(case["kv_heads"]):
            k = s["k_cache"][held, h].reshape(-1, case["head_dim"])[:n].double()
            v = s["v_cache"][held, h].reshape(-1, case["head_dim"])[:n].double()
            mine = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].double()
            logit = torch.einsum("thd,nd->htn", mine, k) / math.sqrt(case["head_dim"])
            logit = torch.where(sees[None], logit, -math.inf)
            z = torch.logsumexp(logit, -1)
            out[cu[b]:cu[b + 1], h * group:(h + 1) * group] = torch.einsum("htn,nd->thd", (logit - z[..., None]).exp(), v)
            lse[cu[b]:cu[b + 1], h * group:(h + 1) * group] = z.T
    return {"out": out, "lse": lse}

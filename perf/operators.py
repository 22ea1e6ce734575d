"""The token operators in front of the decode: cases, plain forms and exact values.

A streaming video model produces the latents that the decoder turns into
frames: it rotates queries and keys by their place in the clip (time, height,
width), appends each new latent frame's keys and values to a paged cache, and
attends over everything cached, a whole frame of tokens at a time or one token.
Five operators, each computed by elementary torch operations (the plain form)
or, with ``own`` set, by this package's kernels:

rotary       y = rotation of x's channel pairs by position x frequency
rotary_grad  its gradient: the rotation by the opposite angles
append       new keys (rotated) and values into the pages of a cache, with the
             queries rotated in the same call
decode       softmax(q k^T * scale) v for one new token per sequence
chunk        the same for many new tokens per sequence, each seeing a range of
             keys
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one denoising step's smallest call: a handful of tokens, where the launch is what counts
        dict(name="rotary_step", op="rotary", dtype="bf16", batch=4, tokens=1, heads=16, head_dim=128,
             sections="22,21,21", grid="1,1,1", interleaved=True, start=27),
        # the queries of a whole 720p clip: 31 latent frames of 44 x 80 in 2 x 2 patches
        dict(name="rotary_clip", op="rotary", dtype="bf16", batch=1, tokens=31 * 22 * 40, heads=16, head_dim=128,
             sections="22,21,21", grid="31,22,40", interleaved=True, start=0),
        # the backward pass of a training step on two smaller clips in 32 bits, halves rotated against each other
        dict(name="rotary_grad", op="rotary_grad", dtype="fp32", batch=2, tokens=7 * 30 * 39, heads=12, head_dim=80,
             sections="8,16,16", grid="7,30,39", interleaved=False, start=0),
        # one new token of each of 16 sequences, queries rotated in the same call
        dict(name="append_step", op="append", dtype="fp16", batch=16, new_min=1, new_max=1, len_min=100, len_max=4000,
             q_heads=32, kv_heads=8, head_dim=128, page=16, sections="64", interleaved=False),
        # four latent frames of a 720p clip, one page a frame
        dict(name="append_frames", op="append", dtype="bf16", batch=1, new_min=3520, new_max=3520, len_min=7040,
             len_max=7040, q_heads=16, kv_heads=16, head_dim=128, page=880, sections="22,21,21", interleaved=True),
        # ragged prompts, keys and values alone, channels past the rotated ones, an odd head dim
        dict(name="append_prompts", op="append", dtype="bf16", batch=7, new_min=1, new_max=8191, len_min=8191,
             len_max=9000, q_heads=0, kv_heads=4, head_dim=96, page=64, sections="40", interleaved=False),
        # one sequence of about a thousand keys, a head of its own for each query head
        dict(name="decode_one", op="decode", dtype="bf16", batch=1, len_min=1000, len_max=1000, q_heads=16,
             kv_heads=16, head_dim=128, page=16),
        # a serving batch: ragged lengths, four query heads on each key head
        dict(name="decode_batch", op="decode", dtype="bf16", batch=64, len_min=200, len_max=8000, q_heads=32,
             kv_heads=8, head_dim=128, page=64),
        # two long sequences, where the keys have to be split over the whole card
        dict(name="decode_long", op="decode", dtype="fp16", batch=2, len_min=98000, len_max=131071, q_heads=64,
             kv_heads=8, head_dim=128, page=256),
        # a group of five query heads, a head dim and a page that are no powers of two
        dict(name="decode_odd", op="decode", dtype="fp16", batch=9, len_min=1, len_max=3001, q_heads=20, kv_heads=4,
             head_dim=80, page=24),
        # one new latent frame of a 720p clip against all 31 frames, every token seeing every key
        dict(name="chunk_frame", op="chunk", dtype="bf16", batch=1, new_min=880, new_max=880, len_min=27280,
             len_max=27280, q_heads=16, kv_heads=16, head_dim=128, page=880, frame=0),
        # ragged chunks of text-like sequences, each token seeing the keys up to its own
        dict(name="chunk_mixed", op="chunk", dtype="fp16", batch=5, new_min=1, new_max=700, len_min=700, len_max=6000,
             q_heads=20, kv_heads=4, head_dim=64, page=32, frame=1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, head_dim):
    """Rotated pairs of each axis: one or three axes, all channels or some."""
    pairs = head_dim // 2 if rng.random() < 0.7 else rng.randint(3, head_dim // 2)
    if rng.random() < 0.4:
        return str(pairs)
    t = max(1, pairs - 2 * (pairs // 3))
    h = (pairs - t) // 2
    return "%d,%d,%d" % (t, h, pairs - t - h)


def draw(rng):
    op = rng.choice(["rotary", "rotary_grad", "append", "decode", "decode", "chunk", "chunk"])
    head_dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 256])
    if op in ("rotary", "rotary_grad"):
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        batch, heads = rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 4, 5, 12, 16, 20, 32, 40])
        most = 55_000_000 * 2 // BYTES[dtype] // (batch * heads * head_dim)
        tokens = _log(rng, 1, max(1, min(30000, most)))
        sections = _sections(rng, head_dim)
        grid = "%d,1,1" % tokens
        if sections.count(","):
            w = min(tokens, rng.randint(1, 45))
            h = min(max(1, tokens // w), rng.randint(1, 30))
            t = max(1, tokens // (w * h))
            tokens, grid = t * h * w, "%d,%d,%d" % (t, h, w)
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, heads=heads, head_dim=head_dim, sections=sections,
                    grid=grid, interleaved=rng.random() < 0.5, start=_log(rng, 1, 1_000_000) - 1)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 12, 16])
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    while kv_heads * group > 64:
        group //= 2
    page = rng.choice([16, 16, 24, 32, 64, 64, 128, 256, 390, 880])
    case = dict(op=op, dtype=dtype, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page)
    if op == "append":
        most = 50_000_000 // ((group + 2) * kv_heads * head_dim)  # tokens of all sequences
        new_max = _log(rng, 1, min(8000, most))
        batch = rng.randint(1, max(1, min(32, most // new_max)))
        length = new_max + _log(rng, 1, 2000)
        return dict(case, batch=batch, new_min=rng.randint(1, new_max), new_max=new_max, len_min=new_max,
                    len_max=length, q_heads=rng.choice([0, kv_heads * group]), sections=_sections(rng, head_dim),
                    interleaved=rng.random() < 0.5)
    if op == "decode":
        most = 240_000_000 // (kv_heads * head_dim)  # keys of all sequences
        batch = _log(rng, 1, 96)
        length = _log(rng, 1, max(1, min(131072, most // batch)))
        return dict(case, batch=batch, len_min=rng.randint(1, length), len_max=length)
    batch = rng.choice([1, 1, 2, 3, 5])
    # the most query-key pairs: by the plain form's scores, and by the arithmetic of the largest listed case
    most = min(27280 * 16 * 880, 27280 * 880 * 2048 // head_dim) // (batch * case["q_heads"])
    new_max = _log(rng, 2, min(1760, math.isqrt(most)))
    length = _log(rng, new_max, min(40000, most // new_max))
    return dict(case, batch=batch, new_min=rng.randint(1, new_max), new_max=new_max, len_min=new_max, len_max=length,
                frame=rng.choice([0, 1, rng.randint(2, max(2, new_max))]))


# ---------------------------------------------------------------- inputs
def _between(case, what, n):
    """n sizes spread over [min, max], the largest among them: a case's own, whatever the seed."""
    lo, hi = case[what + "_min"], case[what + "_max"]
    g = torch.Generator().manual_seed(hi * 7 + lo + n)
    got = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    got[n // 2] = hi
    return got


def _sections_of(case):
    return tuple(int(s) for s in case["sections"].split(","))


def _grid(t, h, w, start, device):
    """Positions (time, height, width) of a clip's tokens in raster order, from time `start` on."""
    n = torch.arange(t * h * w, device=device)
    return torch.stack([n // (h * w) + start, n // w % h, n % w], -1).to(torch.int32)


def prepare(case, seed):
    d = torch.device("cuda")
    g = torch.Generator(device=d).manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=d, dtype=torch.float32).to(dtype)

    s = dict(case=case)
    if case["op"] in ("rotary", "rotary_grad"):
        s["x"] = normal(case["batch"], case["tokens"], case["heads"], case["head_dim"])
        t, h, w = (int(v) for v in case["grid"].split(","))
        pos = _grid(t, h, w, case["start"], d)
        s["positions"] = pos[:, :len(_sections_of(case))].contiguous()
        return s

    batch, page = case["batch"], case["page"]
    kv, hd = case["kv_heads"], case["head_dim"]
    lens = _between(case, "len", batch)
    new = [1] * batch if case["op"] == "decode" else _between(case, "new", batch)
    if case["op"] == "append" and case["len_min"] == case["len_max"]:
        lens = [case["len_max"]] * batch
    lens = [max(a, b) for a, b in zip(lens, new)]
    per = -(-max(lens) // page)  # pages of the longest sequence
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3  # and a few that belong to nobody
    order = torch.randperm(n_pages, generator=g, device=d, dtype=torch.int64).to(torch.int32)
    pages = torch.zeros(batch, per, dtype=torch.int32, device=d)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    total = sum(new)
    s.update(pages=pages, lengths=torch.tensor(lens, dtype=torch.int32, device=d),
             cu=torch.tensor([0] + [sum(new[:b + 1]) for b in range(batch)], dtype=torch.int32, device=d),
             most_keys=max(lens), most_new=max(new), lens=lens, new=new,
             k_cache=normal(n_pages, kv, page, hd), v_cache=normal(n_pages, kv, page, hd))
    if case["q_heads"]:
        # scores of a trained model spread wider than those of independent normal vectors
        s["q"] = (torch.randn(total, case["q_heads"], hd, generator=g, device=d) * 1.5).to(dtype)
    if case["op"] == "append":
        s["k"], s["v"] = normal(total, kv, hd), normal(total, kv, hd)
        place = torch.cat([torch.arange(n - m, n, device=d) for n, m in zip(lens, new)])
        if len(_sections_of(case)) == 1:
            s["positions"] = place[:, None].to(torch.int32)
        else:
            s["positions"] = torch.stack([place // 880, place // 40 % 22, place % 40], -1).to(torch.int32)
    if case["op"] == "chunk":
        s["ranges"] = None
        if case["frame"]:
            # a token sees the keys of its own frame of tokens and of those before it
            f = case["frame"]
            seen = [((torch.arange(n - m, n, device=d) // f + 1) * f).clamp(max=n) for n, m in zip(lens, new)]
            last = torch.cat(seen).to(torch.int32)
            s["ranges"] = torch.stack([torch.zeros_like(last), last], -1).contiguous()
    return s


# ------------------------------------------------------------ plain forms
def _frequencies(sections, device):
    """Radians per position of every rotated pair, and the axis whose position turns it."""
    freq = torch.cat([10000.0 ** (-torch.arange(n, device=device, dtype=torch.float64) / n) for n in sections])
    axis = torch.cat([torch.full((n,), a, device=device) for a, n in enumerate(sections)])
    return freq, axis


def _rotate(x, positions, sections, interleaved, sign=1.0):
    """x [..., tokens, heads, head_dim] turned by positions [tokens, axes], in 32 bits (angles in 64)."""
    freq, axis = _frequencies(sections, x.device)
    angle = positions.to(torch.float64)[:, axis] * freq
    cos, sin = angle.cos().float()[:, None, :], (sign * angle.sin()).float()[:, None, :]
    pairs = freq.numel()
    y = x.float()
    if interleaved:
        a, b = y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :pairs], y[..., pairs:2 * pairs]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., 2 * pairs:]], -1).to(x.dtype)


def _rows(cu, total):
    """The sequence of each row, and the row's place among its sequence's new tokens."""
    row = torch.arange(total, device=cu.device)
    seq = torch.bucketize(row, cu[1:].long(), right=True)
    return seq, row - cu.long()[seq]


def _gathered(cache, pages, keys):
    """The first `keys` entries of every sequence: [batch, keys, kv_heads, head_dim] in 32 bits."""
    page = cache.shape[2]
    at = torch.arange(keys, device=cache.device)
    return cache[pages[:, at // page].long(), :, (at % page)[None]].float()


def _attend(s):
    """q's tokens, padded to the longest chunk, against all keys, padded to the longest sequence."""
    q, cu, lengths = s["q"], s["cu"], s["lengths"]
    total, heads, hd = q.shape
    batch, kv = lengths.numel(), s["k_cache"].shape[1]
    k, v = _gathered(s["k_cache"], s["pages"], s["most_keys"]), _gathered(s["v_cache"], s["pages"], s["most_keys"])
    seq, place = _rows(cu, total)
    at = torch.arange(s["most_keys"], device=q.device)
    qp = torch.zeros(batch, s["most_new"], heads, hd, device=q.device)
    qp[seq, place] = q.float()
    first = torch.zeros(batch, s["most_new"], dtype=torch.int32, device=q.device)
    last = lengths[:, None].expand(batch, s["most_new"]).clone()
    if s.get("ranges") is not None:
        first[seq, place], last[seq, place] = s["ranges"][:, 0], s["ranges"][:, 1]
    last = torch.minimum(last, lengths[:, None])
    qg = qp.view(batch, s["most_new"], kv, heads // kv, hd).permute(0, 2, 3, 1, 4).reshape(batch, kv, -1, hd)
    scores = qg @ k.permute(0, 2, 3, 1)
    scores = scores.view(batch, kv, heads // kv, s["most_new"], -1) * (1.0 / math.sqrt(hd))
    hidden = (at < first[..., None]) | (at >= last[..., None])
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    total_p = p.sum(-1, keepdim=True)
    o = p.view(batch, kv, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3)
    o = o.view(batch, kv, heads // kv, s["most_new"], hd) / total_p.clamp(min=1e-38)
    lse = (top + total_p.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, s["most_new"], heads, hd)[seq, place]
    lse = lse.permute(0, 3, 1, 2).reshape(batch, s["most_new"], heads)[seq, place]
    return o.to(q.dtype), lse


def _append(s):
    sections, inter = _sections_of(s["case"]), s["case"]["interleaved"]
    k, v, cu = s["k"], s["v"], s["cu"]
    page = s["k_cache"].shape[2]
    seq, place = _rows(cu, k.shape[0])
    at = s["lengths"].long()[seq] - (cu[1:] - cu[:-1]).long()[seq] + place
    to = s["pages"].long()[seq, at // page]
    s["k_cache"][to, :, at % page] = _rotate(k, s["positions"], sections, inter)
    s["v_cache"][to, :, at % page] = v
    q = _rotate(s["q"], s["positions"], sections, inter) if "q" in s else None
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": q}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import video_vae_decoding_gb300 as wv

        if op == "rotary":
            return wv.rotary(s["x"], s["positions"], _sections_of(case), interleaved=case["interleaved"])
        if op == "rotary_grad":
            return wv.rotary_grad(s["x"], s["positions"], _sections_of(case), interleaved=case["interleaved"])
        if op == "append":
            q = wv.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"],
                             cu_tokens=None if case["new_max"] == 1 else s["cu"], positions=s["positions"],
                             sections=_sections_of(case), interleaved=case["interleaved"], q=s.get("q"))
            return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": q}
        if op == "decode":
            return wv.kv_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"])
        o, lse = wv.kv_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"], cu_tokens=s["cu"],
                                 ranges=s["ranges"], return_lse=True)
        return {"out": o, "lse": lse}
    if op == "rotary":
        return _rotate(s["x"], s["positions"], _sections_of(case), case["interleaved"])
    if op == "rotary_grad":
        return _rotate(s["x"], s["positions"], _sections_of(case), case["interleaved"], -1.0)
    if op == "append":
        return _append(s)
    o, lse = _attend(s)
    return o if op == "decode" else {"out": o, "lse": lse}


# ------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that a pass cannot do without, at the middle of the ranges of sizes."""
    size, hd = BYTES[case["dtype"]], case["head_dim"]
    if case["op"] in ("rotary", "rotary_grad"):
        n = case["batch"] * case["tokens"] * case["heads"] * hd
        return {"bytes": 2 * n * size + case["tokens"] * 4 * len(_sections_of(case)), "flops": 3 * n}
    batch = case["batch"]

    def mean(what):  # of `batch` sizes, the largest of the range among them
        lo, hi = case[what + "_min"], case[what + "_max"]
        return (hi + (batch - 1) * 0.5 * (lo + hi)) / batch

    new, keys = 1 if case["op"] == "decode" else mean("new"), mean("len")
    total = batch * new
    if case["op"] == "append":
        n = total * (2 * case["kv_heads"] + case["q_heads"]) * hd
        return {"bytes": 2 * n * size + total * 4 * (len(_sections_of(case)) + 1), "flops": 3 * total * (case["kv_heads"] + case["q_heads"]) * hd}
    seen = keys
    if case["op"] == "chunk" and case["frame"]:
        seen = max(1.0, keys - 0.5 * new + 0.5 * min(case["frame"], new))
    lse = 4 * total * case["q_heads"] if case["op"] == "chunk" else 0
    return {"bytes": 2 * batch * keys * case["kv_heads"] * hd * size + 2 * total * case["q_heads"] * hd * size + lse,
            "flops": 4 * total * seen * case["q_heads"] * hd}


# ------------------------------------------------------------------ exact
def _turned(x, positions, sections, interleaved, sign):
    """Channel pairs as complex numbers times exp(i angle), in 64 bits."""
    parts = []
    for axis, n in enumerate(sections):
        rate = torch.tensor([math.exp(-i * math.log(10000.0) / n) for i in range(n)], dtype=torch.float64, device=x.device)
        parts.append(positions[:, axis].double()[:, None] * rate[None])
    angle = sign * torch.cat(parts, 1)
    pairs = angle.shape[1]
    y = x.double()
    if interleaved:
        z = torch.view_as_complex(y[..., :2 * pairs].reshape(*y.shape[:-1], pairs, 2).contiguous())
    else:
        z = torch.complex(y[..., :pairs].contiguous(), y[..., pairs:2 * pairs].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    out = y.clone()
    if interleaved:
        out[..., 0:2 * pairs:2], out[..., 1:2 * pairs:2] = z.real, z.imag
    else:
        out[..., :pairs], out[..., pairs:2 * pairs] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "rotary_grad"):
        return _turned(s["x"], s["positions"], _sections_of(case), case["interleaved"], 1.0 if op == "rotary" else -1.0)
    cu, lens, new, page = s["cu"].tolist(), s["lens"], s["new"], case["page"]
    if op == "append":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k = _turned(s["k"], s["positions"], _sections_of(case), case["interleaved"], 1.0)
        for b in range(case["batch"]):
            place = torch.arange(lens[b] - new[b], lens[b], device=k.device)
            to, off = s["pages"][b][place // page].long(), place % page
            kc[to, :, off] = k[cu[b]:cu[b + 1]]
            vc[to, :, off] = s["v"][cu[b]:cu[b + 1]].double()
        q = _turned(s["q"], s["positions"], _sections_of(case), case["interleaved"], 1.0) if "q" in s else None
        return {"k_cache": kc, "v_cache": vc, "q": q}
    q, group = s["q"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b in range(case["batch"]):
        n = lens[b]
        held = s["pages"][b, :-(-n // page)].long()
        at = torch.arange(n, device=q.device)[None, None]
        for h in range(case["kv_heads"]):
            k = s["k_cache"][held, h].reshape(-1, case["head_dim"])[:n].double()
            v = s["v_cache"][held, h].reshape(-1, case["head_dim"])[:n].double()
            mine = q[cu[b]:cu[b + 1], h * group:(h + 1) * group].double()
            logit = torch.einsum("thd,nd->htn", mine, k) / math.sqrt(case["head_dim"])
            if s.get("ranges") is not None:
                r = s["ranges"][cu[b]:cu[b + 1]].long()
                logit = torch.where((at >= r[None, :, :1]) & (at < r[None, :, 1:]), logit, -math.inf)
            z = torch.logsumexp(logit, -1)
            out[cu[b]:cu[b + 1], h * group:(h + 1) * group] = torch.einsum("htn,nd->thd", (logit - z[..., None]).exp(), v)
            lse[cu[b]:cu[b + 1], h * group:(h + 1) * group] = z.T
    return out if op == "decode" else {"out": out, "lse": lse}

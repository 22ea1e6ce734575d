"""Token operators: rotary positions with several axes, the append to a paged
key-value cache, and the attention that reads it.

They are the steps of the streaming video model whose latents the decoder
turns into frames (wan_rotary, wan_kv_append, wan_kv_attention of
``include/wan_vae.h``).  One step of such a model on new tokens::

    q = kv_append(k, v, k_cache, v_cache, pages, lengths, cu_tokens=cu, positions=pos, sections=(22, 21, 21), q=q)
    out = kv_attention(q, k_cache, v_cache, pages, lengths, cu_tokens=cu)

Work goes to the current stream of the tensors' device, or to ``stream``;
results and workspaces made here are allocated on that stream.  No call
waits for the device.  Calls are not recorded by autograd: they refuse tensors
that require a gradient while gradients are enabled; ``rotary_grad`` is
``rotary``'s backward pass.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._lib import (WAN_BF16, WAN_F16, WAN_F32, WanKvBatch, WanKvCache, WanRotation, check, load)

__all__ = ["Rotation", "rotary", "rotary_grad", "kv_append", "kv_attention", "kv_check", "kv_status"]

_CODES = {torch.float32: WAN_F32, torch.bfloat16: WAN_BF16, torch.float16: WAN_F16}
_I64x3 = ctypes.c_int64 * 3


class Rotation:
    """Which channel pairs turn, by which axis and how fast.

    sections: pairs of each axis, e.g. (22, 21, 21) for time, height and width
    at a head dim of 128; pair i of an axis of n turns theta ** (-i / n)
    radians per position.  freq: instead of theta, the radians per position
    of every pair (all axes in order; host values).  interleaved: pairs are
    neighbouring channels (2j, 2j + 1); otherwise channels (j, j + pairs)."""

    def __init__(self, sections, theta: float = 10000.0, interleaved: bool = True, freq=None):
        sections = tuple(int(n) for n in sections)
        if not sections or min(sections) < 0 or sum(sections) < 1:
            raise ValueError(f"sections must be pair counts, not {sections}")
        if not (theta > 0 and math.isfinite(theta)):
            raise ValueError(f"theta must be positive, not {theta}")
        if freq is None:
            freq = [theta ** (-i / n) for n in sections for i in range(n)]
        else:
            freq = [float(f) for f in freq]
            if len(freq) != sum(sections):
                raise ValueError(f"{len(freq)} frequencies for {sum(sections)} pairs")
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
        self.sections, self.axes, self.interleaved = sections, len(sections), bool(interleaved)
        self.pairs = len(freq)
        self._freq = (ctypes.c_double * self.pairs)(*freq)
        self._axis = (ctypes.c_int32 * self.pairs)(*axis)
        self._c = WanRotation(self.pairs, self.axes, int(self.interleaved), self._freq, self._axis)
        self._ref = ctypes.byref(self._c)


@functools.lru_cache(maxsize=64)
def _made(sections, theta, interleaved) -> Rotation:
    return Rotation(sections, theta, interleaved)


def _rotation(sections, theta, interleaved) -> Rotation:
    return sections if isinstance(sections, Rotation) else _made(tuple(sections), theta, interleaved)


def _refuse_grad(*tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError("the token operators are not recorded by autograd: detach the tensors (rotary_grad is "
                         "rotary's backward pass)")


def _on(t: torch.Tensor, device: torch.device, name: str, dtypes=None, dim: int = 0):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if dim and t.dim() != dim:
        raise ValueError(f"{name} has {t.dim()} dimensions, not {dim}")


def _rows_of(t: torch.Tensor, name: str):
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")


class _Launch:
    """The device and stream of a call: current while it is entered (allocations belong to the stream)."""

    __slots__ = ("ptr", "_guards")

    def __init__(self, device: torch.device, stream):
        if device.type != "cuda":
            raise ValueError(f"the tensors must be CUDA tensors, not on {device}")
        self._guards = []
        if device.index != torch.cuda.current_device():
            self._guards.append(torch.cuda.device(device))
        if stream is None:
            self.ptr = torch.cuda.current_stream(device).cuda_stream
        else:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self.ptr = stream.cuda_stream
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()
        return self.ptr

    def __exit__(self, *exc):
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


def _turn(x, positions, sections, theta, interleaved, out, stream, inverse):
    if x.dtype not in _CODES:
        raise ValueError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    if x.dim() not in (3, 4):
        raise ValueError(f"x must be [tokens, heads, head_dim] or [batch, tokens, heads, head_dim], not {tuple(x.shape)}")
    _refuse_grad(x, out)
    rot = _rotation(sections, theta, interleaved)
    B = x.shape[0] if x.dim() == 4 else 1
    T, H, D = x.shape[-3:]
    dev = x.device
    _on(positions, dev, "positions", (torch.int32, torch.int64))
    shape = tuple(positions.shape)
    shared = shape == (T, rot.axes)
    if not shared and shape != (B, T, rot.axes):
        raise ValueError(f"positions must be [{T}, {rot.axes}] or [{B}, {T}, {rot.axes}], not {shape}")
    if not positions.is_contiguous():
        raise ValueError("positions must be contiguous")
    _rows_of(x, "x")
    with _Launch(dev, stream) as ptr:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        else:
            _on(out, dev, "out", (x.dtype,), x.dim())
            if out.shape != x.shape:
                raise ValueError(f"out must be {tuple(x.shape)}, not {tuple(out.shape)}")
            _rows_of(out, "out")
        xs, os = x.stride(), out.stride()
        if x.dim() == 3:
            xs, os = (0, *xs), (0, *os)
        check(load().wan_rotary(x.data_ptr(), _I64x3(*xs[:3]), out.data_ptr(), _I64x3(*os[:3]), _CODES[x.dtype], B, T, H,
                                D, positions.data_ptr(), positions.dtype == torch.int64,
                                0 if shared else T * rot.axes, rot._ref, inverse, ptr))
    return out


def rotary(x: torch.Tensor, positions: torch.Tensor, sections, theta: float = 10000.0, interleaved: bool = True,
           out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """x [..., tokens, heads, head_dim] (one batch dimension or none; any
    strides with contiguous channels) turned by positions [tokens, axes] (or
    [batch, tokens, axes]; int32 or int64): see Rotation for sections (or pass
    a Rotation).  Computed in fp32 and rounded once.  out may be x."""
    return _turn(x, positions, sections, theta, interleaved, out, stream, 0)


def rotary_grad(dy: torch.Tensor, positions: torch.Tensor, sections, theta: float = 10000.0, interleaved: bool = True,
                out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Gradient of rotary with respect to x, given that of its result: dy turned
    by the opposite angles."""
    return _turn(dy, positions, sections, theta, interleaved, out, stream, 1)


def _cache(k_cache, v_cache) -> WanKvCache:
    dev = k_cache.device
    _on(k_cache, dev, "k_cache", (torch.bfloat16, torch.float16), 4)
    _on(v_cache, dev, "v_cache", (k_cache.dtype,), 4)
    if k_cache.shape != v_cache.shape:
        raise ValueError(f"k_cache is {tuple(k_cache.shape)}, v_cache {tuple(v_cache.shape)}")
    _rows_of(k_cache, "k_cache")
    _rows_of(v_cache, "v_cache")
    pages, heads, size, D = k_cache.shape
    ks, vs = k_cache.stride(), v_cache.stride()
    return WanKvCache(k_cache.data_ptr(), v_cache.data_ptr(), _CODES[k_cache.dtype], heads, size, D, pages,
                      ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])


_INT32 = (torch.int32,)


def _batch(dev, pages, lengths, cu_tokens, tokens, status) -> WanKvBatch:
    _on(pages, dev, "pages", _INT32, 2)
    _on(lengths, dev, "lengths", _INT32, 1)
    B = lengths.shape[0]
    if pages.shape[0] != B:
        raise ValueError(f"pages has {pages.shape[0]} rows for {B} sequences")
    if pages.shape[1] > 1 and pages.stride(1) != 1:
        raise ValueError("the rows of pages must be contiguous")
    if B > 1 and lengths.stride(0) != 1:
        raise ValueError("lengths must be contiguous")
    cu = None
    if cu_tokens is not None:
        _on(cu_tokens, dev, "cu_tokens", _INT32, 1)
        if cu_tokens.shape[0] != B + 1 or cu_tokens.stride(0) != 1:
            raise ValueError(f"cu_tokens must hold {B + 1} contiguous values")
        cu = cu_tokens.data_ptr()
    if status is not None:
        _on(status, dev, "status", _INT32)
        if status.numel() != 1:
            raise ValueError("status must hold one value")
        status = status.data_ptr()
    return WanKvBatch(pages.data_ptr(), pages.stride(0), pages.shape[1], B, lengths.data_ptr(), cu, tokens, status)


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor,
              lengths: torch.Tensor, cu_tokens: torch.Tensor = None, positions: torch.Tensor = None, sections=None,
              theta: float = 10000.0, interleaved: bool = True, q: torch.Tensor = None, q_out: torch.Tensor = None,
              status: torch.Tensor = None, stream=None):
    """Writes new tokens' keys (turned as rotary turns them; sections None: as
    they are) and values into the caches, in place, and returns q turned the
    same way (None without q).

    k, v: [tokens, kv_heads, head_dim]; q: [tokens, q_heads, head_dim].  Caches:
    [pages, kv_heads, page_size, head_dim], bfloat16 or float16, strides that are
    multiples of 8 elements (so a [pages, page_size, kv_heads, head_dim] cache is
    passed as its transpose(1, 2)).  pages [sequences, n] int32: the page that
    holds keys i * page_size onwards of a sequence; lengths [sequences] int32:
    its keys with the new ones; cu_tokens [sequences + 1] int32: its token rows
    (None: one each).  positions [tokens, axes].  q_out: where the turned q goes
    (q itself is allowed; new memory by default, where rows behind the last
    sequence stay uninitialised).  status: an int32 tensor of one value that
    takes a code if the tables name something that is not there (kv_status)."""
    _refuse_grad(k, v, q, k_cache, v_cache, q_out)
    c = _cache(k_cache, v_cache)
    dev, dt = k_cache.device, (k_cache.dtype,)
    _on(k, dev, "k", dt, 3)
    _on(v, dev, "v", dt, 3)
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1] != c.heads or k.shape[2] != c.head_dim:
        raise ValueError(f"k is {tuple(k.shape)} and v {tuple(v.shape)}, the cache's tokens [n, {c.heads}, {c.head_dim}]")
    _rows_of(k, "k")
    _rows_of(v, "v")
    b = _batch(dev, pages, lengths, cu_tokens, T, status)
    rot, pos = None, None
    if sections is not None:
        rot = _rotation(sections, theta, interleaved)
        if positions is None:
            raise ValueError("sections need positions")
        _on(positions, dev, "positions", (torch.int32, torch.int64), 2)
        if tuple(positions.shape) != (T, rot.axes) or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous [{T}, {rot.axes}], not {tuple(positions.shape)}")
        pos = positions.data_ptr()
    elif positions is not None:
        raise ValueError("positions need sections")
    if q is None and q_out is not None:
        raise ValueError("q_out needs q")
    ks, vs = k.stride(), v.stride()
    with _Launch(dev, stream) as ptr:
        if q is None:
            qa = (None, 0, 0, 0, None, 0, 0)
        else:
            _on(q, dev, "q", dt, 3)
            if q.shape[0] != T or q.shape[2] != c.head_dim:
                raise ValueError(f"q is {tuple(q.shape)}, not [{T}, heads, {c.head_dim}]")
            _rows_of(q, "q")
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            else:
                _on(q_out, dev, "q_out", dt, 3)
                if q_out.shape != q.shape:
                    raise ValueError(f"q_out is {tuple(q_out.shape)}, not {tuple(q.shape)}")
                _rows_of(q_out, "q_out")
            qs, os = q.stride(), q_out.stride()
            # an empty tensor has no address, but a call with q is one all the same
            qa = (q.data_ptr() or None, q.shape[1], qs[0], qs[1], q_out.data_ptr() or None, os[0], os[1])
        check(load().wan_kv_append(ctypes.byref(c), ctypes.byref(b), k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0],
                                   vs[1], *qa, rot._ref if rot else None, pos,
                                   pos is not None and positions.dtype == torch.int64, ptr))
    return q_out


def kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor,
                 lengths: torch.Tensor, cu_tokens: torch.Tensor = None, ranges: torch.Tensor = None,
                 scale: float = None, out: torch.Tensor = None, return_lse: bool = False,
                 status: torch.Tensor = None, stream=None):
    """softmax(scale * q k^T) v of each token and query head over the keys of its
    sequence; heads h * g .. h * g + g - 1 of q read key head h.

    q [tokens, q_heads, head_dim]; caches, pages, lengths, cu_tokens, status as
    in kv_append.  ranges [tokens, 2] int32: the first key a token sees and one
    past its last (None: all); a token that sees nothing gets zeros.  scale:
    1 / sqrt(head_dim) by default.  out: like q (new memory by default, where
    rows behind the last sequence stay uninitialised).  return_lse: also the
    fp32 logarithms of the sums, [tokens, q_heads]."""
    _refuse_grad(q, k_cache, v_cache, out)
    c = _cache(k_cache, v_cache)
    dev, dt = k_cache.device, (k_cache.dtype,)
    _on(q, dev, "q", dt, 3)
    T, H, D = q.shape
    if D != c.head_dim:
        raise ValueError(f"q is {tuple(q.shape)}, the cache's head dim {c.head_dim}")
    _rows_of(q, "q")
    b = _batch(dev, pages, lengths, cu_tokens, T, status)
    rp = None
    if ranges is not None:
        _on(ranges, dev, "ranges", _INT32, 2)
        if tuple(ranges.shape) != (T, 2) or not ranges.is_contiguous():
            raise ValueError(f"ranges must be contiguous [{T}, 2], not {tuple(ranges.shape)}")
        rp = ranges.data_ptr()
    lib = load()
    cp, bp = ctypes.byref(c), ctypes.byref(b)
    with _Launch(dev, stream) as ptr:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        else:
            _on(out, dev, "out", dt, 3)
            if out.shape != q.shape:
                raise ValueError(f"out is {tuple(out.shape)}, not {tuple(q.shape)}")
            _rows_of(out, "out")
        lse = torch.empty((T, H), dtype=torch.float32, device=dev) if return_lse else None
        n = lib.wan_kv_attention_workspace(cp, bp, H)
        if n < 0:
            check(lib.wan_kv_attention(cp, bp, None, H, 0, 0, None, 0.0, None, 0, 0, None, None, 0, ptr))
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        qs, os = q.stride(), out.stride()
        check(lib.wan_kv_attention(cp, bp, q.data_ptr(), H, qs[0], qs[1], rp, D ** -0.5 if scale is None else scale,
                                   out.data_ptr(), os[0], os[1], None if lse is None else lse.data_ptr(),
                                   ws.data_ptr(), n, ptr))
    return (out, lse) if return_lse else out


def kv_check(pages: torch.Tensor, lengths: torch.Tensor, page_size: int, n_pages: int, cu_tokens: torch.Tensor = None,
             tokens: int = None, append: bool = False):
    """Checks host (CPU int32) tables as kv_append (append=True) and kv_attention
    would read them; raises WanError naming the sequence at fault."""
    cpu = torch.device("cpu")
    if tokens is None:
        tokens = int(cu_tokens[-1]) if cu_tokens is not None else lengths.shape[0]
    b = _batch(cpu, pages, lengths, cu_tokens, tokens, None)
    check(load().wan_kv_check(ctypes.byref(b), page_size, n_pages, append))


def kv_status(status: torch.Tensor, stream=None):
    """Waits for the stream, then raises WanError if a call left a code in
    `status` (which is cleared)."""
    _on(status, status.device, "status", _INT32)
    with _Launch(status.device, stream) as ptr:
        check(load().wan_kv_status(status.data_ptr(), ptr))

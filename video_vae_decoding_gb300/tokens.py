"""Token operators: rotary positions with several axes, the append to a paged
key-value cache, and the attention that reads it.

They are the steps of the streaming video model whose latents the decoder
turns into frames (wan_rotary, wan_kv_append, wan_kv_attention of
``include/wan_vae.h``).  One step of such a model on new tokens::

    q = kv_append(k, v, k_cache, v_cache, pages, lengths, cu_tokens=cu, positions=pos, sections=(22, 21, 21), q=q)
    out = kv_attention(q, k_cache, v_cache, pages, lengths, cu_tokens=cu)

Work goes to the current stream of the tensors' device, or to ``stream``
(which has to wait for what makes the tensors; they may be dropped after the
call); results and workspaces made here are allocated on that stream.  No call
waits for the device.  Calls are not recorded by autograd: they refuse tensors
that require a gradient while gradients are enabled, and dual tensors;
``rotary_grad`` is ``rotary``'s backward pass.
"""

from __future__ import annotations

import ctypes
import functools
import math
import struct
import warnings

import torch
from torch.autograd import forward_ad

from ._lib import WAN_BF16, WAN_F16, WAN_F32, WanRotation, check, load

__all__ = ["Rotation", "rotary", "rotary_grad", "kv_append", "kv_attention", "kv_check", "kv_status"]

_CODES = {torch.float32: WAN_F32, torch.bfloat16: WAN_BF16, torch.float16: WAN_F16}
_HALVES = (torch.bfloat16, torch.float16)
_INT32 = (torch.int32,)
# The C structs as bytes: packing costs a quarter of building a ctypes Structure
# (the launch path's host time is what a small call costs).
_pack3 = struct.Struct("@qqq").pack             # const int64_t[3]
_pack_cache = struct.Struct("@PPiiiiqqqqqqq").pack  # wan_kv_cache
_pack_batch = struct.Struct("@PqiiPPiP").pack       # wan_kv_batch


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
        self._addr = ctypes.addressof(self._c)


@functools.lru_cache(maxsize=64)
def _made(sections, theta, interleaved) -> Rotation:
    return Rotation(sections, theta, interleaved)


def _rotation(sections, theta, interleaved) -> Rotation:
    return sections if isinstance(sections, Rotation) else _made(tuple(sections), theta, interleaved)


def _refuse_grad(*tensors):
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError("the token operators are not recorded by autograd: detach the tensors (rotary_grad is "
                         "rotary's backward pass)")
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError("the token operators are not recorded by autograd: a dual tensor's tangent would be lost")


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


def _int32(n: int, what: str):
    """Refuses a size that the library's 32-bit argument cannot hold (ctypes would cut it)."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{n} {what}: more than 32 bits hold")


def _written(*tensors):
    """Counts the version of tensors that a call wrote to, for autograd's check of what it saved."""
    for t in tensors:
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)


class _Guard:
    """Makes the tensors' device and the caller's stream current (allocations then belong to that stream).  The memory of
    `tensors` is not given to other work before the stream is done with the call, even if the caller drops them."""

    __slots__ = ("_guards", "_stream", "_tensors")

    def __init__(self, device: torch.device, stream, *tensors):
        self._guards = [torch.cuda.device(device)]
        self._stream, self._tensors = stream, tensors
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
            self._guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self._guards:
            g.__enter__()

    def __exit__(self, *exc):
        if self._stream is not None and exc[0] is None:
            for t in self._tensors:
                if t is not None:
                    t.record_stream(self._stream)
        for g in reversed(self._guards):
            g.__exit__(*exc)
        return False


def _elsewhere(device: torch.device, stream) -> bool:
    """Whether a call needs a _Guard; refuses tensors that are not on a GPU."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be CUDA tensors, not on {device}")
    return stream is not None or device.index != torch.cuda.current_device()


# The calling stream's handle without building a torch.cuda.Stream (2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Absent:
    """In the place of _tokens where it is not there: takes no call, so all are marshalled in Python."""

    @staticmethod
    def _none(*args):
        return None

    rotary = append = attention = _none


def _short_way():
    """The C++ marshalling of ordinary calls (_tokens), made at the first call: its functions return None for a call
    that they do not take."""
    global _short
    from . import build

    lib = load()
    try:
        if not build.binding_fits():
            raise ImportError("it is missing, or made for another Python or torch")
        from . import _tokens

        _tokens.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.wan_rotary, lib.wan_kv_append, lib.wan_kv_attention, lib.wan_kv_attention_workspace)))
        _short = _tokens
    except ImportError as e:
        warnings.warn(f"the token operators are marshalled in Python, which takes three times the host's time: _tokens.so "
                      f"cannot be used ({e}); build.build() makes it", RuntimeWarning)
        _short = _Absent
    return _short


_short = None


def _turn(x, positions, sections, theta, interleaved, out, stream, inverse):
    code = _CODES.get(x.dtype)
    if code is None:
        raise ValueError(f"x must be float32, bfloat16 or float16, not {x.dtype}")
    shape, xs = x.shape, x.stride()
    if len(shape) == 4:
        B, T, H, D = shape
    elif len(shape) == 3:
        B, (T, H, D), xs = 1, shape, (0, *xs)
    else:
        raise ValueError(f"x must be [tokens, heads, head_dim] or [batch, tokens, heads, head_dim], not {tuple(shape)}")
    for n, what in (B, "sequences"), (T, "tokens"), (H, "heads"), (D, "channels"):
        _int32(n, what)
    _refuse_grad(x, out)
    rot = _rotation(sections, theta, interleaved)
    dev = x.device
    _on(positions, dev, "positions", (torch.int32, torch.int64))
    pshape = positions.shape
    shared = pshape == (T, rot.axes)
    if not shared and pshape != (B, T, rot.axes):
        raise ValueError(f"positions must be [{T}, {rot.axes}] or [{B}, {T}, {rot.axes}], not {tuple(pshape)}")
    if not positions.is_contiguous():
        raise ValueError("positions must be contiguous")
    if xs[3] != 1:
        _rows_of(x, "x")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream, x, positions, out):
            return _turn(x, positions, rot, theta, interleaved, out, None, inverse)
    given = out is not None
    if not given:
        out = torch.empty(shape, dtype=x.dtype, device=dev)
        os = (T * H * D, H * D, D)
    else:
        _on(out, dev, "out", (x.dtype,), len(shape))
        if out.shape != shape:
            raise ValueError(f"out must be {tuple(shape)}, not {tuple(out.shape)}")
        _rows_of(out, "out")
        os = out.stride()[:-1]
        if len(os) == 2:
            os = (0, *os)
    status = load().wan_rotary(x.data_ptr(), _pack3(*xs[:3]), out.data_ptr(), _pack3(*os), code, B, T, H, D,
                               positions.data_ptr(), positions.dtype is torch.int64, 0 if shared else T * rot.axes,
                               rot._ref, inverse, _raw_stream(dev.index))
    if status:
        check(status)
    if given:
        _written(out)
    return out


def rotary(x: torch.Tensor, positions: torch.Tensor, sections, theta: float = 10000.0, interleaved: bool = True,
           out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """x [..., tokens, heads, head_dim] (one batch dimension or none; any
    strides with contiguous channels) turned by positions [tokens, axes] (or
    [batch, tokens, axes]; int32 or int64): see Rotation for sections (or pass
    a Rotation).  Computed in fp32 and rounded once.  out may be x."""
    short = _short or _short_way()
    if stream is None:
        rot = _rotation(sections, theta, interleaved)
        got = short.rotary(x, positions, rot._addr, rot.axes, out, 0)
        if got is not None:
            return got
    return _turn(x, positions, sections, theta, interleaved, out, stream, 0)


def rotary_grad(dy: torch.Tensor, positions: torch.Tensor, sections, theta: float = 10000.0, interleaved: bool = True,
                out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Gradient of rotary with respect to x, given that of its result: dy turned
    by the opposite angles."""
    short = _short or _short_way()
    if stream is None:
        rot = _rotation(sections, theta, interleaved)
        got = short.rotary(dy, positions, rot._addr, rot.axes, out, 1)
        if got is not None:
            return got
    return _turn(dy, positions, sections, theta, interleaved, out, stream, 1)


def _cache(k_cache, v_cache, dev):
    """wan_kv_cache of the two tensors (packed), and their common shape."""
    dt = k_cache.dtype
    if dt not in _HALVES:
        _on(k_cache, dev, "k_cache", _HALVES, 4)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.dtype is not dt or v_cache.device != dev:
        _on(k_cache, dev, "k_cache", _HALVES, 4)
        _on(v_cache, dev, "v_cache", (dt,), 4)
    if v_cache.shape != shape:
        raise ValueError(f"k_cache is {tuple(shape)}, v_cache {tuple(v_cache.shape)}")
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if k3 != 1 or v3 != 1:
        _rows_of(k_cache, "k_cache")
        _rows_of(v_cache, "v_cache")
    pages, heads, size, D = shape
    for n, what in (heads, "heads"), (size, "keys as page size"), (D, "channels"):
        _int32(n, what)
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), _CODES[dt], heads, size, D, pages, k0, k1, k2, v0, v1,
                       v2), heads, size, D


def _batch(dev, pages, lengths, cu_tokens, tokens, status):
    """wan_kv_batch of the tables (packed), and the number of sequences."""
    i32 = torch.int32
    if pages.dtype is not i32 or lengths.dtype is not i32 or pages.device != dev or lengths.device != dev or \
            pages.dim() != 2 or lengths.dim() != 1:
        _on(pages, dev, "pages", _INT32, 2)
        _on(lengths, dev, "lengths", _INT32, 1)
    B, n = pages.shape
    for m, what in (B, "sequences"), (n, "pages a sequence"), (tokens, "tokens"):
        _int32(m, what)
    if lengths.shape[0] != B:
        raise ValueError(f"pages has {B} rows for {lengths.shape[0]} sequences")
    p0, p1 = pages.stride()
    if p1 != 1 and n > 1:
        raise ValueError("the rows of pages must be contiguous")
    if B > 1 and lengths.stride(0) != 1:
        raise ValueError("lengths must be contiguous")
    cu = st = 0
    if cu_tokens is not None:
        _on(cu_tokens, dev, "cu_tokens", _INT32, 1)
        if cu_tokens.shape[0] != B + 1 or cu_tokens.stride(0) != 1:
            raise ValueError(f"cu_tokens must hold {B + 1} contiguous values")
        cu = cu_tokens.data_ptr()
    if status is not None:
        _on(status, dev, "status", _INT32)
        if status.numel() != 1:
            raise ValueError("status must hold one value")
        st = status.data_ptr()
    return _pack_batch(pages.data_ptr(), p0, n, B, lengths.data_ptr(), cu, tokens, st), B


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
    short = _short or _short_way()
    if stream is None:
        rot = None if sections is None else _rotation(sections, theta, interleaved)
        got = short.append(k, v, k_cache, v_cache, pages, lengths, cu_tokens, positions, rot._addr if rot else 0,
                           rot.axes if rot else 0, q, q_out, status)
        if got is not None:
            return None if got is True else got
    _refuse_grad(k, v, q, k_cache, v_cache, q_out)
    dev = k_cache.device
    c, heads, size, D = _cache(k_cache, v_cache, dev)
    dt = k_cache.dtype
    if k.dtype is not dt or v.dtype is not dt or k.device != dev or v.device != dev or k.dim() != 3:
        _on(k, dev, "k", (dt,), 3)
        _on(v, dev, "v", (dt,), 3)
    shape = k.shape
    T = shape[0]
    if v.shape != shape or shape[1] != heads or shape[2] != D:
        raise ValueError(f"k is {tuple(shape)} and v {tuple(v.shape)}, the cache's tokens [n, {heads}, {D}]")
    ks, vs = k.stride(), v.stride()
    if ks[2] != 1 or vs[2] != 1:
        _rows_of(k, "k")
        _rows_of(v, "v")
    b, _ = _batch(dev, pages, lengths, cu_tokens, T, status)
    rot = pos = None
    pos64 = False
    if sections is not None:
        rot = _rotation(sections, theta, interleaved)
        if positions is None:
            raise ValueError("sections need positions")
        _on(positions, dev, "positions", (torch.int32, torch.int64), 2)
        if positions.shape != (T, rot.axes) or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous [{T}, {rot.axes}], not {tuple(positions.shape)}")
        pos, pos64, rot = positions.data_ptr(), positions.dtype is torch.int64, rot._ref
    elif positions is not None:
        raise ValueError("positions need sections")
    if _elsewhere(dev, stream):
        with _Guard(dev, stream, k, v, k_cache, v_cache, pages, lengths, cu_tokens, positions, q, q_out, status):
            return kv_append(k, v, k_cache, v_cache, pages, lengths, cu_tokens, positions, sections, theta, interleaved, q,
                             q_out, status)
    given = q_out is not None
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs q")
        qa = (None, 0, 0, 0, None, 0, 0)
    else:
        _on(q, dev, "q", (dt,), 3)
        qshape, qs = q.shape, q.stride()
        _int32(qshape[1], "heads")
        if qshape[0] != T or qshape[2] != D:
            raise ValueError(f"q is {tuple(qshape)}, not [{T}, heads, {D}]")
        if qs[2] != 1:
            _rows_of(q, "q")
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dt, device=dev)
            os = (qshape[1] * D, D)
        else:
            _on(q_out, dev, "q_out", (dt,), 3)
            if q_out.shape != qshape:
                raise ValueError(f"q_out is {tuple(q_out.shape)}, not {tuple(qshape)}")
            _rows_of(q_out, "q_out")
            os = q_out.stride()
        # an empty tensor has no address, but a call with q is one all the same
        qa = (q.data_ptr() or None, qshape[1], qs[0], qs[1], q_out.data_ptr() or None, os[0], os[1])
    status = load().wan_kv_append(c, b, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], *qa, rot, pos, pos64,
                                  _raw_stream(dev.index))
    if status:
        check(status)
    _written(k_cache, v_cache, *([q_out] if given else []))
    return q_out


@functools.lru_cache(maxsize=1024)
def _workspace(dtype, heads, size, D, columns, B, T, q_heads, device_index) -> int:
    """Bytes of workspace of a call of these sizes (wan_kv_attention_workspace), whatever the addresses."""
    step = 8 * -(-D // 8)
    c = _pack_cache(16, 16, dtype, heads, size, D, 1, step, step, step, step, step, step)
    n = load().wan_kv_attention_workspace(c, _pack_batch(16, columns, columns, B, 16, 16, T, 0), q_heads)
    if n < 0:
        msg = load().wan_vae_last_error()
        raise ValueError(msg.decode())
    return n


def kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, pages: torch.Tensor,
                 lengths: torch.Tensor, cu_tokens: torch.Tensor = None, ranges: torch.Tensor = None,
                 scale: float = None, out: torch.Tensor = None, return_lse: bool = False,
                 status: torch.Tensor = None, stream=None):
    """softmax(scale * q k^T) v of each token and query head over the keys of its
    sequence; heads h * g .. h * g + g - 1 of q read key head h.

    q [tokens, q_heads, head_dim]; caches, pages, lengths, cu_tokens, status as
    in kv_append.  ranges [tokens, 2] int32: the first key a token sees and one
    past its last (None: all); a token that sees nothing gets zeros.  scale:
    1 / sqrt(head_dim) by default.  out: like q, or q itself (new memory by
    default, where rows behind the last sequence stay uninitialised).  return_lse: also the
    fp32 logarithms of the sums, [tokens, q_heads].  Rows of NaN throughout
    mean that a wait inside the kernels ran out (status then holds a code).

    Calls of few rows (tokens * q_heads / kv_heads; under 64 a sequence on
    average, or a small call) give results off by their own rounding alone; the
    tensor-core kernel for more rows rounds the weights to 16 bits, so its results
    are off by 1.2 to 1.4 times that.  It takes page sizes that are multiples of 8
    or above 64, and caches whose k and v order their dimensions alike; with
    others, calls of many rows take ten times as long."""
    short = _short or _short_way()
    if stream is None:
        got = short.attention(q, k_cache, v_cache, pages, lengths, cu_tokens, ranges, scale, out, return_lse, status)
        if got is not None:
            return got
    _refuse_grad(q, k_cache, v_cache, out)
    dev = k_cache.device
    c, heads, size, D = _cache(k_cache, v_cache, dev)
    dt = k_cache.dtype
    shape, qs = q.shape, q.stride()
    if q.dtype is not dt or q.device != dev or len(shape) != 3:
        _on(q, dev, "q", (dt,), 3)
    T, H, qD = shape
    _int32(H, "heads")
    if qD != D:
        raise ValueError(f"q is {tuple(shape)}, the cache's head dim {D}")
    if qs[2] != 1:
        _rows_of(q, "q")
    b, B = _batch(dev, pages, lengths, cu_tokens, T, status)
    rp = None
    if ranges is not None:
        _on(ranges, dev, "ranges", _INT32, 2)
        if ranges.shape != (T, 2) or not ranges.is_contiguous():
            raise ValueError(f"ranges must be contiguous [{T}, 2], not {tuple(ranges.shape)}")
        rp = ranges.data_ptr()
    if _elsewhere(dev, stream):
        with _Guard(dev, stream, q, k_cache, v_cache, pages, lengths, cu_tokens, ranges, out, status):
            return kv_attention(q, k_cache, v_cache, pages, lengths, cu_tokens, ranges, scale, out, return_lse, status)
    given = out is not None
    if not given:
        out = torch.empty(shape, dtype=dt, device=dev)
        os = (H * D, D)
    else:
        _on(out, dev, "out", (dt,), 3)
        if out.shape != shape:
            raise ValueError(f"out is {tuple(out.shape)}, not {tuple(shape)}")
        _rows_of(out, "out")
        os = out.stride()
    n = _workspace(_CODES[dt], heads, size, D, pages.shape[1], B, T, H, dev.index)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    lse, lp = None, None
    if return_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
        lp = lse.data_ptr()
    status = load().wan_kv_attention(c, b, q.data_ptr(), H, qs[0], qs[1], rp, D ** -0.5 if scale is None else scale,
                                     out.data_ptr(), os[0], os[1], lp, ws.data_ptr(), n, _raw_stream(dev.index))
    if status:
        check(status)
    if given:
        _written(out)
    return (out, lse) if return_lse else out


def kv_check(pages: torch.Tensor, lengths: torch.Tensor, page_size: int, n_pages: int, cu_tokens: torch.Tensor = None,
             tokens: int = None, append: bool = False):
    """Checks host (CPU int32) tables as kv_append (append=True) and kv_attention
    would read them; raises WanError naming the sequence at fault."""
    cpu = torch.device("cpu")
    if tokens is None:
        tokens = int(cu_tokens[-1]) if cu_tokens is not None else lengths.shape[0]
    _int32(page_size, "keys as page size")
    b, _ = _batch(cpu, pages, lengths, cu_tokens, tokens, None)
    check(load().wan_kv_check(b, page_size, n_pages, append))


def kv_status(status: torch.Tensor, stream=None):
    """Waits for the stream, then raises WanError if a call left a code in
    `status` (which is cleared)."""
    dev = status.device
    _on(status, dev, "status", _INT32)
    if _elsewhere(dev, stream):
        with _Guard(dev, stream):
            return kv_status(status)
    check(load().wan_kv_status(status.data_ptr(), _raw_stream(dev.index)))

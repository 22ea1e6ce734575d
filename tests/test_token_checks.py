"""The token operators' refusals, and the host check of page tables (no GPU:
every call here returns before any CUDA work)."""

import ctypes

import pytest
import torch

from video_vae_decoding_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    from video_vae_decoding_gb300 import build
    build.build()
    return _lib.load()


vp = ctypes.c_void_p
I3 = ctypes.c_int64 * 3


def _rotation(pairs=4, axes=1, interleaved=1, freq=None, axis=None):
    f = (ctypes.c_double * max(1, pairs))(*(freq or [1.0] * pairs))
    a = (ctypes.c_int32 * max(1, pairs))(*(axis or [0] * pairs))
    r = _lib.WanRotation(pairs, axes, interleaved, f, a)
    r.keep = (f, a)
    return r


def _rotary(lib, rot=None, dtype=1, B=1, T=2, H=3, D=8, x=4096, out=8192, pos=64, xs=(48, 24, 8), os=(48, 24, 8),
            pos64=0, pb=0):
    r = ctypes.byref(rot or _rotation())
    return lib.wan_rotary(vp(x), I3(*xs), vp(out), I3(*os), dtype, B, T, H, D, vp(pos), pos64, pb, r, 0, None)


def test_rotary_refusals(lib):
    assert _rotary(lib, dtype=3) == 2
    assert _rotary(lib, D=7) == 1 and _rotary(lib, D=6) == 1        # odd; too few channels for the pairs
    assert _rotary(lib, D=258) == 5
    assert _rotary(lib, H=0) == 1 and _rotary(lib, T=-1) == 1
    assert _rotary(lib, B=65536, T=65536) == 5
    assert _rotary(lib, rot=_rotation(pairs=0)) == 1 and _rotary(lib, rot=_rotation(pairs=129), D=256) == 1
    assert _rotary(lib, rot=_rotation(axes=0)) == 1 and _rotary(lib, rot=_rotation(axes=5)) == 1
    assert _rotary(lib, rot=_rotation(interleaved=2)) == 1
    assert _rotary(lib, rot=_rotation(axis=[0, 0, 1, 0])) == 1
    assert b"pair 2" in lib.wan_vae_last_error()
    assert _rotary(lib, rot=_rotation(freq=[1.0, float("inf"), 1.0, 1.0])) == 1
    assert _rotary(lib, os=(48, 24, 0)) == 1                         # a broadcast output
    assert _rotary(lib, x=4097) == 1 and _rotary(lib, pos=66) == 1 and _rotary(lib, pos=68, pos64=1) == 1
    assert _rotary(lib, x=0) == 1 and _rotary(lib, pb=-1) == 1
    assert _rotary(lib, T=0, x=0, out=0, pos=0) == 0                  # nothing to do


def _cache(**kw):
    a = dict(k=4096, v=8192, dtype=1, heads=2, page_size=16, head_dim=64, pages=10, k_page=2048, k_head=1024, k_row=64,
             v_page=2048, v_head=1024, v_row=64)
    a.update(kw)
    return _lib.WanKvCache(*a.values())


def _batch(**kw):
    a = dict(pages=64, page_stride=4, max_pages=4, batch=3, lengths=64, cu_tokens=None, tokens=3, status=None)
    a.update(kw)
    return _lib.WanKvBatch(*a.values())


def _append(lib, c=None, b=None, rot=None, q=None, qo=None, qh=0, k=4096, v=4096, pos=None, qos=(256, 64)):
    r = ctypes.byref(rot) if rot else None
    return lib.wan_kv_append(ctypes.byref(c or _cache()), ctypes.byref(b or _batch()), k, 128, 64, v, 128, 64, q, qh, 256,
                             64, qo, *qos, r, pos, 0, None)


def _attend(lib, c=None, b=None, heads=4, q=4096, out=4096, scale=1.0, os=(256, 64), ranges=None, lse=None):
    return lib.wan_kv_attention(ctypes.byref(c or _cache()), ctypes.byref(b or _batch()), q, heads, 256, 64, ranges, scale,
                                out, *os, lse, None, 0, None)


CACHE_FAULTS = [(dict(k=None), 1), (dict(dtype=0), 2), (dict(heads=0), 1), (dict(page_size=0), 1), (dict(pages=0), 1),
                (dict(head_dim=60), 1), (dict(head_dim=264), 5), (dict(k=4104), 1), (dict(v_row=68), 1),
                (dict(k_head=-8), 1), (dict(page_size=1 << 30), 5)]
BATCH_FAULTS = [(dict(pages=None), 1), (dict(lengths=None), 1), (dict(batch=0), 1), (dict(max_pages=0), 1),
                (dict(page_stride=-1), 1), (dict(page_stride=2), 1), (dict(tokens=-1), 1), (dict(tokens=2), 4)]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS, ids=lambda f: str(f))
def test_cache_refusals(lib, fault, status):
    assert _append(lib, c=_cache(**fault)) == status
    assert _attend(lib, c=_cache(**fault)) == status
    assert lib.wan_kv_attention_workspace(ctypes.byref(_cache(**fault)), ctypes.byref(_batch()), 4) == -1
    assert lib.wan_vae_last_error()


@pytest.mark.parametrize("fault,status", BATCH_FAULTS, ids=lambda f: str(f))
def test_batch_refusals(lib, fault, status):
    assert _append(lib, b=_batch(**fault)) == status
    assert _attend(lib, b=_batch(**fault)) == status


def test_append_refusals(lib):
    assert _append(lib, k=None) == 1 and _append(lib, k=4097) == 1
    assert _append(lib, q=4096) == 1                                   # q without q_out
    assert _append(lib, q=4096, qo=4096, qh=0) == 1
    assert _append(lib, q=4096, qo=4096, qh=4, qos=(256, 0)) == 1
    assert _append(lib, rot=_rotation()) == 1                          # a rotation without positions
    assert _append(lib, rot=_rotation(pairs=33), pos=64) == 1
    assert _append(lib, c=_cache(k_head=0)) == 1                       # heads would share their rows
    assert b"broadcast" in lib.wan_vae_last_error()
    assert _append(lib, b=_batch(tokens=0, cu_tokens=64), k=None, v=None) == 0


def test_attention_refusals(lib):
    assert _attend(lib, heads=3) == 4 and _attend(lib, heads=0) == 4
    assert _attend(lib, scale=float("nan")) == 1 and _attend(lib, scale=float("inf")) == 1
    assert _attend(lib, q=None) == 1 and _attend(lib, out=4097) == 1
    assert _attend(lib, os=(0, 64)) == 1
    assert _attend(lib, ranges=66) == 1 and _attend(lib, lse=66) == 1
    assert _attend(lib, b=_batch(tokens=0, cu_tokens=64), q=None, out=None) == 0


def test_status_refusal(lib):
    assert lib.wan_kv_status(None, None) == 1


def _check(pages, lengths, size, n, **kw):
    import video_vae_decoding_gb300 as wv
    i = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    if "cu_tokens" in kw:
        kw["cu_tokens"] = i(kw["cu_tokens"])
    wv.kv_check(i(pages), i(lengths), size, n, **kw)


def test_kv_check_finds_what_the_kernels_leave_out(lib):
    import video_vae_decoding_gb300 as wv
    good = dict(pages=[[4, 0], [2, 9], [1, 0]], lengths=[16, 17, 0], size=16, n=5)
    with pytest.raises(wv.WanError, match="sequence 1: page 1 is number 9"):
        _check(**good)
    good["pages"][1][1] = 3
    _check(**good)
    _check(**dict(good, lengths=[16, 32, 0]))
    with pytest.raises(wv.WanError, match="sequence 2: page 0 is number -1"):
        _check(**dict(good, pages=[[4, 0], [2, 3], [-1, 0]], lengths=[16, 17, 1]))
    _check(**dict(good, pages=[[4, 0], [2, 3], [-1, 0]]))              # a page that no key is on
    with pytest.raises(wv.WanError, match="sequence 0: length 33"):
        _check(**dict(good, lengths=[33, 1, 0]))
    with pytest.raises(wv.WanError, match="sequence 1: length -1"):
        _check(**dict(good, lengths=[3, -1, 0]))


def test_kv_check_token_ranges(lib):
    import video_vae_decoding_gb300 as wv
    t = dict(pages=[[4, 0], [2, 3]], lengths=[16, 17], size=16, n=5)
    _check(**t, cu_tokens=[0, 3, 4])
    _check(**t, cu_tokens=[0, 0, 4], tokens=9)                         # rows behind the last sequence
    for cu, tokens in ([0, 5, 4], 5), ([-1, 2, 4], 4), ([0, 2, 6], 5):
        with pytest.raises(wv.WanError, match="token range"):
            _check(**t, cu_tokens=cu, tokens=tokens)
    _check(**t, cu_tokens=[0, 16, 33], append=True)
    with pytest.raises(wv.WanError, match="sequence 0: 17 new tokens among 16"):
        _check(**t, cu_tokens=[0, 17, 18], append=True)
    with pytest.raises(wv.WanError, match="shares its row"):
        _check(pages=[[1], [1]], lengths=[5, 5], size=16, n=5, append=True)
    _check(pages=[[1], [1]], lengths=[5, 5], size=16, n=5)             # reading a shared page is fine
    _check(pages=[[1], [1]], lengths=[5, 6], size=16, n=5, append=True)


def test_binding_refusals():
    import video_vae_decoding_gb300 as wv
    x, pos = torch.zeros(3, 2, 8), torch.zeros(3, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        wv.rotary(x, pos, (4,))
    with pytest.raises(ValueError, match="float64"):
        wv.rotary(x.double(), pos, (4,))
    with pytest.raises(ValueError, match="positions must be"):
        wv.rotary(x, pos, (2, 2))
    with pytest.raises(ValueError, match="autograd"):
        wv.rotary(x.clone().requires_grad_(), pos, (4,))
    with pytest.raises(ValueError, match="contiguous"):
        wv.rotary(x.transpose(1, 2), pos, (1,))
    with pytest.raises(ValueError, match="sections"):
        wv.Rotation(())
    with pytest.raises(ValueError, match="theta"):
        wv.Rotation((4,), theta=0.0)
    with pytest.raises(ValueError, match="frequencies"):
        wv.Rotation((4,), freq=[1.0])
    b = torch.bfloat16
    kc, k = torch.zeros(5, 2, 16, 8, dtype=b), torch.zeros(3, 2, 8, dtype=b)
    pages, lens = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        wv.kv_append(k, k, kc, kc, pages, lens)
    with pytest.raises(ValueError, match="the cache's tokens"):
        wv.kv_append(k[:, :1], k[:, :1], kc, kc, pages, lens)
    with pytest.raises(ValueError, match="float32"):
        wv.kv_append(k.float(), k, kc, kc, pages, lens)
    with pytest.raises(ValueError, match="float32"):
        wv.kv_attention(k, kc.float(), kc.float(), pages, lens)
    with pytest.raises(ValueError, match="sections need positions"):
        wv.kv_append(k, k, kc, kc, pages, lens, sections=(4,))
    with pytest.raises(ValueError, match="pages has"):
        wv.kv_attention(k, kc, kc, pages[:2], lens)
    with pytest.raises(ValueError, match="int64"):
        wv.kv_attention(k, kc, kc, pages.long(), lens)
    with pytest.raises(ValueError, match="ranges must be"):
        wv.kv_attention(k, kc, kc, pages, lens, ranges=pages[:2])
    with pytest.raises(ValueError, match="cu_tokens must hold"):
        wv.kv_attention(k, kc, kc, pages, lens, cu_tokens=lens)
    with pytest.raises(ValueError, match="head dim"):
        wv.kv_attention(k[..., :4], kc, kc, pages, lens)
    with pytest.raises(ValueError, match="autograd"):
        wv.kv_attention(k.clone().requires_grad_(), kc, kc, pages, lens)


def test_selftest_refusal(lib):
    code = ctypes.c_int32(7)
    for D in 0, 60, 264:
        assert lib.wan_selftest_kv_attention_timeout(D, ctypes.byref(code), None) == 1
        assert code.value == 0 and lib.wan_vae_last_error()


def test_attention_refuses_a_scale_that_overflows(lib):
    """A finite scale whose product with log2(e) is no finite float: every score would become NaN or infinite."""
    for scale in 2.5e38, -3.4e38:
        assert _attend(lib, scale=scale) == 1, scale
        assert b"scale" in lib.wan_vae_last_error()


def test_sizes_past_32_bits_are_refused_by_name(lib):
    """Not cut to their lower half on the way to C (2^32 + 3 tokens of a broadcast tensor cost no memory)."""
    import video_vae_decoding_gb300 as wv
    big = 2 ** 32 + 3
    b = torch.bfloat16
    kc, pages, lens = torch.zeros(5, 2, 16, 8, dtype=b), torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 8, dtype=b).expand(big, 2, 8)
    with pytest.raises(ValueError, match="4294967299 tokens"):
        wv.rotary(k, torch.zeros(3, 1, dtype=torch.int32), (4,))
    with pytest.raises(ValueError, match="4294967299 tokens"):
        wv.kv_append(k, k, kc, kc, pages, lens)
    with pytest.raises(ValueError, match="4294967299 tokens"):
        wv.kv_attention(k, kc, kc, pages, lens)
    with pytest.raises(ValueError, match="4294967299 heads"):
        wv.kv_attention(torch.zeros(1, 1, 8, dtype=b).expand(1, big, 8), kc, kc, pages, lens)
    with pytest.raises(ValueError, match="4294967299 heads"):
        wv.rotary(torch.zeros(1, 1, 8).expand(1, big, 8), torch.zeros(1, 1, dtype=torch.int32), (4,))
    wide = torch.zeros(5, 2, 1, 8, dtype=b).expand(5, 2, big, 8)
    with pytest.raises(ValueError, match="page size"):
        wv.kv_attention(torch.zeros(1, 2, 8, dtype=b), wide, wide, pages, lens)
    with pytest.raises(ValueError, match="page size"):
        wv.kv_check(pages, lens, 2 ** 32 + 16, 5)
    with pytest.raises(ValueError, match="tokens"):
        wv.kv_check(pages, lens, 16, 5, tokens=2 ** 32 + 1)


def test_dual_tensors_are_refused(lib):
    """A tangent would be dropped in silence: the operators are not recorded, forward or backward."""
    import video_vae_decoding_gb300 as wv
    fwd = torch.autograd.forward_ad
    pos = torch.zeros(3, 1, dtype=torch.int32)
    kc, pages, lens = torch.zeros(5, 2, 16, 8).bfloat16(), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with fwd.dual_level():
        x = fwd.make_dual(torch.zeros(3, 2, 8), torch.ones(3, 2, 8))
        k = fwd.make_dual(torch.zeros(3, 2, 8).bfloat16(), torch.ones(3, 2, 8).bfloat16())
        plain = torch.zeros(3, 2, 8).bfloat16()
        for call in (lambda: wv.rotary(x, pos, (4,)), lambda: wv.rotary_grad(x, pos, (4,)),
                     lambda: wv.kv_append(k, plain, kc, kc, pages, lens), lambda: wv.kv_append(plain, k, kc, kc, pages, lens),
                     lambda: wv.kv_attention(k, kc, kc, pages, lens)):
            with pytest.raises(ValueError, match="autograd"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="autograd"):
                call()
        with pytest.raises(ValueError, match="CUDA"):            # a plain tensor inside a dual level is none
            wv.rotary(torch.zeros(3, 2, 8), pos, (4,))

"""Refusals of the operators that see, copy and move keys by their place (no
GPU: every call here returns before any CUDA work)."""

import ctypes

import pytest
import torch

from tests.test_token_checks import BATCH_FAULTS, CACHE_FAULTS, _batch, _cache
from video_vae_decoding_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    from video_vae_decoding_gb300 import build
    build.build()
    return _lib.load()


ref = ctypes.byref


def _window(lib, c=None, b=None, heads=4, q=4096, out=4096, scale=1.0, os=(256, 64), window=5, sinks=1, frame=1, lse=None):
    return lib.wan_kv_window_attention(ref(c or _cache()), ref(b or _batch()), q, heads, 256, 64, window, sinks, frame, scale,
                                       out, *os, lse, None, 0, None)


def _tree(lib, c=None, b=None, heads=4, q=4096, out=4096, scale=1.0, os=(256, 64), parents=4096, lse=None):
    return lib.wan_kv_tree_attention(ref(c or _cache()), ref(b or _batch()), q, heads, 256, 64, parents, scale, out, *os, lse,
                                     None, 0, None)


def _fork(lib, c=None, pages=64, stride=4, columns=4, B=3, lengths=64, sources=64, targets=64, fresh=64, fs=1, fp=1, n=2, share=1,
          status=None):
    return lib.wan_kv_fork(ref(c or _cache()), pages, stride, columns, B, lengths, sources, targets, fresh, fs, fp, n, share,
                           status, None)


def _compact(lib, c=None, b=None, keep=4096, lengths=8192):
    return lib.wan_kv_compact(ref(c or _cache()), ref(b or _batch(cu_tokens=128)), keep, lengths, None)


@pytest.mark.parametrize("fault,status", CACHE_FAULTS, ids=lambda f: str(f))
def test_cache_refusals(lib, fault, status):
    c = _cache(**fault)
    assert _window(lib, c) == _tree(lib, c) == _fork(lib, c) == _compact(lib, c) == status
    assert lib.wan_kv_masked_attention_workspace(ref(c), ref(_batch()), 4) == -1
    assert lib.wan_vae_last_error()


@pytest.mark.parametrize("fault,status", BATCH_FAULTS, ids=lambda f: str(f))
def test_batch_refusals(lib, fault, status):
    b = _batch(**fault)
    assert _window(lib, b=b) == _tree(lib, b=b) == status
    if fault != dict(tokens=2):
        assert _compact(lib, b=_batch(cu_tokens=128, **fault)) == status


def test_window_refusals(lib):
    assert _window(lib, window=0) == 1 and _window(lib, frame=0) == 1 and _window(lib, sinks=-1) == 1
    assert b"first keys" in lib.wan_vae_last_error()
    assert _window(lib, heads=3) == 4 and _window(lib, scale=float("nan")) == 1 and _window(lib, os=(0, 64)) == 1
    assert _window(lib, q=None) == 1 and _window(lib, out=4097) == 1 and _window(lib, lse=66) == 1
    assert _window(lib, b=_batch(tokens=0, cu_tokens=64), q=None, out=None) == 0


def test_tree_refusals(lib):
    assert _tree(lib, parents=None) == 1 and _tree(lib, parents=4098) == 1
    assert _tree(lib, heads=0) == 4 and _tree(lib, scale=float("inf")) == 1 and _tree(lib, out=None) == 1
    assert _tree(lib, b=_batch(tokens=0, cu_tokens=64), q=None, out=None, parents=None) == 0


def test_fork_refusals(lib):
    for kw in (dict(pages=None), dict(lengths=None), dict(sources=None), dict(targets=None), dict(fresh=None), dict(B=0),
               dict(columns=0), dict(stride=3), dict(stride=0), dict(n=-1), dict(fp=-1), dict(fp=2), dict(share=2), dict(pages=66),
               dict(sources=65), dict(fresh=66), dict(status=66)):
        assert _fork(lib, **kw) == 1, kw
        assert lib.wan_vae_last_error()
    assert _fork(lib, c=_cache(k_head=0)) == 1
    assert b"broadcast" in lib.wan_vae_last_error()
    assert _fork(lib, n=1025) == 5
    # memory in common: fresh in the table's columns, in the lengths; sources in either; but not other columns of the same rows
    at = dict(pages=4096, stride=8, columns=4, B=3, lengths=8192, sources=12288, targets=16384, n=3, fp=2)
    for kw in (dict(fresh=4096, fs=8), dict(fresh=4096 + 32 + 12, fs=8), dict(fresh=4096 + 16, fs=7), dict(fresh=4096 + 28, fs=8),
               dict(fresh=8192, fs=2), dict(fresh=1 << 20, fs=2, sources=4096), dict(fresh=1 << 20, fs=2, targets=8200),
               dict(fresh=1 << 20, fs=2, lengths=4100)):
        assert _fork(lib, **{**at, **kw}) == 1, kw
        assert b"share" in lib.wan_vae_last_error(), kw
    assert _fork(lib, n=0, sources=None, targets=None, fresh=None) == 0


def test_compact_refusals(lib):
    assert _compact(lib, b=_batch()) == 1                    # no ranges
    assert _compact(lib, keep=None) == 1 and _compact(lib, lengths=None) == 1
    assert _compact(lib, keep=4098) == 1 and _compact(lib, lengths=8193) == 1
    assert _compact(lib, c=_cache(v_row=0)) == 1
    assert b"broadcast" in lib.wan_vae_last_error()
    for over in 64, 60, 72, 128, 4100:                       # in the memory of lengths and the table, of the ranges, of keep
        assert _compact(lib, lengths=over) == 1, over
        assert b"share" in lib.wan_vae_last_error()
    assert _compact(lib, c=_cache(heads=1001, k_page=2 ** 20, v_page=2 ** 20)) == 5


def test_binding_refusals(lib):
    import video_vae_decoding_gb300 as wv
    b = torch.bfloat16
    kc, q = torch.zeros(5, 2, 16, 8, dtype=b), torch.zeros(3, 2, 8, dtype=b)
    i = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    pages, lens, up = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32), i([-1, 0, 0])
    window = lambda *a, **kw: wv.kv_window_attention(*a, **kw)  # noqa: E731
    for match, call in [
        ("CUDA", lambda: window(q, kc, kc, pages, lens, 5)),
        ("float32", lambda: window(q.float(), kc, kc, pages, lens, 5)),
        ("head dim", lambda: window(q[..., :4], kc, kc, pages, lens, 5)),
        ("pages has", lambda: window(q, kc, kc, pages[:2], lens, 5)),
        ("cu_tokens must hold", lambda: window(q, kc, kc, pages, lens, 5, cu_tokens=lens)),
        ("4294967299 frames", lambda: window(q, kc, kc, pages, lens, 2 ** 32 + 3)),
        ("4294967299 first", lambda: window(q, kc, kc, pages, lens, 5, 2 ** 32 + 3)),
        ("4294967299 keys", lambda: window(q, kc, kc, pages, lens, 5, 0, 2 ** 32 + 3)),
        ("autograd", lambda: window(q.clone().requires_grad_(), kc, kc, pages, lens, 5)),
        ("CUDA", lambda: wv.kv_tree_attention(q, kc, kc, pages, lens, up)),
        ("int64", lambda: wv.kv_tree_attention(q, kc, kc, pages, lens, up.long())),
        ("parents must be", lambda: wv.kv_tree_attention(q, kc, kc, pages, lens, up[:2])),
        ("parents must be", lambda: wv.kv_tree_attention(q, kc, kc, pages, lens, i([0] * 6)[::2])),
        ("autograd", lambda: wv.kv_tree_attention(q.clone().requires_grad_(), kc, kc, pages, lens, up)),
        ("CUDA", lambda: wv.kv_fork(kc, kc, pages, lens, i([0]), i([1]), i([[4]]))),
        ("targets has", lambda: wv.kv_fork(kc, kc, pages, lens, i([0]), i([1, 2]), i([[4]]))),
        ("fresh has", lambda: wv.kv_fork(kc, kc, pages, lens, i([0]), i([1]), i([[4], [3]]))),
        ("fresh", lambda: wv.kv_fork(kc, kc, pages, lens, i([0]), i([1]), i([4]))),
        ("int64", lambda: wv.kv_fork(kc, kc, pages, lens, i([0]).long(), i([1]), i([[4]]))),
        ("contiguous", lambda: wv.kv_fork(kc, kc, pages, lens, i([0]), i([1]), i([[4, 3, 2]])[:, ::2])),
        ("autograd", lambda: wv.kv_fork(kc.clone().requires_grad_(), kc, pages, lens, i([0]), i([1]), i([[4]]))),
        ("CUDA", lambda: wv.kv_compact(kc, kc, pages, lens, i([3]), i([0, 1, 1, 1]))),
        ("cu_tokens must hold", lambda: wv.kv_compact(kc, kc, pages, lens, i([3]), i([0, 1, 1]))),
        ("int64", lambda: wv.kv_compact(kc, kc, pages, lens, i([3]).long(), i([0, 1, 1, 1]))),
        ("lengths must hold", lambda: wv.kv_compact(kc, kc, pages, lens, i([3]), i([0, 1, 1, 1]), i([1]))),
        ("contiguous", lambda: wv.kv_compact(kc, kc, pages, lens, i([3, 4, 5])[::2], i([0, 1, 1, 1]))),
        ("autograd", lambda: wv.kv_compact(kc.clone().requires_grad_(), kc, pages, lens, i([3]), i([0, 1, 1, 1]))),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError):
        window(q, kc, kc, pages, lens, 5.5)


def test_dual_tensors_are_refused(lib):
    import video_vae_decoding_gb300 as wv
    fwd = torch.autograd.forward_ad
    kc, pages, lens = torch.zeros(5, 2, 16, 8).bfloat16(), torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    with fwd.dual_level():
        q = fwd.make_dual(torch.zeros(3, 2, 8).bfloat16(), torch.ones(3, 2, 8).bfloat16())
        k2 = fwd.make_dual(torch.zeros(5, 2, 16, 8).bfloat16(), torch.ones(5, 2, 16, 8).bfloat16())
        for call in (lambda: wv.kv_window_attention(q, kc, kc, pages, lens, 5), lambda: wv.kv_tree_attention(q, kc, kc, pages, lens, lens),
                     lambda: wv.kv_fork(k2, kc, pages, lens, lens[:1], lens[:1], pages[:1]),
                     lambda: wv.kv_compact(k2, kc, pages, lens, lens[:1], lens[:1].expand(4).contiguous())):
            with torch.no_grad(), pytest.raises(ValueError, match="autograd"):
                call()

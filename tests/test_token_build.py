"""Building with and without the token operators' marshalling module (no GPU)."""

import os
import sys
import warnings

import pytest
import torch

import video_vae_decoding_gb300 as wv
from video_vae_decoding_gb300 import build, tokens


@pytest.fixture
def fakes(monkeypatch, tmp_path):
    """build() with its commands replaced: a list of what ran, in order."""
    ran = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "_nvcc", lambda: "nvcc")
    monkeypatch.setattr(build, "_compile", lambda nvcc, src, verbose: src)
    monkeypatch.setattr(build, "_link", lambda nvcc, objs: ran.append(("link", len(objs))))
    monkeypatch.setattr(build, "_compile_binding", lambda: ran.append(("binding", 0)))
    return ran


def _broken():
    raise RuntimeError("no g++ here")


def test_the_library_is_linked_without_the_binding(fakes, monkeypatch, capsys):
    monkeypatch.setattr(build, "_compile_binding", _broken)
    assert build.build(force=True) == build.LIB
    assert fakes == [("link", len(build.sources()))]
    assert "no g++ here" in capsys.readouterr().err


def test_a_broken_kernel_still_fails_the_build(fakes, monkeypatch):
    def compile(nvcc, src, verbose):
        raise RuntimeError("nvcc failed")
    monkeypatch.setattr(build, "_compile", compile)
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build(force=True)
    assert ("link", len(build.sources())) not in fakes


def test_each_part_is_built_for_itself(fakes, monkeypatch):
    for library, binding, want in ((True, True, []), (True, False, [("binding", 0)]),
                                   (False, True, [("link", len(build.sources()))])):
        fakes.clear()
        monkeypatch.setattr(build, "library_up_to_date", lambda: library)
        monkeypatch.setattr(build, "binding_up_to_date", lambda: binding)
        build.build()
        assert fakes == want


def test_a_binding_that_cannot_be_made_anew_is_not_used(monkeypatch, tmp_path, capsys):
    so, tag = tmp_path / "_tokens.so", tmp_path / "tag"
    so.write_text("")
    tag.write_text(build.binding_tag())
    for name, value in ("BINDING", str(so)), ("TAG", str(tag)), ("BUILD", str(tmp_path)), ("library_up_to_date", lambda: True):
        monkeypatch.setattr(build, name, value)
    os.utime(so, (1, 1))
    assert build.binding_fits() and not build.binding_up_to_date()

    def no_toolkit():
        raise RuntimeError("no toolkit here")
    monkeypatch.setattr(build, "_nvcc", no_toolkit)
    assert build.build() == build.LIB                           # the library is up to date and needs none
    assert "no toolkit here" in capsys.readouterr().err and not build.binding_fits()


def test_a_binding_for_another_torch_is_stale(monkeypatch, tmp_path):
    so, tag = tmp_path / "_tokens.so", tmp_path / "tag"
    monkeypatch.setattr(build, "BINDING", str(so))
    monkeypatch.setattr(build, "TAG", str(tag))
    assert not build.binding_up_to_date()
    so.write_text("")
    assert not build.binding_up_to_date()                       # nothing says what it was made for
    assert build.binding_tag() == f"{sys.implementation.cache_tag} torch {torch.__version__}"
    tag.write_text(build.binding_tag())
    assert build.binding_up_to_date()
    tag.write_text(f"{sys.implementation.cache_tag} torch 1.0")
    assert not build.binding_fits() and not build.binding_up_to_date()
    tag.write_text(build.binding_tag())
    os.utime(so, (1, 1))                                         # older than its source
    assert build.binding_fits() and not build.binding_up_to_date()


@pytest.mark.parametrize("how", ["absent", "stale", "broken"])
def test_calls_are_marshalled_in_python_without_the_binding(how, monkeypatch):
    build.build()
    monkeypatch.setattr(tokens, "_short", None)
    if how == "broken":
        monkeypatch.setitem(sys.modules, "video_vae_decoding_gb300._tokens", None)  # importing it raises
        monkeypatch.delattr(wv, "_tokens", raising=False)
        monkeypatch.setattr(build, "binding_fits", lambda: True)
    else:
        monkeypatch.setattr(build, "BINDING" if how == "absent" else "TAG", os.devnull + ".none")
    x, pos = torch.zeros(3, 2, 8), torch.zeros(3, 1, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="marshalled in Python"), pytest.raises(ValueError, match="CUDA"):
        wv.rotary(x, pos, (4,))
    with warnings.catch_warnings():                             # said once
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="CUDA"):
            wv.rotary_grad(x, pos, (4,))
    b = torch.bfloat16
    kc, pages, lens = torch.zeros(5, 2, 16, 8, dtype=b), torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    for call in lambda: wv.kv_append(x.to(b), x.to(b), kc, kc, pages, lens), lambda: wv.kv_attention(x.to(b), kc, kc, pages, lens):
        with pytest.raises(ValueError, match="CUDA"):
            call()

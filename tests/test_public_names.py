"""What the package offers by name (no GPU)."""

import video_vae_decoding_gb300 as wv
from video_vae_decoding_gb300 import tokens


def test_token_operators_are_the_packages():
    for name in tokens.__all__:
        assert getattr(wv, name) is getattr(tokens, name)
    assert set(tokens.__all__) <= set(wv.__all__)


def test_a_star_import_gives_what_is_named():
    got = {}
    exec("from video_vae_decoding_gb300 import *", got)
    assert set(wv.__all__) <= set(got)
    assert len(set(wv.__all__)) == len(wv.__all__)

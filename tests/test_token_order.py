"""Ordering rules of the tensor-core attention kernel that no result can show
reliably (a rule broken gives a right answer almost always): read off its source."""

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(ROOT, "video_vae_decoding_gb300", "csrc", "kv_chunk.cu")) as f:
        return f.read()


def test_weights_are_stored_behind_a_fence(source):
    """The softmax learns from a barrier, asked ahead, that the product which read the weights' room is complete:
    a tcgen05 fence has to stand between that answer and the stores, on every way."""
    asked = source.index("const uint32_t o_there")
    store = source.index("tmem_st16(myP", asked)
    loop = source.rindex("for (int q = 0; q < 4; ++q)", asked, store)
    slow = source.index("if (__builtin_expect(__any_sync(0xffffffffu, mb > m + kSlack", asked)
    behind = source.index("const float2 sc2", slow)  # the slow way, which has a fence of its own, is over
    assert "tc_fence_after();" in source[source.rindex("}\n", slow, behind):loop]


def test_products_are_committed_by_the_thread_that_issued_them(source):
    """A commit speaks of the products of its own thread: the last one, ahead of giving tensor memory back, has to be
    made by the elected thread, as the products are."""
    assert "const bool one = elect();" in source
    last = source.index("umma_commit(smem_u32(&done[")
    assert "elect()" in source[source.rindex("if (", 0, last):last]


def test_one_half_cleans_the_values_that_both_read(source):
    """Where both halves of a tile read a block's values, only the half whose product comes first may change them, and
    it decides by what the rows of either half see."""
    decided = source.index("if (cleans) hidden = ")
    line = source[decided:source.index("\n", decided)]
    for name in "all_lo[0]", "all_lo[1]", "all_hi[0]", "all_hi[1]":
        assert name in line
    assert "cleans = !turns || half == 0" in source

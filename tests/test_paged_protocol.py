"""The barrier protocol of the paged attention kernel under random interleavings.

What the model takes from the kernel's source: which ``ml`` entries a warp of a few-row segment
uses, and whether it fences the exchange area before it frees it."""

import functools
import os
import random
import re

import pytest

from paged_protocol import Fault, random_segments, run

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "block_sparse_long_sm_b200", "csrc", "paged_attn.cuh")


@functools.lru_cache(None)
def source():
    with open(SOURCE) as f:
        return f.read()


def few_segment():
    text = source()
    start = text.index("few_segment(const PagedAttnArgs& a")
    return text[start:text.index("\n}\n", start)]


def few_entry(warp, row):
    """The ml index of a warp's row when rows are few, as few_segment writes it."""
    index = re.search(r"ml\[(.+)\] = m\[e\];", few_segment()).group(1)
    body = re.search(r"constexpr int few_ml\(int warp, int row\) \{\s*return (.+);",
                     source())
    few_ml = (lambda warp, row: eval(body.group(1), {}, dict(warp=warp, row=row))) if body else None
    return eval(index, {}, dict(warp=warp, rr=row, few_ml=few_ml))


@functools.lru_cache(None)
def few_block(warp):
    return few_entry(warp, 0) // 16


def fence_before_free():
    tail = few_segment()
    tail = tail[tail.rindex("for (int rr = warp;"):]      # the join of the eight warps
    return "fence_proxy_async_smem();" in tail[:tail.index("mbar_arrive(bars.qfree(0))")]


def play(seeds, block=few_block, fenced=None):
    fenced = fence_before_free() if fenced is None else fenced
    for seed in seeds:
        rng = random.Random(seed)
        segs = random_segments(rng)
        try:
            run(segs, rng, block, fenced)
        except Fault as e:
            return f"seed {seed}, {[(s['kind'], s['n']) for s in segs]}: {e}"
    return None


def test_few_row_statistics_have_entries_of_their_own():
    at = {(w, r): few_entry(w, r) for w in range(8) for r in range(16)}
    assert sorted(at.values()) == list(range(128))
    assert all(at[w, r] == 16 * few_block(w) + r for w, r in at)


@pytest.mark.parametrize("part", range(4))
def test_random_interleavings(part):
    assert play(range(250 * part, 250 * part + 250)) is None


def test_the_model_sees_statistics_written_before_they_are_read():
    # sixteen entries per warp in the warps' order: warp 1 writes what warp 0 still reads
    found = play(range(400), block=lambda w: w, fenced=True)
    assert found is not None and "unread by" in found


def test_the_model_sees_a_copy_over_unfenced_stores():
    found = play(range(400), fenced=False)
    assert found is not None and "unfenced" in found

"""CPU-only: the flags "NaN of V were taken out" of ragged cache attention, modelled on the host under random interleavings
of the kernel's warps.

The conversion runs at most two blocks ahead of the products, which wait for every warp of a tile that has rows in the
item.  At the end of a run of blocks of one item (a segment) the converting warps leave a flag, and each warp of a
tile reads it once its sums are complete.  A tile is held to the products only by the segments that it has rows in: while
items with one tile follow one with two, the second tile's warps may be late by any number of segments.  So each
tile has flags of its own, numbered by its own segments; the model takes every step one at a time and checks that no
flag is written over before all warps of its tile have read it."""
import os
import random
import re

import pytest

from tiled_tensor_core_03_gb300 import _build

WARPS = 4   # of a tile


def run_once(segments, slots, of_tile, rng, late):
    """segments: (blocks, has a second tile) each; of_tile: flags numbered by a tile's own segments, or by all.
    True if every warp read the flag that was written for its segment."""
    blocks = [(s, j + 1 == n, two) for s, (n, two) in enumerate(segments) for j in range(n)]
    state = dict(converted=0, products=0)
    brought = [[0] * WARPS, [0] * WARPS]   # P of so many blocks, by each warp
    outputs = [0, 0]                       # segments whose sums are complete
    flags = [dict(), dict()]
    good = [True]

    def conversion():
        number = [0, 0]
        for i, (s, last, two) in enumerate(blocks):
            while state["products"] < i - 1:
                yield False
            if last:
                for t in range(1 + two):
                    flags[t][(number[t] if of_tile else s) % slots] = s
                    number[t] += 1
                if not of_tile:            # one set for both tiles
                    flags[1][s % slots] = s
            yield True
            state["converted"] = i + 1

    def products():
        turns = [0, 0]
        for i, (s, last, two) in enumerate(blocks):
            while state["converted"] <= i:
                yield False
            for t in range(1 + two):
                turns[t] += 1
                while min(brought[t]) < turns[t]:
                    yield False
            yield True
            state["products"] = i + 1
            if last:
                for t in range(1 + two):
                    outputs[t] += 1

    def softmax(t, w):
        first, done = 0, 0
        for s, (n, two) in enumerate(segments):
            if t == 0 or two:
                for i in range(first, first + n):
                    # its scores follow the products of the block before
                    while state["converted"] <= i or state["products"] < i:
                        yield False
                    yield True
                    brought[t][w] += 1
                while outputs[t] <= done:
                    yield False
                yield True
                good[0] = good[0] and flags[t][(done if of_tile else s) % slots] == s
                done += 1
            first += n

    actors = [conversion(), products()] + [softmax(t, w) for t in range(2) for w in range(WARPS)]
    slow = rng.randrange(len(actors)) if late else -1
    live = list(range(len(actors)))
    idle = 0
    while live:
        a = rng.choice(live)
        if a == slow and idle < 40 and len(live) > 1 and rng.random() < 0.99:
            idle += 1                      # (the others go on until they wait for it)
            continue
        try:
            idle = 0 if next(actors[a]) else idle + 1
        except StopIteration:
            live.remove(a)
        assert idle < 20000, "nobody can go on"
    return good[0]


def _cases(rng):
    yield [(3, True)] + [(1, False)] * 12 + [(2, True)]
    yield [(1, True)] * 9
    yield [(1, False)] * 9
    yield [(1, True), (1, False)] * 8
    for _ in range(6):
        yield [(rng.choice([1, 1, 2, 5]), rng.random() < 0.4) for _ in range(14)]


def _kept():
    with open(os.path.join(_build.CSRC, "kv_ragged.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return text, int(re.search(r"constexpr int kDirty = (\d+);", text).group(1))


@pytest.mark.parametrize("late", [False, True])
def test_no_flag_is_written_over_before_it_is_read(late):
    slots = _kept()[1]
    rng = random.Random(5 + late)
    for _ in range(30):
        for segments in _cases(rng):
            assert run_once(segments, slots, True, rng, late), segments


def test_the_model_finds_what_one_numbering_for_both_tiles_loses():
    rng = random.Random(7)
    assert not all(run_once([(3, True)] + [(1, False)] * 12, 4, False, rng, True) for _ in range(200))
    # and a slot fewer than the argument beside kDirty asks for
    assert not all(run_once([(1, True)] * 9, 1, True, rng, True) for _ in range(200))


def test_the_kernel_numbers_flags_by_tile():
    text = _kept()[0]
    uses = re.findall(r"dirty\[([^\]]*)\]", text)
    assert sorted(uses) == sorted(["kDirty * mine + segments0 % kDirty",
                                   "kDirty * (kConvWarps + mine) + segments1 % kDirty",
                                   "kDirty * (kConvWarps * t + x) + outputs % kDirty"])

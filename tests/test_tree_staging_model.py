"""The q tile of the tree attention kernel's softmax warpgroups, byte by byte, run on the CPU.

A tile holds q (warp w of the warpgroup writes rows 32 w ... 32 w + 31 of 128 bytes, here of the first
64 columns), then the references of a piece of one tile, then, a warp at a time, the output on its way
to memory.  Only q_full (the warpgroup's four warps), the outputs' commit and, after a piece of one
tile, merge (the eight warps of both) hold a warp back: behind a piece of two tiles a warp goes on to the
next piece's q while the others may still write outputs.  The four warps of each warpgroup are
coroutines under a random scheduler; at every read the model checks whose bytes are there.

Where a warp's outputs lie is read from the kernel's source.  The planted fault is the place they once
had: 1024 + 2048 w overlaps the q rows of other warps."""
import os
import random
import re

import pytest

from test_prompt_protocol_model import Barrier

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "mxfp4_quantized_gemm_token_gb300", "csrc", "attn_tree.cu")
ROWS, ROW, UNIT = 32, 128, 16          # rows of a warp, bytes of one, bytes that move together
STAGE = 32 * 64                        # bytes of a warp's outputs on their way
TILE = 128 * ROW


def stage_of(warp):
    with open(SOURCE) as f:
        at = re.search(r"uint8_t\* stage = q_tile \+ ([^;]+);", f.read()).group(1)
    return eval(at, {"__builtins__": {}}, {"warp": warp})


def old_stage(warp):
    return 1024 + (warp & 3) * 2048


class Model:
    def __init__(self, pieces, seed, stage, steps=2):
        self.pieces, self.rng, self.stage, self.steps = pieces, random.Random(seed), stage, steps
        self.tile = [[None] * (TILE // UNIT) for _ in range(2)]
        self.q_full = [Barrier(4), Barrier(4)]
        self.o_full = [Barrier(1), Barrier(1)]
        self.merge = [Barrier(8), Barrier(8)]
        self.done = []

    def write(self, s, at, size, tag):
        for u in range(at // UNIT, (at + size) // UNIT):
            self.tile[s][u] = tag

    def holds(self, s, at, size, tag):
        return all(self.tile[s][u] == tag for u in range(at // UNIT, (at + size) // UNIT))

    def turns(self, piece, s):
        n, single = piece
        return (n - s + 1) // 2 if single else n

    def mma(self, s):
        """The products of a warpgroup: q is read until its last one is complete."""
        n = 0
        for i, piece in enumerate(self.pieces):
            if not self.turns(piece, s):
                continue
            yield self.q_full[s], n & 1
            for _ in range(1 + self.turns(piece, s)):
                assert self.holds(s, 0, TILE, ("q", i)), "another item's q, or outputs in it"
                yield None
            self.o_full[s].arrive()
            n += 1

    def softmax(self, s, w):
        no = nm = 0
        for i, piece in enumerate(self.pieces):
            single = piece[1]
            if self.turns(piece, s):
                for r in range(0, ROWS, 8):
                    self.write(s, (w * ROWS + r) * ROW, 8 * ROW, ("q", i))
                    yield None
                self.q_full[s].arrive()
                yield self.o_full[s], no & 1
                no += 1
            if single:
                self.write(s, w * 256, 256, ("ml", i, s, w))
                self.merge[0].arrive()
                yield self.merge[0], nm & 1
                for t in range(2):
                    assert self.holds(t, w * 256, 256, ("ml", i, t, w)), "another's references"
            at = self.stage(4 * s + w)
            assert 0 <= at and at + STAGE <= TILE
            for step in range(self.steps):
                for half in range(2):
                    self.write(s, at + half * STAGE // 2, STAGE // 2, ("out", i, w, step))
                    yield None
                assert self.holds(s, at, STAGE, ("out", i, w, step)), "outputs overwritten"
                yield None
            if single:
                for t in range(2):
                    assert self.holds(t, w * 256, 256, ("ml", i, t, w)), "references overwritten"
                self.merge[1].arrive()
                yield self.merge[1], nm & 1
                nm += 1
            self.done.append((s, w, i))

    def run(self):
        roles = [self.mma(s) for s in range(2)]
        roles += [self.softmax(s, w) for s in range(2) for w in range(4)]
        # a warp may be far slower than another
        speed = [self.rng.choice([1, 1, 20]) for _ in roles]
        waits = [next(r, StopIteration) for r in roles]
        while True:
            able = [k for k, w in enumerate(waits) if w is not StopIteration
                    and (w is None or w[0].passes(w[1]))]
            if not able:
                break
            k = self.rng.choices(able, [speed[k] for k in able])[0]
            waits[k] = next(roles[k], StopIteration)
        return all(w is StopIteration for w in waits) and len(self.done) == 8 * len(self.pieces)


LISTS = [[(1, True)] * 4, [(1, False)] * 4, [(3, False), (1, True), (2, False), (5, True)],
         [(1, False), (1, True)] * 3, [(2, True), (1, False), (1, False), (4, True)]]


@pytest.mark.parametrize("pieces", LISTS)
@pytest.mark.parametrize("steps", [1, 2, 8])
def test_tiles(pieces, steps):
    for seed in range(40):
        assert Model(pieces, seed, stage_of, steps).run(), "deadlock"


def test_a_warps_outputs_lie_in_its_own_rows():
    """and clear of the references in the first 1024 bytes: no barrier has to stand between."""
    for warp in range(8):
        at = stage_of(warp)
        assert at % UNIT == 0 and at >= 1024
        assert (warp & 3) * ROWS * ROW <= at and at + STAGE <= ((warp & 3) + 1) * ROWS * ROW


@pytest.mark.parametrize("pieces", [[(1, False)] * 4, [(2, False), (1, True), (3, False)]])
def test_planted_stages_in_other_warps_rows_show(pieces):
    def fails(stage):
        for seed in range(60):
            try:
                if not Model(pieces, seed, stage).run():
                    return True
            except AssertionError:
                return True
        return False

    assert fails(old_stage) and not fails(stage_of)

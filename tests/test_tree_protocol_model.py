"""An executable model of the tree attention kernel's barriers, run on the CPU, after that of
the prompt kernel (test_prompt_protocol_model): the warp that finds the pieces, the loading
warps and, for an e4m3 cache, the converting ones, MMA issue and the two softmax warpgroups are
coroutines; copies land in any order, tensor-core work in order but later; a random scheduler
interleaves everything.

A piece is (blocks, single): the blocks of one tile, taken by both warpgroups in turn and
joined at the end, or of two, each taken by both.  At every use the model checks that a ring
slot holds the whole block that is meant, that the masks of loaded keys are the block's,
that scores, weights and outputs are whose they should be; at the end nothing may be left
waiting.

Planted faults: a ring of masks that is too short for the copies that run ahead, and a joined
output that is written again before both warpgroups have read it."""
import random

import pytest

from test_prompt_protocol_model import Barrier

PIECES = 8            # pieces under way


def is_value(f, n):
    return (f > 0 and f % 2 == 0) or f == 2 * n - 1


def block(f, n):
    return 0 if f == 0 else (f - 1) // 2 if is_value(f, n) else (f + 1) // 2


class Model:
    def __init__(self, pieces, stages, seed, raw=0, loaders=6, seen=16, no_second_merge=False):
        """raw: stages of e4m3 rows as they are cached (0: a bf16 cache)."""
        self.pieces, self.stages, self.raw_stages = pieces, stages, raw
        self.rng, self.seen_size = random.Random(seed), seen
        self.no_second_merge = no_second_merge
        self.loaders = 2 if raw else loaders
        others = self.loaders + (4 if raw else 0) + 3
        self.piece_full = [Barrier(1) for _ in range(PIECES)]
        self.piece_empty = [Barrier(others) for _ in range(PIECES)]
        self.ring_of_pieces = [None] * PIECES
        self.q_full = [Barrier(1), Barrier(1)]
        self.s_full, self.o_full = [Barrier(1), Barrier(1)], [Barrier(1), Barrier(1)]
        self.p_full = [[Barrier(1), Barrier(1)], [Barrier(1), Barrier(1)]]
        self.merge = [Barrier(2), Barrier(2)]
        self.kv_full = [Barrier(4 if raw else 8) for _ in range(stages)]
        self.kv_empty = [Barrier(1) for _ in range(stages)]
        self.raw_full = [Barrier(4) for _ in range(raw)]      # two warps, copies landed and word
        self.raw_empty = [Barrier(4) for _ in range(raw)]
        self.ring = [[None] * 4 for _ in range(stages)]
        self.raw = [[None] * 4 for _ in range(raw)]
        self.seen = [[None] * 4 for _ in range(seen)]
        self.q, self.scores = [None, None], [None, None]
        self.weights, self.out = [[None, None], [None, None]], [[], []]
        self.copies, self.tensor, self.results = [], [], []

    # ---- roles: yield a (barrier, parity) to wait for, or None to let others run
    def walk(self):
        for n, p in enumerate(list(enumerate(self.pieces)) + [None]):
            at = n % PIECES
            yield self.piece_empty[at], ((n // PIECES) & 1) ^ 1
            self.ring_of_pieces[at] = p
            self.piece_full[at].arrive()

    def each_piece(self, body):
        n = 0
        while True:
            at = n % PIECES
            yield self.piece_full[at], (n // PIECES) & 1
            p = self.ring_of_pieces[at]
            if p is None:
                return
            yield from body(*p)
            assert self.ring_of_pieces[at] == p, "piece overwritten"
            self.piece_empty[at].arrive()
            n += 1

    def load(self, w):
        """bf16: units of a quarter of a copy, round the warps."""
        at = {"unit": w, "base": 0, "blocks": 0}

        def body(i, piece):
            n = piece[0]
            while at["unit"] // 4 - at["base"] < 2 * n:
                u = at["unit"]
                fill, g = u // 4, u % 4
                f = fill - at["base"]
                j, v = block(f, n), is_value(f, n)
                if not v:
                    self.seen[(at["blocks"] + j) % self.seen_size][g] = (i, j)
                st = fill % self.stages
                yield self.kv_empty[st], ((fill // self.stages) & 1) ^ 1
                self.copies.append((self.ring[st], [g], (i, "v" if v else "k", j),
                                    self.kv_full[st]))
                self.kv_full[st].arrive()
                at["unit"] += self.loaders
            at["base"] += 2 * n
            at["blocks"] += n

        yield from self.each_piece(body)

    def fetch(self, w):
        """e4m3: two quarters of every copy."""
        at = {"fill": 0, "blocks": 0}

        def copy(what):
            st = at["fill"] % self.raw_stages
            yield self.raw_empty[st], ((at["fill"] // self.raw_stages) & 1) ^ 1
            self.copies.append((self.raw[st], [w, w + 2], what, self.raw_full[st]))
            self.raw_full[st].arrive()
            at["fill"] += 1

        def body(i, piece):
            n = piece[0]
            for j in range(n + 1):
                if j < n:
                    for g in (w, w + 2):
                        self.seen[(at["blocks"] + j) % self.seen_size][g] = (i, j)
                    yield from copy((i, "k", j))
                if j > 0:
                    yield from copy((i, "v", j - 1))
            at["blocks"] += n

        yield from self.each_piece(body)

    def convert(self, g):
        at = {"fill": 0}

        def body(i, piece):
            n = piece[0]
            for f in range(2 * n):
                fill = at["fill"]
                r, st = fill % self.raw_stages, fill % self.stages
                yield self.raw_full[r], (fill // self.raw_stages) & 1
                what = (i, "v" if is_value(f, n) else "k", block(f, n))
                assert self.raw[r][g] == what, "other rows"
                yield self.kv_empty[st], ((fill // self.stages) & 1) ^ 1
                self.ring[st][g] = what
                self.kv_full[st].arrive()
                self.raw_empty[r].arrive()
                at["fill"] += 1

        yield from self.each_piece(body)

    def mma(self):
        at = {"base": 0, "nq": [0, 0], "np": [0, 0]}

        def kv(fill):
            return self.kv_full[fill % self.stages], (fill // self.stages) & 1

        def commit(bar):
            self.tensor.append(("commit", bar))

        def body(i, piece):
            n, single = piece
            turns, base = (n if single else 2 * n), at["base"]
            of = lambda t: t if single else t // 2
            k_fill = lambda j: base + (0 if j == 0 else 2 * j - 1)
            v_fill = lambda j: base + (2 * j + 2 if j + 1 < n else 2 * j + 1)

            def scores(s, j, fill):
                self.tensor.append(("s", s, i, j, fill % self.stages))
                commit(self.s_full[s])
                if single or s == 1:
                    commit(self.kv_empty[fill % self.stages])

            for t in range(min(2, turns)):
                yield kv(k_fill(of(t)))
                yield self.q_full[t], at["nq"][t] & 1
                at["nq"][t] += 1
                scores(t, of(t), k_fill(of(t)))
            for t in range(turns):
                s, vf = t & 1, v_fill(of(t))
                yield kv(vf)
                for part in (1, 0):
                    yield self.p_full[s][part], at["np"][s] & 1
                    self.tensor.append(("o", s, i, of(t), vf % self.stages, part, t < 2))
                at["np"][s] += 1
                if single or s == 1:
                    commit(self.kv_empty[vf % self.stages])
                if t + 2 < turns:
                    yield kv(k_fill(of(t + 2)))
                    scores(s, of(t + 2), k_fill(of(t + 2)))
                else:
                    commit(self.o_full[s])
            at["base"] += 2 * n

        yield from self.each_piece(body)

    def softmax(self, s):
        at = {"ns": 0, "no": 0, "nm": 0, "blocks": 0}

        def want(w, i, n, single):
            blocks = [j for j in range(n) if not single or j % 2 == w]
            return [(i, j, part) for j in blocks for part in (1, 0)]

        def body(i, piece):
            n, single = piece
            turns = (n - s + 1) // 2 if single else n
            if turns:
                self.q[s] = i
                yield None
                self.q_full[s].arrive()
            for t in range(turns):
                j = 2 * t + s if single else t
                yield self.s_full[s], at["ns"] & 1
                at["ns"] += 1
                assert self.scores[s] == (i, j), "scores of another block"
                assert self.seen[(at["blocks"] + j) % self.seen_size] == [(i, j)] * 4, "masks"
                yield None
                for part in (1, 0):
                    assert self.weights[s][part] is None, "weights overwritten"
                    self.weights[s][part] = (i, j)
                    yield None
                    self.p_full[s][part].arrive()
                    yield None
            at["blocks"] += n
            if turns:
                yield self.o_full[s], at["no"] & 1
                at["no"] += 1
            if single:
                self.merge[0].arrive()
                yield self.merge[0], at["nm"] & 1
            read = [0] + [1] * (n > 1) if single else [s]
            for w in read:
                assert self.out[w] == want(w, i, n, single), "another item's output"
            yield None
            for w in read:
                assert self.out[w] == want(w, i, n, single), "output overwritten while it was read"
            self.results.append((s, i))
            if single:
                self.merge[1].arrive()
                if not self.no_second_merge:
                    yield self.merge[1], at["nm"] & 1
                at["nm"] += 1

        yield from self.each_piece(body)

    # ---- asynchronous work
    def finish_copy(self):
        slot, quarters, what, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
        for g in quarters:
            slot[g] = what
        bar.arrive()

    def finish_tensor(self):
        op = self.tensor.pop(0)
        if op[0] == "commit":
            op[1].arrive()
        elif op[0] == "s":
            _, s, i, j, slot = op
            assert self.ring[slot] == [(i, "k", j)] * 4 and self.q[s] == i, "wrong operand"
            assert self.weights[s] == [None, None], "weights overwritten by scores"
            self.scores[s] = (i, j)
        else:
            _, s, i, j, slot, part, first = op
            assert self.ring[slot] == [(i, "v", j)] * 4, "wrong values"
            assert self.weights[s][part] == (i, j), "wrong weights"
            self.weights[s][part] = None
            if first and part == 1:
                self.out[s] = []
            self.out[s].append((i, j, part))

    def run(self):
        roles = [self.walk(), self.mma(), self.softmax(0), self.softmax(1)]
        if self.raw_stages:
            roles += [self.fetch(w) for w in range(2)] + [self.convert(g) for g in range(4)]
        else:
            roles += [self.load(w) for w in range(self.loaders)]
        waits = [next(r, StopIteration) for r in roles]
        while True:
            able = [k for k, w in enumerate(waits) if w is not StopIteration
                    and (w is None or w[0].passes(w[1]))]
            able += ["copy"] * bool(self.copies) + ["tensor"] * bool(self.tensor)
            if not able:
                break
            k = self.rng.choice(able)
            if k == "copy":
                self.finish_copy()
            elif k == "tensor":
                self.finish_tensor()
            else:
                waits[k] = next(roles[k], StopIteration)
        return all(w is StopIteration for w in waits)


LISTS = [[], [(1, True)], [(1, False)], [(2, True), (3, False)], [(5, True), (1, True), (4, False)],
         [(1, True)] * 12, [(1, False), (1, True)] * 5, [(9, True)], [(8, False), (7, True)],
         [(2, False)] * 6, [(12, True), (11, False), (1, True), (3, True)]]


@pytest.mark.parametrize("pieces", LISTS)
@pytest.mark.parametrize("stages,raw", [(5, 0), (10, 0), (3, 4), (6, 8)])
def test_protocol(pieces, stages, raw):
    for seed in range(25):
        m = Model(pieces, stages, seed, raw)
        assert m.run(), "deadlock"
        assert sorted(m.results) == sorted((s, i) for s in range(2) for i in range(len(pieces)))


def fails(pieces=((9, True), (6, False), (14, True)), **planted):
    for seed in range(60):
        try:
            if not Model(list(pieces), seed=seed, **planted).run():
                return True
        except AssertionError:
            return True
    return False


def test_planted_short_ring_of_masks_shows():
    assert fails(stages=6, raw=8, seen=4)
    assert not fails(stages=6, raw=8)


def test_planted_missing_second_merge_shows():
    # the next piece's output is written without the other warpgroup where it has one block
    pieces = [(4, True), (1, True)] * 8
    assert fails(pieces, stages=5, no_second_merge=True)
    assert not fails(pieces, stages=5)


def test_a_ring_of_one_stage_is_too_short():
    assert fails(stages=1)

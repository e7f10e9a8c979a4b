"""What the prompt attention kernel leaves behind when a bounded wait gives up, on the
CPU model of its barriers: at a random moment one role's wait runs out, the others leave
at their next wait that does not pass, and the loads' and the MMAs' roles then wait for
their own work in flight.  When all roles have ended, and with them the block's
hold on its shared and tensor memory, no copy and no product may be under way.

Two faults the kernel once had are planted: waiting for work in flight only where the
role itself saw a wait give up, so that one that had ended before leaves its last copies
under way; and copies of Q counted by items begun, so that one that was never
issued is waited for until that wait, too, runs out."""
import random

import pytest

from test_prompt_protocol_model import ITEMS, Barrier, Model


class GaveUp(Exception):
    pass


class Aborting(Model):
    def __init__(self, items, stages, seed, count_items=False, only_if_seen=False):
        super().__init__(items, stages, seed)
        self.count_items, self.only_if_seen = count_items, only_if_seen
        self.drain = Barrier(1)
        self.draining = set()

    def load(self):
        fill, n, q = 0, 0, [0, 0]
        seen = False
        try:
            for i, blocks in enumerate(self.items):
                if blocks == 0:
                    continue
                n += 1
                order = [("q", 0), ("k", 0), ("q", 1), ("v", 0)]
                order += [(c, j) for j in range(1, blocks) for c in "kv"]
                for what, j in order:
                    if what == "q":
                        yield self.q_empty[j], (q[j] & 1) ^ 1
                        self.copies.append((self.q, j, (i, "q"), self.q_full[j]))
                        q[j] += 1
                    else:
                        st = fill % self.stages
                        yield self.kv_empty[st], ((fill // self.stages) & 1) ^ 1
                        self.copies.append((self.ring, st, (i, what, j), self.kv_full[st]))
                        fill += 1
        except GaveUp:
            seen = True
        if self.only_if_seen and not seen:
            return
        if self.count_items:
            q = [n, n]
        self.draining.add(0)
        for f in range(max(0, fill - self.stages), fill):
            yield self.kv(f)
        for s in range(2):
            if q[s]:
                yield self.q_full[s], (q[s] - 1) & 1

    def mma(self):
        seen = False
        try:
            yield from super().mma()
        except GaveUp:
            seen = True
        if self.only_if_seen and not seen:
            return
        self.tensor.append(("commit", self.drain))
        self.draining.add(1)
        yield self.drain, 0

    def softmax(self, s):
        try:
            yield from super().softmax(s)
        except GaveUp:
            pass

    def run(self, moment):
        """True if nothing is in flight when the last role ends."""
        roles = [self.load(), self.mma(), self.softmax(0), self.softmax(1)]
        waits = [next(r, StopIteration) for r in roles]
        aborted, step = False, 0
        while any(w is not StopIteration for w in waits):
            step += 1
            able, stuck = [], []
            for k, w in enumerate(waits):
                if w is StopIteration:
                    continue
                if w is None or w[0].passes(w[1]):
                    able.append(k)
                elif k not in self.draining:
                    stuck.append(k)
            if stuck and (aborted or step >= moment):
                aborted = True
                able += [-1 - k for k in stuck]
            able += ["copy"] * bool(self.copies) + ["tensor"] * bool(self.tensor)
            assert able, "deadlock"
            k = self.rng.choice(able)
            if k == "copy":
                self.finish_copy()
            elif k == "tensor":
                self.finish_tensor()
            elif k < 0:
                try:
                    waits[-1 - k] = roles[-1 - k].throw(GaveUp())
                except StopIteration:
                    waits[-1 - k] = StopIteration
            else:
                waits[k] = next(roles[k], StopIteration)
        return not self.copies and not self.tensor


def clean(items, stages, seeds, **planted):
    return all(Aborting(items, stages, seed, **planted).run(
        random.Random(seed).randrange(1, 40 * (1 + sum(items)))) for seed in range(seeds))


@pytest.mark.parametrize("items", ITEMS)
@pytest.mark.parametrize("stages", [4, 8])
def test_nothing_is_in_flight_at_the_end(items, stages):
    assert clean(items, stages, 150)


def test_planted_leaving_early_shows():
    assert not all(clean(items, 4, 300, only_if_seen=True) for items in ITEMS)


def test_planted_count_of_items_waits_for_nothing():
    with pytest.raises(AssertionError, match="deadlock"):
        for items in ITEMS:
            clean(items, 4, 300, count_items=True)

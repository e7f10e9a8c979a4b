"""The counters of the prompt attention's list of items, restated on the CPU with the
kernel's integer widths, over packed offsets within the limits that the entry point
accepts: B <= 65535 sequences of Tq <= 2^30 rows, which may run backwards and overlap.

The fault that the longer list once had is planted: items counted in 32 bits with a single
test `place < room` let a count that had wrapped to a negative place write before the list."""
import random

import pytest

BUCKETS = 512
WRAP = 1 << 32


def int32(n):
    return (n + (1 << 31)) % WRAP - (1 << 31)


def room(Tq, B, per):
    return Tq // per + min(B, Tq) + 1


def items(n, per):
    return -(-n // per)


def histogram(n, per):
    """Items of a causal sequence of n rows and keys by their bucket, most blocks first."""
    h = [0] * BUCKETS
    count = items(n, per)
    # item i ends at key min(n, (i + 1) per): ceil of that over 128 blocks
    for blocks in range(1, BUCKETS - 1):
        last = min(count, max(0, (128 * blocks) // per if 128 * blocks < n else count))
        first = min(count, (128 * (blocks - 1)) // per if 128 * (blocks - 1) < n else count)
        h[BUCKETS - 1 - blocks] = last - first
    h[0] = count - sum(h)
    return h


def lengths(cu, Tq):
    return [e - a for a, e in zip(cu, cu[1:]) if 0 <= a <= e <= Tq]


def places(cu, Tq, per, old=False):
    """Ranges of the list's places that are written."""
    B = len(cu) - 1
    cap = room(Tq, B, per)
    seqs = lengths(cu, Tq)
    if not old:
        counted, all_items = [0] * BUCKETS, 0
        for n in seqs:
            all_items += items(n, per)
            if all_items > cap:
                continue
            counted = [c + h for c, h in zip(counted, histogram(n, per))]
        assert all_items < 1 << 64 and all(0 <= c < 1 << 31 for c in counted)
        if all_items > cap:
            return [], cap
    each = {n: histogram(n, per) for n in set(seqs)}
    totals = [sum(each[n][k] * seqs.count(n) for n in each) for k in range(BUCKETS)]
    start, out = 0, []
    for c in totals:
        begin = int32(start)
        start = int32(start + int32(c)) if old else start + c
        # what passes the test `place < room` of the places begin, begin + 1, ... (mod 2^32)
        if begin + c > 1 << 31:
            out.append((-(1 << 31), int32(begin + c)))
        if c and begin < cap:
            out.append((begin, min(begin + c, cap)))
    return out, cap


SAWTOOTH = [(1 << 30, 65535, 2), (132000, 65535, 2), (17000000, 65535, 256), (1 << 30, 9, 2)]


@pytest.mark.parametrize("Tq,B,per", SAWTOOTH + [(5000, 6, 8), (1 << 20, 1, 2)])
def test_nothing_is_written_outside_the_list(Tq, B, per):
    cu = [0 if b % 2 == 0 else Tq for b in range(B + 1)]
    written, cap = places(cu, Tq, per)
    assert all(0 <= a <= e <= cap for a, e in written)


@pytest.mark.parametrize("seed", range(40))
def test_offsets_in_order_always_fit(seed):
    rng = random.Random(seed)
    Tq, B = int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 8))
    per = 2 * (128 // rng.choice([1, 2, 3, 4, 5, 8, 16, 20, 100, 128]))
    cu = sorted(rng.randrange(Tq + 1) for _ in range(B + 1))
    written, cap = places(cu, Tq, per)
    total = sum(items(n, per) for n in lengths(cu, Tq))
    assert total <= cap and sum(e - a for a, e in written) == total
    assert all(0 <= a <= e <= cap for a, e in written)


def test_the_short_list_counts_in_range():
    """Up to 512 items' room: no sequence has more, so that 65535 of them stay below 2^31."""
    assert 65535 * 512 < 1 << 31


@pytest.mark.parametrize("Tq,B,per", SAWTOOTH)
def test_planted_32_bit_counts_write_before_the_list(Tq, B, per):
    cu = [0 if b % 2 == 0 else Tq for b in range(B + 1)]
    written, _ = places(cu, Tq, per, old=True)
    assert any(a < 0 for a, _ in written)

"""Which pages a window may leave behind while drafts are under way, on the lists that
cache_resize is tested against."""
import pytest

import cache_util as ref

WIDTH = 30


def grown(n, size, window, first):
    """A row that has been decoded token by token with the window."""
    refs, row, at = [0] * 40, [-1] * WIDTH, 0
    while at < n:
        (row,), refs = ref.resize([row], [at], [at + 1], refs, size, window, first)
        at += 1
    return row, refs


def missing(row, size, keys):
    return [j for j in keys if row[j // size] < 0]


def seen(position, window, first):
    return [j for j in range(position + 1) if j > position - window or j < first]


def losses(size, window, first, n, drafts, grow):
    """Keys that a step misses: its tree's rows, the rows after any number of accepted drafts."""
    row, refs = grown(n, size, window, first)
    (row,), refs = ref.resize([row], [n], [n + drafts], refs, size, *grow)
    lost = []
    for i in range(drafts):
        lost += missing(row, size, seen(n + i, window, first))
    for accepted in range(drafts + 1):
        m = n + accepted
        (cut,), _ = ref.resize([row], [n + drafts], [m], refs, size, window, first)
        (on,), _ = ref.resize([cut], [m], [m + 1], refs, size)
        lost += missing(cut, size, seen(m - 1, window, first))
        lost += missing(on, size, seen(m, window, first))
    return lost


@pytest.mark.parametrize("size", [1, 2, 3, 4])
@pytest.mark.parametrize("window,first", [(1, 0), (3, 0), (4, 2), (7, 5), (9, 1)])
def test_drafts_grow_with_a_longer_window_or_none(size, window, first):
    for n in range(1, 20):
        for drafts in range(1, 7):
            for grow in ((0, 0), (window + drafts, first)):
                assert losses(size, window, first, n, drafts, grow) == []


def test_the_window_itself_would_free_what_drafts_see():
    assert losses(1, 3, 0, 10, 4, (3, 0))
    assert losses(2, 4, 1, 15, 6, (4, 1))

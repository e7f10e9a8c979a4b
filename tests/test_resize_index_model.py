"""The places of a table's row that cache_resize frees behind a window, restated on the CPU with
the kernel's 32-bit integers, over the windows and first keys that the entry point accepts.

The fault that the call once had is planted: with `first` as it is given, pages of one token and
`first` near 2^31 wrap the next lane's index to a negative one, which is below the end."""
import pytest

LIMIT = 1 << 30
MOST = (1 << 31) - 1


def int32(n):
    return (n + (1 << 31)) % (1 << 32) - (1 << 31)


def freed(pages_before, new_len, page_size, window, first, bounded=True):
    """Indexes that the 32 lanes touch, in their first round (later ones lie above)."""
    if bounded:
        window, first = min(window, LIMIT), min(first, LIMIT)
    begin = int32(((first + page_size - 1) % (1 << 32)) // page_size)
    end = min(pages_before, -(-new_len // page_size), max(0, int32(new_len - window)) // page_size)
    return [i for i in (int32(begin + lane) for lane in range(32)) if i < end]


@pytest.mark.parametrize("page_size", [1, 2, 3, 64, 1 << 20, LIMIT])
@pytest.mark.parametrize("first", [0, 1, 33, LIMIT - 1, LIMIT, LIMIT + 5, MOST - 31, MOST])
@pytest.mark.parametrize("window", [1, 7, LIMIT, MOST])
def test_indexes_stay_in_the_row(page_size, first, window):
    for new_len in (0, 1, 40, 1000, LIMIT):
        pages = -(-new_len // page_size)
        got = freed(pages, new_len, page_size, window, first)
        want = [i for i in range(-(-first // page_size), pages)[:32]
                if (i + 1) * page_size <= new_len - window]
        assert got == want and all(0 <= i < pages for i in got)


def test_planted_unbounded_first_shows():
    assert min(freed(40, 40, 1, 7, MOST, bounded=False)) < 0
    assert freed(40, 40, 64, 7, MOST, bounded=False) == []

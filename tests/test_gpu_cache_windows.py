"""Pages that a window leaves behind: the ends of the arguments' ranges."""
import pytest
import torch

import cache_util as ref
import mxfp4_quantized_gemm_token_gb300 as mxq

pytestmark = pytest.mark.gpu
MOST = (1 << 31) - 1


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page", [1, 3, 64])
@pytest.mark.parametrize("first", [0, 2, 1 << 30, (1 << 30) + 1, MOST - 31, MOST])
@pytest.mark.parametrize("window", [1, 5, 1 << 30, MOST])
def test_first_and_window_at_the_ends_of_their_ranges(page, first, window):
    """Rows in the middle of a larger buffer, whose other entries stay."""
    pages, rows, width = 100, 3, 20
    lens, new = [40 % (20 * page), 7, 20 * page], [min(41, 20 * page), 6, 20 * page]
    buffer = torch.full((rows + 20, width + 12), 5, dtype=torch.int32, device="cuda")
    order, table = list(range(pages)), []
    for n in lens:
        row = [order.pop() for _ in range(ref.pages_of(n, page))]
        table.append(row + [-1] * (width - len(row)))
    counts = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                counts[p] += 1
    t, r = buffer[10:10 + rows, 6:6 + width], ints(counts)
    t.copy_(ints(table))
    kept = buffer.clone()
    mxq.cache_resize(t, ints(lens), ints(new), r, page, window=window, first=first)
    mxq.sync_status()
    wt, wr = ref.resize(table, lens, new, counts, page, window, first)
    assert t.tolist() == wt and r.tolist() == wr
    kept[10:10 + rows, 6:6 + width] = t
    assert torch.equal(buffer, kept)

"""A row cut inside a page that a fork shared: its siblings' keys stay, once it is forked onto
itself before it is written."""
import pytest
import torch

import cache_util as ref
import mxfp4_quantized_gemm_token_gb300 as mxq

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page,n,cuts", [(4, 14, [5, 14, 14]), (16, 40, [17, 31, 33]),
                                         (8, 16, [3, 8, 9]), (1, 9, [4, 9, 0])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_cut_row_is_forked_onto_itself(page, n, cuts, dtype):
    KV, D, pages, width = 2, 64, 60, -(-(n + 8) // page)
    g = torch.Generator(device="cuda").manual_seed(page)
    randn = lambda m: torch.randn(m, KV, D, generator=g, device="cuda").to(torch.bfloat16)
    kc = torch.zeros(pages, page, KV, D, dtype=torch.bfloat16, device="cuda").to(dtype)
    vc = kc.clone()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    mxq.cache_resize(table, ints([0]), ints([n]), refs, page)

    def slots(b, begin, end):
        p = torch.arange(begin, end, device="cuda")
        return table[b].long()[p // page] * page + p % page

    def append(b, begin, k, v):
        mxq.rope_append_kv(k, v, kc, vc, slots(b, begin, begin + len(k)))

    def held(b, m):
        at = slots(b, 0, m)
        return [c.view(torch.uint8)[at // page, at % page].clone() for c in (kc, vc)]

    append(0, 0, randn(n), randn(n))
    # three samples, then cut
    table, lens, copies = mxq.cache_fork(table, ints([n]), refs, ints([0, 0, 0]), page)
    mxq.cache_copy_pages(kc, vc, copies)
    whole = held(0, n)
    mxq.cache_resize(table, lens, ints(cuts), refs, page)
    rows, counts = table.tolist(), refs.tolist()
    table, lens, copies = mxq.cache_fork(table, ints(cuts), refs, ints([0, 1, 2]), page)
    mxq.cache_copy_pages(kc, vc, copies)
    want = ref.fork(rows, cuts, counts, [0, 1, 2], page)
    assert table.tolist() == want[0] and lens.tolist() == cuts and refs.tolist() == want[3]
    # no open page is held twice
    for b, m in enumerate(cuts):
        if m % page:
            assert counts[rows[b][m // page]] == 1 or table[b, m // page] != rows[b][m // page]
            assert refs[table[b, m // page]] == 1
    # all rows grow at once, and hold their own prefix and what they appended
    new = [m + 7 for m in cuts]
    mxq.cache_resize(table, lens, ints(new), refs, page)
    added = []
    for b, m in enumerate(cuts):
        k, v = randn(7), randn(7)
        append(b, m, k, v)
        added.append((k, v))
    mxq.sync_status()
    for b, m in enumerate(cuts):
        for c, w, x in zip(held(b, new[b]), whole, added[b]):
            assert torch.equal(c[:m], w[:m])
            assert torch.equal(c[m:], x.to(dtype).view(torch.uint8))

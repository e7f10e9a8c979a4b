"""Steps of a streaming layer that drafts: pages taken for a tree's rows, the tree verified within a
window and first keys, rejected drafts cut off, pages behind the window freed, the next token
decoded; against plain lists of keys, in 64 bits."""
import random

import pytest
import torch

import cache_util as ref
import mxfp4_quantized_gemm_token_gb300 as mxq
from attention_util import assert_within, attend
from test_gpu_tree_attention import cumulated, gen, ints, randn, tree, visible

pytestmark = pytest.mark.gpu
H, KV, D = 8, 2, 64


@pytest.mark.parametrize("page,window,first", [(1, 5, 0), (1, 20, 3), (4, 9, 2), (16, 40, 20)])
@pytest.mark.parametrize("longer", [False, True])
def test_steps_of_drafts_within_a_window(page, window, first, longer):
    """longer: the table grows with window + drafts, so that pages are freed there too, and not
    without a window."""
    g, rng = gen(page), random.Random(window)
    lens, drafts = [30, 6, 50], 7
    B, width = len(lens), -(-120 // page)
    pages = B * width
    kc = torch.zeros(pages, page, KV, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    lists, counts = table.tolist(), refs.tolist()

    def resize(a, b, w, f):
        nonlocal lists, counts
        mxq.cache_resize(table, ints(a), ints(b), refs, page, window=w, first=f)
        lists, counts = ref.resize(lists, a, b, counts, page, w, f)
        assert table.tolist() == lists and refs.tolist() == counts

    def slots(b, begin, end):
        p = torch.arange(begin, end, device="cuda")
        return table[b].long()[p // page] * page + p % page

    resize([0] * B, lens, 0, 0)
    k = [randn(g, n, KV, D) for n in lens]
    v = [randn(g, n, KV, D) for n in lens]
    for b in range(B):
        mxq.rope_append_kv(k[b], v[b], kc, vc, slots(b, 0, lens[b]))
    resize(lens, lens, window, first)
    args = dict(window=window, first=first)
    for accepted in ([0, 3, 1], [2, 0, 5], [1, 1, 0], [4, 2, 3]):
        most = [n + drafts for n in lens]
        resize(lens, most, *((window + drafts, first) if longer else (0, 0)))
        nk, nv, q = randn(g, B * drafts, KV, D), randn(g, B * drafts, KV, D), randn(g, B * drafts,
                                                                                 H, D)
        mxq.rope_append_kv(nk, nv, kc, vc, torch.cat([slots(b, lens[b], most[b])
                                                      for b in range(B)]))
        trees = [tree("random", drafts, rng) for _ in range(B)]
        out = mxq.paged_attention_tree(q, kc, vc, table, ints(most), cumulated([drafts] * B),
                                       ints([p for t in trees for p in t]), **args)
        mxq.sync_status()
        paths = []
        for b, t in enumerate(trees):
            rows = slice(b * drafts, (b + 1) * drafts)
            kk, vv = torch.cat([k[b], nk[rows]]), torch.cat([v[b], nv[rows]])
            see = visible(t, most[b], window, first)
            for h in range(H):
                r = attend(q[rows, h], kk[:, h // 4], vv[:, h // 4], see, D ** -0.5)
                assert_within(out[rows, h], r[0], r[2], "tree")
            # a path from its root, `accepted` rows of it at most
            path, i = [], drafts - 1
            while i >= 0:
                path.insert(0, i)
                i = t[i]
            paths.append(path[:accepted[b]])
        kept = ints([p + [0] * (drafts - len(p)) for p in paths])
        mxq.cache_compact(kc, vc, table, ints(lens), kept, ints([len(p) for p in paths]))
        new = [n + len(p) for n, p in zip(lens, paths)]
        resize(most, new, window, first)
        for b, path in enumerate(paths):
            at = torch.tensor(path, dtype=torch.long, device="cuda") + b * drafts
            k[b], v[b] = torch.cat([k[b], nk[at]]), torch.cat([v[b], nv[at]])
        lens = new
        q = randn(g, B, H, D)
        got = mxq.paged_attention_decode(q, kc, vc, table, ints(lens), **args)
        mxq.sync_status()
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            see = ((j >= n - window) | (j < first))[None]
            for h in range(H):
                r = attend(q[b:b + 1, h], k[b][:, h // 4], v[b][:, h // 4], see, D ** -0.5)
                assert_within(got[b:b + 1, h], r[0], r[2], "decode")
    # what a window left behind is free
    assert sum(counts) < sum(-(-n // page) for n in lens) or page == 16

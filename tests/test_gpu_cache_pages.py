"""The pages of a cache: tables and counts against loops over lists, moved rows bit for bit."""
import random

import pytest
import torch

import cache_util as ref
import mxfp4_quantized_gemm_token_gb300 as mxq

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


def ints(x, shape=None):
    t = torch.tensor(x, dtype=torch.int32, device="cuda")
    return t if shape is None else t.reshape(shape)


def tables(rng, rows, width, pages, size, shared=0.3, released=0.1):
    """A table whose rows share some leading pages, with its lengths and counts."""
    order = list(range(pages))
    rng.shuffle(order)
    table, lens, refs = [], [], [0] * pages
    for b in range(rows):
        want = rng.randint(0, width)
        row = []
        if table and rng.random() < shared:
            n = lens[-1] // size
            row = table[-1][:min(n, want)]
        while len(row) < want and order:
            row.append(order.pop())
        n = max(0, len(row) * size - rng.choice([0, rng.randint(0, size - 1)])) if row else 0
        assert ref.pages_of(n, size) == len(row)
        row = [-1 if rng.random() < released and i + 1 < len(row) else p
               for i, p in enumerate(row)]
        for p in row:
            if p >= 0:
                refs[p] += 1
        table.append(row + [-1] * (width - len(row)))
        lens.append(n)
    return table, lens, refs


@pytest.mark.parametrize("rows,width,pages,size,window,first", [
    (1, 1, 1, 1, 0, 0), (1, 7, 50, 16, 0, 0), (5, 9, 33, 3, 0, 0), (64, 20, 3000, 16, 0, 0),
    (300, 12, 5000, 5, 0, 0), (40, 30, 2000, 4, 17, 0), (40, 30, 2000, 4, 33, 9),
    (40, 30, 2000, 1, 1, 1), (10, 8, 70001, 64, 100, 1 << 30), (10000, 3, 40000, 8, 0, 0)])
def test_resize(rows, width, pages, size, window, first):
    rng = random.Random(rows * 31 + width)
    table, lens, refs = tables(rng, rows, width, pages, size)
    free = sum(n == 0 for n in refs)
    new = []
    for n in lens:
        want = rng.choice([0, n, n + 1, rng.randint(0, width * size)])
        want = max(0, min(want, width * size))
        more = ref.pages_of(want, size) - ref.pages_of(n, size)
        if more > free:
            want, more = n, 0
        free -= max(0, more)
        new.append(want)
    t, r = ints(table, (rows, width)), ints(refs)
    got = mxq.cache_resize(t, ints(lens), ints(new), r, size, window=window, first=first)
    assert got is t
    wt, wr = ref.resize(table, lens, new, refs, size, window, first)
    # what lies behind a row's pages is as it was
    assert t.tolist() == wt and r.tolist() == wr


def test_resize_strided_table_and_workspace():
    rng = random.Random(7)
    table, lens, refs = tables(rng, 12, 10, 200, 8)
    new = [min(80, n + 9) for n in lens]
    wide = torch.full((12, 17), 77, dtype=torch.int32, device="cuda")
    wide[:, :10] = ints(table)
    ws = torch.full((mxq.cache_pages_workspace_size(12, 200),), 255, dtype=torch.uint8,
                    device="cuda")
    r = ints(refs)
    mxq.cache_resize(wide[:, :10], ints(lens), ints(new), r, 8, workspace=ws)
    wt, wr = ref.resize(table, lens, new, refs, 8)
    assert wide[:, :10].tolist() == wt and r.tolist() == wr
    assert bool((wide[:, 10:] == 77).all())


def test_resize_without_pages_left():
    t, r = torch.full((3, 4), -1, dtype=torch.int32, device="cuda"), ints([1, 0, 1, 0, 0])
    mxq.cache_resize(t, ints([0, 0, 0]), ints([8, 3, 9]), r, 4)
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    assert t.tolist() == [[1, 3, -1, -1], [4, -1, -1, -1], [-1, -1, -1, -1]]
    assert r.tolist() == [1, 1, 1, 1, 1]


@pytest.mark.parametrize("lens,new", [([-1], [4]), ([4], [99]), ([9], [4])])
def test_resize_bad_lengths(lens, new):
    """They are clamped to the table's eight keys, and flagged."""
    t, r = ints([[0, 1]]), ints([1, 1, 0, 0])
    mxq.cache_resize(t, ints(lens), ints(new), r, 4)
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    clamp = lambda x: [max(0, min(8, n)) for n in x]
    wt, wr = ref.resize([[0, 1]], clamp(lens), clamp(new), [1, 1, 0, 0], 4)
    assert t.tolist() == wt and r.tolist() == wr


def test_resize_bad_pages_and_counts():
    t, r = ints([[9, 0, 1]]), ints([0, 1, 0, 0])
    mxq.cache_resize(t, ints([12]), ints([0]), r, 4)     # page 9 of 4, page 0 held by none
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    assert t.tolist() == [[-1, -1, -1]] and r.tolist() == [-1, 0, 0, 0]


@pytest.mark.parametrize("rows,n,width,pages,size", [
    (1, 1, 1, 2, 1), (1, 4, 5, 40, 16), (8, 8, 9, 200, 3), (16, 64, 20, 3000, 16),
    (256, 256, 12, 9000, 5), (3, 0, 4, 20, 4), (64, 1, 40, 5000, 8), (9000, 10000, 2, 60000, 4)])
def test_fork(rows, n, width, pages, size):
    rng = random.Random(rows * 7 + n)
    table, lens, refs = tables(rng, rows, width, pages, size)
    parents = [rng.choice([-1, rng.randrange(rows), rng.randrange(rows)]) for _ in range(n)]
    r = ints(refs)
    new, new_lens, copies = mxq.cache_fork(ints(table, (rows, width)), ints(lens), r,
                                           ints(parents), size)
    wt, wl, wc, wr = ref.fork(table, lens, refs, parents, size)
    assert new.tolist() == wt and new_lens.tolist() == wl
    assert copies.tolist() == wc and r.tolist() == wr
    # every count is the number of entries that hold the page
    held = [0] * pages
    for row in wt:
        for p in row:
            if p >= 0:
                held[p] += 1
    assert held == wr


def test_fork_into_given_table():
    rng = random.Random(3)
    table, lens, refs = tables(rng, 6, 7, 90, 4)
    parents = [5, 5, 0, -1, 2]
    wide = torch.full((5, 9), 55, dtype=torch.int32, device="cuda")
    out = wide[:, :7]
    r = ints(refs)
    ws = torch.full((mxq.cache_pages_workspace_size(6, 90),), 255, dtype=torch.uint8,
                    device="cuda")
    new, new_lens, copies = mxq.cache_fork(ints(table), ints(lens), r, ints(parents), 4, out=out,
                                           workspace=ws)
    assert new is out
    wt, wl, wc, wr = ref.fork(table, lens, refs, parents, 4)
    assert out.tolist() == wt and new_lens.tolist() == wl and copies.tolist() == wc
    assert r.tolist() == wr and bool((wide[:, 7:] == 55).all())


def test_fork_page_held_elsewhere_is_copied():
    """An open page that another batch's table holds too is nobody's to write."""
    r = ints([2, 0, 0])
    new, lens, copies = mxq.cache_fork(ints([[0]]), ints([3]), r, ints([0]), 4)
    assert new.tolist() == [[1]] and copies.tolist() == [[0, 1, 3]] and r.tolist() == [1, 1, 0]


def test_fork_without_pages_left_and_bad_parents():
    r = ints([1, 1, 0])
    new, lens, copies = mxq.cache_fork(ints([[0, 1]]), ints([6]), r, ints([0, 0, 0, 7, -2]), 4)
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    assert new.tolist() == [[0, 1], [0, 2], [0, -1], [-1, -1], [-1, -1]]
    assert lens.tolist() == [6, 6, 6, 0, 0] and r.tolist() == [3, 1, 1]
    assert copies.tolist() == [[-1, -1, 0], [1, 2, 2], [-1, -1, 0], [-1, -1, 0], [-1, -1, 0]]


def caches(pages, size, heads, dim, dtype, layout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = {"token": (pages, size, heads, dim), "head": (pages, heads, size, dim),
             "wide": (pages, size, heads, dim + 64)}[layout]
    res = []
    for _ in range(2):
        x = torch.randint(0, 256, shape + (2,), generator=g, device="cuda", dtype=torch.uint8)
        x = x.view(torch.int16)[..., 0] if dtype == torch.bfloat16 else x[..., 0]
        x = x.contiguous().view(dtype)              # any bits, NaN among them
        res.append(x.transpose(1, 2) if layout == "head" else x[..., :dim])
    return res


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16)


@pytest.mark.parametrize("size,heads,dim,dtype,layout", [
    (16, 8, 128, torch.bfloat16, "token"), (1, 1, 64, torch.bfloat16, "token"),
    (24, 3, 64, FP8, "head"), (7, 5, 16, FP8, "token"), (64, 2, 128, FP8, "wide"),
    (33, 4, 80, torch.bfloat16, "head"), (128, 8, 512, torch.bfloat16, "wide")])
@pytest.mark.parametrize("n", [1, 9, 200])
def test_copy_pages(size, heads, dim, dtype, layout, n):
    rng = random.Random(n)
    pages = 2 * n + 3
    k, v = caches(pages, size, heads, dim, dtype, layout)
    order = list(range(pages))
    rng.shuffle(order)
    copies = [[rng.choice(order[n:]), order[i], rng.randint(0, size)] for i in range(n)]
    for c in copies[::5]:
        c[rng.randrange(2)] = -1
    copies[0][2] = size
    wk, wv = bits(k).clone(), bits(v).clone()
    for src, dst, t in copies:
        if src >= 0 and dst >= 0:
            wk[dst, :t], wv[dst, :t] = bits(k)[src, :t], bits(v)[src, :t]
    mxq.cache_copy_pages(k, v, ints(copies))
    assert torch.equal(bits(k), wk) and torch.equal(bits(v), wv)


def test_copy_pages_refused_entries():
    k, v = caches(4, 4, 2, 64, torch.bfloat16, "token")
    wk = bits(k).clone()
    wk[1] = wk[0]
    mxq.cache_copy_pages(k, v, ints([[0, 4, 4], [9, 2, 4], [0, 1, 99], [0, 3, -1]]))
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    assert torch.equal(bits(k), wk)
    mxq.cache_copy_pages(k, v, ints([], (0, 3)))
    assert torch.equal(bits(k), wk)


@pytest.mark.parametrize("lens,most,size,heads,dim,dtype,layout", [
    ([5], 1, 16, 8, 128, torch.bfloat16, "token"),
    ([40, 7, 100], 6, 16, 8, 128, torch.bfloat16, "token"),
    ([0, 1, 300, 17], 64, 24, 3, 64, FP8, "head"),
    ([900], 700, 1, 1, 64, torch.bfloat16, "token"),
    ([5000, 3], 4000, 64, 8, 128, torch.bfloat16, "token"),
    ([2500] * 40, 2000, 7, 2, 80, torch.bfloat16, "wide"),
    ([70] * 700, 9, 16, 1, 16, FP8, "token"),
    ([3000], 3000, 128, 5, 512, FP8, "head")])
@pytest.mark.parametrize("order", ["random", "tail", "all", "reverse"])
def test_compact(lens, most, size, heads, dim, dtype, layout, order):
    rng = random.Random(len(lens) * 3 + most)
    need = [ref.pages_of(n, size) for n in lens]
    pages, width = sum(need) + 2, max(need) + 1
    k, v = caches(pages, size, heads, dim, dtype, layout)
    free = list(range(pages))
    rng.shuffle(free)
    table = [[free.pop() for _ in range(n)] for n in need]
    starts, kept, counts = [], [], []
    for n in lens:
        s = rng.randint(0, n // 3) if order != "all" else 0
        m = min(most, n - s)
        if order == "tail":
            rows = list(range(n - s - m, n - s))
        elif order == "all":
            rows = list(range(m))
        elif order == "reverse":
            # no order is asked for, only that none is below its index
            rows = sorted(rng.sample(range((n - s) // 2, n - s), min(m, (n - s) // 2)),
                          reverse=True)
        else:
            rows = sorted(rng.sample(range(n - s), rng.randint(0, m)))
        starts.append(s), kept.append(rows), counts.append(len(rows))
    wk, wv = bits(k).clone(), bits(v).clone()
    for row, s, rows in zip(table, starts, kept):
        if not rows:
            continue
        src = torch.tensor([s + r for r in rows], device="cuda")
        dst = torch.arange(s, s + len(rows), device="cuda")
        row = torch.tensor(row, device="cuda")
        for w, c in ((wk, k), (wv, v)):
            w[row[dst // size], dst % size] = bits(c)[row[src // size], src % size]
    t = ints([r + [-1] * (width - len(r)) for r in table], (len(lens), width))
    # the list's rows are longer than what is used of them
    wide = torch.full((len(lens), most + 3), -5, dtype=torch.int32, device="cuda")
    for b, rows in enumerate(kept):
        wide[b, :len(rows)] = ints(rows)
    mxq.cache_compact(k, v, t, ints(starts), wide[:, :most], ints(counts))
    assert torch.equal(bits(k), wk) and torch.equal(bits(v), wv)


def test_compact_refused_entries():
    k, v = caches(4, 4, 2, 64, torch.bfloat16, "token")
    before, (w0, w1) = bits(k).clone(), (bits(k).clone(), bits(v).clone())
    table = ints([[0, 1, 9], [2, 3, -1], [0, 1, 2]])
    # row 0: 3 -> 0 moves, 0 is below its index, 9 lies in page 9, 99 past the table;
    # row 1: a count above the list's width is its width; row 2: a negative start
    kept = ints([[3, 0, 9, 99], [1, 2, 3, 4], [1, 2, 3, 4]])
    mxq.cache_compact(k, v, table, ints([0, 0, -1]), kept, ints([4, 5, 4]))
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    w0[0, 0], w1[0, 0] = w0[0, 3], w1[0, 3]
    flat0, flat1 = w0[2:].view(8, 2, 64), w1[2:].view(8, 2, 64)
    flat0[:4], flat1[:4] = flat0[1:5].clone(), flat1[1:5].clone()
    assert torch.equal(bits(k), w0) and torch.equal(bits(v), w1) and not torch.equal(w0, before)


def test_a_captured_step_replays():
    """Fork, copy and resize in a graph: every replay works on what the tables hold then."""
    rng = random.Random(11)
    size, rows, width, pages = 8, 12, 20, 400
    table, lens, refs = tables(rng, rows, width - 2, pages, size, released=0)
    table = [r + [-1, -1] for r in table]
    k, v = caches(pages, size, 2, 64, torch.bfloat16, "token")
    t, n, r = ints(table), ints(lens), ints(refs)
    parents, out = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.empty_like(t)
    ws = torch.empty(mxq.cache_pages_workspace_size(rows, pages), dtype=torch.uint8, device="cuda")

    def step():
        _, new, copies = mxq.cache_fork(t, n, r, parents, size, out=out, workspace=ws)
        mxq.cache_copy_pages(k, v, copies)
        grown = new + 1
        mxq.cache_resize(out, new, grown, r, size, workspace=ws)
        t.copy_(out)
        n.copy_(grown)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        keep = [x.clone() for x in (t, n, r, k, v)]
        step()
        for x, y in zip((t, n, r, k, v), keep):
            x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    wk, wv = k.clone(), v.clone()
    for i in range(3):
        p = [rng.randrange(rows) for _ in range(rows)]
        parents.copy_(ints(p))
        graph.replay()
        new, new_lens, copies, refs = ref.fork(table, lens, refs, p, size)
        for src, dst, m in copies:
            if src >= 0:
                wk[dst, :m], wv[dst, :m] = wk[src, :m].clone(), wv[src, :m].clone()
        lens = [x + 1 for x in new_lens]
        table, refs = ref.resize(new, new_lens, lens, refs, size)
        assert t.tolist() == table and n.tolist() == lens and r.tolist() == refs
    assert torch.equal(bits(k), bits(wk)) and torch.equal(bits(v), bits(wv))


def test_rows_past_32_bits():
    """Copies and compaction in a cache of more than 2^32 elements."""
    pages, size, heads, dim = 70, 16, 2, 64
    flat = torch.empty(pages << 26, dtype=torch.bfloat16, device="cuda")      # 4.7e9 elements
    k, v = (flat.as_strided((pages, size, heads, dim), (1 << 26, heads * dim, dim, 1),
                            half << 25) for half in range(2))
    sk, sv = caches(pages, size, heads, dim, torch.bfloat16, "token")
    k.copy_(sk), v.copy_(sv)
    table, copies = ints([[69, 3, 66, 68]]), ints([[69, 65, 16], [1, 67, 5], [68, 0, 9]])
    kept = ints([[1, 2, 17, 30, 31, 33, 50, 63]])
    for a, b in ((k, v), (sk, sv)):
        mxq.cache_compact(a, b, table, ints([0]), kept, ints([8]))
        mxq.cache_copy_pages(a, b, copies)
    mxq.sync_status()
    assert torch.equal(bits(k), bits(sk)) and torch.equal(bits(v), bits(sv))


def test_compact_takes_a_row_twice_and_replays():
    """A row that is kept twice, and a captured call that works on what the lists hold then."""
    rng = random.Random(5)
    size, heads, dim, n, most = 24, 3, 64, 700, 300
    k, v = caches(64, size, heads, dim, torch.bfloat16, "token")
    pages = list(range(64))
    rng.shuffle(pages)
    rows = [pages[:30], pages[30:60]]
    table, starts = ints(rows), ints([3, 0])
    kept, counts = torch.zeros(2, most, dtype=torch.int32, device="cuda"), ints([0, 0])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        mxq.cache_compact(k, v, table, starts, kept, counts)            # nothing is kept
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            mxq.cache_compact(k, v, table, starts, kept, counts)
    for m in (1, 9, 300):
        lists = [[max(i, rng.randrange(n)) for i in range(m)] for _ in range(2)]
        lists[0] = [x for x in lists[0][::2] for _ in range(2)][:m] if m > 1 else lists[0]
        lists = [[max(i, x) for i, x in enumerate(row)] for row in lists]
        wk, wv = bits(k).clone(), bits(v).clone()
        for row, s, list_ in zip(rows, (3, 0), lists):
            src = torch.tensor([s + x for x in list_], device="cuda")
            dst = torch.arange(s, s + len(list_), device="cuda")
            at = torch.tensor(row, device="cuda")
            for w, c in ((wk, k), (wv, v)):
                w[at[dst // size], dst % size] = bits(c)[at[src // size], src % size]
        for b, list_ in enumerate(lists):
            kept[b, :len(list_)] = ints(list_)
        counts.copy_(ints([len(x) for x in lists]))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        mxq.sync_status()
        assert torch.equal(bits(k), wk) and torch.equal(bits(v), wv)

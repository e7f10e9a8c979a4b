"""paged_attention_tree against a plain 64-bit form within the bounds of attention_util:
trees, chunks, lengths, groups, page sizes, windows with first keys, caches of both types,
strides, and what unseen places hold."""
import random

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib
from attention_util import assert_within, attend

pytestmark = pytest.mark.gpu
NAN = float("nan")
FP8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def cumulated(n):
    return ints([sum(n[:i]) for i in range(len(n) + 1)])


def tree(kind, n, rng):
    """Parents of n rows."""
    if kind == "chain" or kind is None:
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] * n
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(n)]
    return [rng.randint(max(-1, i - 9), i - 1) for i in range(n)]


def visible(parents, n, window, first):
    """[rows, n keys]"""
    m = len(parents)
    P = n - m
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    j = torch.arange(P)
    res = torch.zeros(m, n, dtype=torch.bool)
    for i, d in enumerate(depth):
        res[i, :P] = True if not window else (j > P + d - window) | (j < first)
        up = i
        while up >= 0:
            pos = P + depth[up]
            res[i, P + up] = not window or pos > P + d - window or pos < first
            up = parents[up]
    return res.cuda()


class Case:
    def __init__(self, nq, lens, H, KV, D, page=16, kind="random", window=0, first=0, fp8=False,
                 sinks=False, seed=0, layout="token"):
        self.__dict__.update(locals())
        g = self.g = gen(seed + 13 * sum(lens) + H)
        rng = random.Random(seed + sum(nq))
        need = [-(-n // page) for n in lens]
        pages, width = sum(need) + 2, max(1, max(need))
        shape = (pages, page, KV, D) if layout == "token" else (pages, KV, page, D)
        self.kc, self.vc = randn(g, *shape), randn(g, *shape)
        self.ks = self.vs = None
        if fp8:
            self.kc, self.vc = ((t.float() * 100).clamp(-448, 448).to(FP8)
                                for t in (self.kc, self.vc))
            self.ks, self.vs = (0.01 + 0.01 * torch.rand(KV, generator=g, device="cuda")
                                for _ in range(2))
        if layout == "head":
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        order = list(range(pages))
        rng.shuffle(order)
        self.rows = [[order.pop() for _ in range(n)] for n in need]
        self.table = ints([r + [-1] * (width - len(r)) for r in self.rows])
        self.q = randn(g, sum(nq), H, D)
        self.s = torch.randn(H, generator=g, device="cuda") * 2 if sinks else None
        self.trees = [tree(kind, n, rng) for n in nq]
        self.parents = None if kind is None else ints([p for t in self.trees for p in t])
        self.scale = D ** -0.5

    def call(self, **changed):
        args = dict(scale=self.scale, window=self.window, first=self.first, sinks=self.s,
                    k_scale=self.ks, v_scale=self.vs, return_lse=True)
        args.update(changed)
        return mxq.paged_attention_tree(self.q, self.kc, self.vc, self.table, ints(self.lens),
                                        cumulated(self.nq), self.parents, **args)

    def reference(self):
        H, KV, page = self.H, self.KV, self.page
        res, a = [], 0
        for b, (m, n) in enumerate(zip(self.nq, self.lens)):
            if m == 0:
                continue
            seen = visible(self.trees[b], n, self.window, self.first)
            j = torch.arange(n, device="cuda")
            at = ints(self.rows[b]).long()[j // page]
            rows = []
            for h in range(H):
                kv = h // (H // KV)
                k, v = self.kc[at, j % page, kv].double(), self.vc[at, j % page, kv].double()
                if self.fp8:
                    k, v = k * self.ks[kv].double(), v * self.vs[kv].double()
                rows.append(attend(self.q[a:a + m, h], k, v, seen, self.scale,
                                   None if self.s is None else self.s[h], self.fp8))
            res.append([torch.stack([r[i] for r in rows], 1) for i in range(4)])
            a += m
        return [torch.cat([r[i] for r in res]) for i in range(4)]

    def check(self):
        ref = self.reference()
        out, lse = self.call()
        mxq.sync_status()
        assert_within(out, ref[0], ref[2], "out")
        assert_within(lse, ref[1], ref[3], "lse")
        return out, lse


SHAPES = [([1], [1]), ([1], [500]), ([7], [7]), ([16], [127]), ([16], [128]), ([16], [129]),
          ([33], [300]), ([64], [1000]), ([1, 5, 0, 17], [40, 5, 9, 600]), ([100], [100]),
          ([130, 3], [700, 3])]


@pytest.mark.parametrize("nq,lens", SHAPES)
@pytest.mark.parametrize("kind", [None, "random", "star"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_lengths(nq, lens, kind, D, fp8):
    Case(nq, lens, 4, 2, D, kind=kind, fp8=fp8).check()


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 3), (6, 2), (8, 1), (5, 1), (7, 1), (16, 2), (20, 1),
                                  (64, 1), (100, 1), (128, 1), (64, 64), (80, 40)])
@pytest.mark.parametrize("fp8", [False, True])
def test_groups(H, KV, fp8):
    Case([20, 3, 51], [300, 3, 77], H, KV, 64, fp8=fp8, seed=1).check()
    Case([9, 40], [150, 257], H, KV, 128, fp8=fp8, seed=2, sinks=True).check()


@pytest.mark.parametrize("page", [1, 3, 24, 64, 100, 128, 1000])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("fp8", [False, True])
def test_pages(page, layout, fp8):
    Case([12, 30, 1], [700, 31, 90], 8, 2, 128, page, fp8=fp8, layout=layout, seed=3).check()
    Case([12, 30, 1], [700, 31, 90], 6, 3, 64, page, fp8=fp8, layout=layout, seed=4).check()


@pytest.mark.parametrize("window,first", [(1, 0), (3, 0), (16, 4), (100, 0), (128, 128), (200, 33),
                                          (50, 700), (1000, 5), (260, 130)])
@pytest.mark.parametrize("kind", [None, "random", "binary"])
@pytest.mark.parametrize("fp8", [False, True])
def test_windows(window, first, kind, fp8):
    Case([20, 64, 2, 150], [900, 64, 400, 700], 4, 1, 64, kind=kind, window=window, first=first,
         fp8=fp8, seed=5).check()
    Case([33, 5], [1500, 140], 4, 2, 128, kind=kind, window=window, first=first, fp8=fp8, seed=6,
         sinks=True).check()


@pytest.mark.parametrize("nq,lens,H,KV,D", [
    ([16], [20000], 8, 2, 128), ([40, 3], [9000, 12000], 32, 8, 64), ([300], [5000], 8, 1, 128),
    ([2] * 70, [150 + 40 * i for i in range(70)], 4, 4, 128),
    ([64] * 5, [3000, 100, 64, 2000, 700], 64, 8, 128),
    ([1] * 400, [1 + i % 97 for i in range(400)], 2, 1, 64),
    ([700], [2500], 16, 2, 64), ([5, 9], [300, 140], 200, 200, 64),
    ([4100, 30], [4500, 3000], 2, 1, 64)])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_and_many(nq, lens, H, KV, D, fp8):
    Case(nq, lens, H, KV, D, 16, fp8=fp8, seed=7).check()


def test_many_sequences():
    """More than threads: 3000 sequences."""
    n = 3000
    Case([i % 3 for i in range(n)], [i % 3 + i % 40 for i in range(n)], 1, 1, 64, 8, seed=8).check()


def test_chunk_agrees_with_prompts_and_one_row_with_decode():
    c = Case([150, 64], [700, 64], 8, 2, 128, 128, kind=None, seed=9)
    out, lse = c.check()
    # the packed keys of attention_varlen
    j = [torch.arange(n, device="cuda") for n in c.lens]
    k, v = (torch.cat([t[ints(r).long()[i // 128], i % 128] for r, i in zip(c.rows, j)])
            for t in (c.kc, c.vc))
    other, _ = mxq.attention_varlen(c.q, k, v, cumulated(c.nq), cumulated(c.lens), return_lse=True)
    ref = c.reference()
    assert_within(other, ref[0], ref[2], "prompt")
    c = Case([1, 1, 1], [300, 1, 77], 8, 2, 64, seed=10)
    ref = c.reference()
    other = mxq.paged_attention_decode(c.q, c.kc, c.vc, c.table, ints(c.lens))
    assert_within(c.check()[0], ref[0], ref[2], "tree")
    assert_within(other, ref[0], ref[2], "decode")


@pytest.mark.parametrize("fp8", [False, True])
def test_what_unseen_places_hold(fp8):
    """NaN behind the lengths, in other pages, and in what a window hides from every row."""
    c = Case([12, 3], [900, 140], 8, 2, 128, 16, window=100, first=20, fp8=fp8, seed=11)
    want = c.check()
    for cache in (c.kc, c.vc):
        raw = cache.view(torch.uint8) if fp8 else cache
        bad = 0x7f if fp8 else NAN
        mark = torch.ones(raw.shape[:2], dtype=torch.bool, device="cuda")
        for r, n, m in zip(c.rows, c.lens, c.nq):
            j = torch.arange(n, device="cuda")
            seen = (j < 20) | (j > n - m - 100)
            mark[ints(r).long()[j[seen] // 16], j[seen] % 16] = False
        raw[mark] = bad
    # and the pages of what the windows hide are freed
    for b, (n, m) in enumerate(zip(c.lens, c.nq)):
        for i in range(len(c.rows[b])):
            if i * 16 >= 20 and (i + 1) * 16 <= n - m - 100:
                c.table[b, i] = -1
    got = c.call()
    mxq.sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_what_is_seen_shows():
    """A NaN key, value or query that a row sees makes that row NaN, and no row of another
    sequence."""
    for what in range(3):
        for fp8 in (False, True):
            c = Case([4, 4], [300, 200], 4, 2, 64, kind="chain", fp8=fp8, seed=12)
            want, _ = c.call()
            if what < 2:
                t = (c.kc, c.vc)[what]
                raw = t.view(torch.uint8) if fp8 else t
                raw[c.rows[0][2], 3, 1, 5] = 0x7f if fp8 else NAN
            else:
                c.q[1, 2] = NAN
            out, lse = c.call()
            mxq.sync_status()
            assert torch.equal(out[4:], want[4:]) and torch.equal(out[:, :2], want[:, :2])
            if what == 0:
                assert bool(torch.isnan(out[:4, 2:]).all()) and bool(torch.isnan(lse[:4, 2:]).all())
            elif what == 1:
                assert bool(torch.isnan(out[:4, 2:, 5]).all())
            else:
                assert bool(torch.isnan(out[1, 2]).all()) and bool(torch.isnan(lse[1, 2]))
                assert torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e4])
@pytest.mark.parametrize("fp8", [False, True])
def test_scales_and_large_scores(scale, fp8):
    """Rows whose scores are all alike, and rows that one key wins."""
    c = Case([10], [400], 4, 2, 64, fp8=fp8, seed=13)
    c.scale = scale
    ref = c.reference()
    out, lse = c.call()
    # a score's error grows with the score: at 1e4 only the winner is compared
    if scale <= 1:
        assert_within(out, ref[0], ref[2], "out")
        assert_within(lse, ref[1], ref[3], "lse")
    else:
        assert_within(lse, ref[1], ref[3], "lse")
        assert bool(torch.isfinite(out).all())


def test_key_scales_of_zero_and_below():
    c = Case([5], [200], 4, 2, 64, fp8=True, seed=14)
    c.ks = torch.tensor([0.0, -0.02], device="cuda")
    c.check()
    c.ks = torch.tensor([NAN, 0.01], device="cuda")
    out, lse = c.call()
    assert bool(torch.isnan(out[:, :2]).all()) and bool(torch.isfinite(out[:, 2:]).all())


def test_strides_and_given_outputs():
    c = Case([9, 20], [130, 400], 8, 2, 64, 16, seed=15)
    want, wl = c.call()
    qkv = randn(c.g, 29, 12, 64)
    qkv[:, :8] = c.q
    big = torch.full((29, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[..., 64:]
    c.q = qkv[:, :8]
    t = torch.full((2, 60), 12345678, dtype=torch.int32, device="cuda")
    t[:, :c.table.shape[1]] = c.table
    c.table = t[:, :c.table.shape[1]]
    ws = torch.full((mxq.paged_attention_tree_workspace_size(29, 2, 8, 2, 64) + 256,), 255,
                    dtype=torch.uint8, device="cuda")
    got, gl = c.call(out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want) and torch.equal(gl, wl)
    assert bool((big[..., :64] == 7).all())


def test_caches_past_32_bits():
    """Pages whose offsets pass 2^31 elements."""
    g = gen(16)
    pages, page, KV, D = 150000, 16, 8, 128                     # 2.4e9 elements each
    kc = torch.empty(pages, page, KV, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    used = [149999, 3, 140001, 131080]
    for p in used:
        kc[p], vc[p] = randn(g, page, KV, D), randn(g, page, KV, D)
    c = Case([4], [60], 8, 8, 128, 16, seed=17)
    c.kc, c.vc, c.rows, c.table = kc, vc, [used], ints([used])
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_input_is_left_out_and_reported(fp8):
    c = Case([4, 3, 5, 2], [100, 50, 90, 40], 4, 2, 64, fp8=fp8, kind="chain", seed=18)
    want, _ = c.call()
    mxq.sync_status()

    def reported(**changed):
        out = torch.full_like(c.q, 5.0)
        got, lse = c.call(out=out, **changed)
        with pytest.raises(mxq.MxqError) as e:
            mxq.sync_status()
        assert e.value.status == _lib.ERR_DEVICE
        return got

    # fewer keys than rows, a length past the table
    lens = c.lens
    c.lens = [100, 2, 90, 40]
    got = reported()
    assert bool((got[4:7] == 5).all())
    assert torch.equal(got[:4], want[:4]) and torch.equal(got[7:], want[7:])
    c.lens = [100, 50, 90, 40 + 10 * 16 * 7]
    got = reported()
    assert torch.equal(got[:12], want[:12])
    c.lens = [100, 50, 90, -7]
    assert torch.equal(reported()[:12], want[:12])
    c.lens = lens
    # parents that are no earlier rows count as none
    keep = c.parents.clone()
    for bad in (1, 3, 99, -2, 1 << 30):
        c.parents[1] = bad
        got = reported()
        c.parents[1] = -1
        assert torch.equal(got, c.call()[0])
        c.parents.copy_(keep)
    # a page outside the cache: its keys are not seen
    t = c.table.clone()
    for bad in (-1, 1 << 30, c.kc.shape[0]):
        c.table[0, 2] = bad
        got = reported()
        c.table.copy_(t)
        assert torch.equal(got[4:], want[4:]) and not torch.equal(got[:4], want[:4])
        assert bool(torch.isfinite(got).all())
    # offsets that run backwards or leave the rows
    mxq.sync_status()
    for cu in ([0, 4, 3, 12, 14], [0, 4, 7, 12, 99], [-3, 4, 7, 12, 14]):
        out = torch.full_like(c.q, 5.0)
        mxq.paged_attention_tree(c.q, c.kc, c.vc, c.table, ints(c.lens), ints(cu), c.parents,
                                 k_scale=c.ks, v_scale=c.vs, out=out)
        with pytest.raises(mxq.MxqError):
            mxq.sync_status()


def test_rows_outside_every_sequence_stay():
    c = Case([4, 3], [100, 50], 4, 2, 64, kind=None, seed=19)
    want, _ = c.call()
    c.q = torch.cat([randn(c.g, 2, 4, 64), c.q, randn(c.g, 5, 4, 64)])
    out = torch.full_like(c.q, 5.0)
    mxq.paged_attention_tree(c.q, c.kc, c.vc, c.table, ints(c.lens), ints([2, 6, 9]), out=out)
    mxq.sync_status()
    assert torch.equal(out[2:9], want)
    assert bool((out[:2] == 5).all()) and bool((out[9:] == 5).all())


def test_sequences_without_keys_or_a_table():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    table = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    mxq.paged_attention_tree(q, kc, kc, table, ints([0, 0]), ints([0, 0, 0]), out=out)
    mxq.sync_status()
    assert bool((out == 5).all())


def test_empty_calls():
    c = Case([0, 0], [5, 0], 4, 2, 64)
    assert c.call()[0].shape == (0, 4, 64)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    out = mxq.paged_attention_tree(c.q, c.kc, c.vc, c.table[:0], e, ints([0]))
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_repeat_bit_for_bit_on_two_streams_and_in_graphs(fp8):
    a = Case([16, 40, 3], [5000, 900, 60], 8, 2, 128, fp8=fp8, seed=20)
    b = Case([5], [3000], 8, 4, 64, fp8=fp8, seed=21, window=500, first=9)
    wa, wb = a.call()[0], b.call()[0]
    torch.cuda.synchronize()
    ins = [(x, ints(x.lens), cumulated(x.nq)) for x in (a, b)]

    def run(i):
        x, n, cu = ins[i]
        return mxq.paged_attention_tree(x.q, x.kc, x.vc, x.table, n, cu, x.parents,
                                        window=x.window, first=x.first, k_scale=x.ks,
                                        v_scale=x.vs)

    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(run(i))
    torch.cuda.synchronize()
    for i, w in enumerate((wa, wb)):
        assert all(torch.equal(o, w) for o in outs[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ga, gb, ga2 = run(0), run(1), run(0)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb) and torch.equal(ga2, wa)


def test_a_verified_tree_end_to_end():
    """Append a tree's rows, attend, keep the accepted path, compact, cut off the rest, and
    decode the next token: as if only the accepted tokens had been appended."""
    g, rng = gen(22), random.Random(22)
    B, H, KV, D, page, width, pages = 3, 8, 2, 64, 4, 20, 100
    lens, drafts = [17, 4, 30], 9
    kc = torch.zeros(pages, page, KV, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    zero, n0 = ints([0] * B), ints(lens)
    mxq.cache_resize(table, zero, n0, refs, page)

    def slots(b, positions):
        p = torch.tensor(positions, device="cuda")
        return table[b].long()[p // page] * page + p % page

    context = [(randn(g, n, KV, D), randn(g, n, KV, D)) for n in lens]
    for b, (k, v) in enumerate(context):
        mxq.rope_append_kv(k, v, kc, vc, slots(b, list(range(lens[b]))))
    n1 = n0 + drafts
    mxq.cache_resize(table, n0, n1, refs, page)
    k, v, q = randn(g, B * drafts, KV, D), randn(g, B * drafts, KV, D), randn(g, B * drafts, H, D)
    at = torch.cat([slots(b, list(range(lens[b], lens[b] + drafts))) for b in range(B)])
    mxq.rope_append_kv(k, v, kc, vc, at)
    trees = [tree("random", drafts, rng) for _ in range(B)]
    out = mxq.paged_attention_tree(q, kc, vc, table, n1, ints([0, 9, 18, 27]),
                                   ints([p for t in trees for p in t]))
    # the path of the last row is accepted
    paths = []
    for t in trees:
        path, i = [], drafts - 1
        while i >= 0:
            path.insert(0, i)
            i = t[i]
        paths.append(path)
    most = max(len(p) for p in paths)
    kept = ints([p + [0] * (most - len(p)) for p in paths])
    counts = ints([len(p) for p in paths])
    mxq.cache_compact(kc, vc, table, n0, kept, counts)
    n2 = n0 + counts
    mxq.cache_resize(table, n1, n2, refs, page)
    got = mxq.paged_attention_decode(q[[8, 17, 26]], kc, vc, table, n2)
    mxq.sync_status()
    assert int(refs.sum()) == sum(-(-n // page) for n in n2.tolist())
    for b, path in enumerate(paths):
        rows = torch.tensor(path, device="cuda") + 9 * b
        kk, vv = torch.cat([context[b][0], k[rows]]), torch.cat([context[b][1], v[rows]])
        seen = torch.ones(1, len(kk), dtype=torch.bool, device="cuda")
        for h in range(H):
            r = attend(q[9 * b + 8:9 * b + 9, h], kk[:, h // 4], vv[:, h // 4], seen, D ** -0.5)
            assert_within(got[b:b + 1, h], r[0], r[2], "decode")
            assert_within(out[9 * b + 8:9 * b + 9, h], r[0], r[2], "tree")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nq,lens", [([16], [3000]), ([64, 3], [500, 40])])
def test_stalled_loads_time_out_and_recover(nq, lens, fp8):
    """With the test-only switch nothing is loaded: every wait runs out, the status
    says so, and the next call is right."""
    c = Case(nq, lens, 8, 2, 128, fp8=fp8, seed=23)
    mxq.sync_status()
    old = mxq.get_option(_lib.OPT_WAIT_BUDGET_NS)
    try:
        mxq.set_option(_lib.OPT_WAIT_BUDGET_NS, 20_000_000)
        mxq.set_option(_lib.OPT_INJECT_STALL, 1)
        c.call()
        with pytest.raises(mxq.MxqError) as e:
            mxq.sync_status()
        assert e.value.status == _lib.ERR_TIMEOUT
    finally:
        mxq.set_option(_lib.OPT_INJECT_STALL, 0)
        mxq.set_option(_lib.OPT_WAIT_BUDGET_NS, old)
    c.check()


def test_pages_further_apart_than_64_gib():
    """Pages of keys and of values by turns, 2^30 bytes from one of the keys to the next."""
    page, KV, pages = 24, 2, 67
    buffer = torch.empty(pages << 30, dtype=torch.uint8, device="cuda")
    for dtype in (torch.bfloat16, FP8):
        flat = buffer.view(dtype)
        size = flat.element_size()
        for D, nq, lens in ((128, 16, 60), (128, 40, 300), (64, 5, 301)):
            c = Case([nq], [lens], 8, KV, D, page, seed=71, fp8=dtype == FP8)
            kc, vc = (flat.as_strided((pages, page, KV, D), ((1 << 30) // size, KV * D, D, 1),
                                      half * (1 << 29) // size) for half in range(2))
            used = [66, 0, 65, 64, 1, 63, 59, 8, 33, 2, 3, 4, 62][:-(-lens // page)]
            for mine, theirs in zip(used, c.rows[0]):
                kc[mine], vc[mine] = c.kc[theirs], c.vc[theirs]
            want, wl = c.call()
            c.table = ints([used])
            out, lse = mxq.paged_attention_tree(
                c.q, kc, vc, c.table, ints([lens]), cumulated([nq]), c.parents, scale=c.scale,
                k_scale=c.ks, v_scale=c.vs, return_lse=True)
            mxq.sync_status()
            assert torch.equal(out, want) and torch.equal(lse, wl)
    del buffer, flat, kc, vc
    torch.cuda.empty_cache()

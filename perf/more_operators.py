"""Workloads of the paged cache's further operators: attention of drafted token trees over
the cache, windows whose first keys stay visible, and the cache's pages (forked, copied,
taken, freed, compacted).

`listed()` gives the fixed cases, `draw()` further ones of the same ranges.
With `own` false, `run` computes an operator from elementary torch operations
in 32 bits, rounded once at the end; with `own` true it calls the package.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def _tree(name, batch, shortest, longest, drafts, heads, kv_heads, dim, page, cache="bf16",
          tree=True, window=0, first=0, sinks=False, lse=False, lens_seed=1):
    return {"name": name, "op": "tree", "batch": batch, "shortest": shortest, "longest": longest,
            "drafts": drafts, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "cache": cache, "tree": tree, "window": window, "first": first, "sinks": sinks,
            "lse": lse, "lens_seed": lens_seed}


def _decode(name, batch, shortest, longest, heads, kv_heads, dim, page, window, first,
            cache="bf16", sinks=False, lse=False, lens_seed=1):
    return {"name": name, "op": "decode", "batch": batch, "shortest": shortest,
            "longest": longest, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "cache": cache, "window": window, "first": first, "sinks": sinks, "lse": lse,
            "lens_seed": lens_seed}


def _prompt(name, batch, tokens, heads, kv_heads, dim, window, first, history=0, sinks=False,
            lse=False, lens_seed=1):
    return {"name": name, "op": "prompt", "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "window": window, "first": first,
            "history": history, "sinks": sinks, "lse": lse, "lens_seed": lens_seed}


def _beams(name, groups, beams, shared, grown, kv_heads, dim, page, window=0, first=0,
           lens_seed=1):
    return {"name": name, "op": "beams", "groups": groups, "beams": beams, "shared": shared,
            "grown": grown, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "first": first, "lens_seed": lens_seed}


def _compact(name, batch, shortest, longest, tail, kept, kv_heads, dim, page, lens_seed=1):
    return {"name": name, "op": "compact", "batch": batch, "shortest": shortest,
            "longest": longest, "tail": tail, "kept": kept, "kv_heads": kv_heads, "dim": dim,
            "page": page, "lens_seed": lens_seed}


def listed():
    return [
        # one user's drafted tree over a short conversation: latency counts
        _tree("tree_one_1500", 1, 1500, 1500, 16, 32, 8, 128, 16),
        # a full server: 64 conversations of a few tokens to 8192, each with a tree
        _tree("tree_64_ragged_8192", 64, 5, 8192, 32, 32, 8, 128, 64),
        # long documents in an FP8 cache, large trees, the log-sum-exp kept
        _tree("tree_16_long_fp8", 16, 9000, 32768, 48, 64, 8, 128, 128, cache="e4m3", lse=True),
        # chunks of two prompts over the paged cache: no tree, a window with first keys, sinks
        _tree("tree_chunk_window", 2, 6000, 8192, 300, 64, 8, 64, 24, tree=False, window=1024,
              first=4, sinks=True),
        # one long-running conversation in a streaming layer: latency counts
        _decode("decode_one_first", 1, 20000, 20000, 32, 8, 128, 16, 1024, 4),
        # many conversations, wide windows, a system prompt that stays visible
        _decode("decode_96_first", 96, 1, 16384, 32, 8, 128, 64, 2048, 100, sinks=True),
        # a short prompt past its window: latency counts
        _prompt("prompt_first_700", 1, 700, 32, 8, 128, 256, 4),
        # packed prompts in a streaming layer
        _prompt("prompt_first_8192", 5, 8192, 32, 8, 128, 1024, 16, lse=True),
        # one step of a small beam search: fork, copy the open pages, make room
        _beams("beams_2x4", 2, 4, 300, 50, 8, 128, 16),
        # one step of a large one, streaming: what the window left behind is freed
        _beams("beams_64x4", 64, 4, 1500, 500, 8, 128, 64, window=1024, first=64),
        # the accepted tokens of 64 verified trees close up
        _compact("compact_accepted_64", 64, 40, 4096, 32, 6, 8, 128, 64),
        # half of eight long conversations' keys evicted
        _compact("compact_evict_8", 8, 9000, 16384, 0, 4096, 8, 128, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "decode", "prompt", "beams", "compact"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([1, 16, 24, 64, 128])
    seed = rng.randrange(1 << 20)
    if op == "tree":
        longest = _log(rng, 40, 32768)
        drafts = _log(rng, 1, min(longest, 300))
        room = max(1, (1 << 18) // longest)
        batch = _log(rng, 1, max(1, min(128, room, (1 << 23) // (longest * drafts))))
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        c = _tree("", batch, max(drafts, int(longest * rng.random())), longest, drafts, heads, kv,
                  dim, page, rng.choice(["bf16", "e4m3"]), rng.random() < 0.8, window,
                  rng.choice([0, 4, _log(rng, 1, 300)]) if window else 0, rng.random() < 0.3,
                  rng.random() < 0.3, seed)
    elif op == "decode":
        longest = _log(rng, 1, 32768)
        batch = _log(rng, 1, max(1, min(256, (1 << 18) // longest)))
        c = _decode("", batch, max(1, int(longest * rng.random())), longest, heads, kv, dim, page,
                    _log(rng, 1, 4096), _log(rng, 1, 1000), rng.choice(["bf16", "e4m3"]),
                    rng.random() < 0.3, rng.random() < 0.3, seed)
    elif op == "prompt":
        tokens = _log(rng, 1, 8192 if heads <= 32 else 4096)
        batch = _log(rng, 1, max(1, min(64, tokens)))
        history = rng.choice([0, 0, _log(rng, 1, 4096)])
        if (tokens + batch * history) * tokens * heads > 8192 * 8192 * 16:
            history = 0
        c = _prompt("", batch, tokens, heads, kv, dim, _log(rng, 1, 2048), _log(rng, 1, 300),
                    history, rng.random() < 0.3, rng.random() < 0.3, seed)
    elif op == "beams":
        beams = rng.choice([1, 2, 3, 4, 5, 8])
        window = rng.choice([0, _log(rng, 1, 2048)])
        c = _beams("", _log(rng, 1, 256 // beams), beams, _log(rng, 1, 1500), _log(rng, 1, 500),
                   kv, dim, page, window, _log(rng, 1, 100) if window else 0, seed)
    else:
        longest = _log(rng, 2, 16384)
        batch = _log(rng, 1, max(1, min(128, (1 << 17) // longest)))
        tail = rng.choice([0, _log(rng, 1, min(longest, 64))])
        c = _compact("", batch, max(1, tail, int(longest * rng.random())), longest, tail,
                     _log(rng, 1, tail or max(1, longest // 2)), kv, dim, page, seed)
    del c["name"]
    return c


# Lengths and trees are part of the case: its work depends on them.

def _lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["shortest"], case["longest"]) for _ in range(case["batch"])]


def _drafts(case, lens):
    """The number of drafted tokens of each sequence, and each one's parent among them."""
    r = random.Random(case["lens_seed"] + 1)
    most = [min(case["drafts"], n) for n in lens]
    counts = [r.randint((n + 1) // 2, n) for n in most]
    parents = []
    for n in counts:
        # a tree as drafting makes it: a token continues one of the last few, or the context
        parents.append([r.randint(max(-1, i - 6), i - 1) for i in range(n)] if case["tree"]
                       else list(range(-1, n - 1)))
    return counts, parents


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _prompt_lens(case):
    """Query lengths (their sum is `tokens`) and key lengths of the packed sequences."""
    r = random.Random(case["lens_seed"])
    w = [r.random() ** 2 + 0.02 for _ in range(case["batch"])]
    spare = case["tokens"] - case["batch"]
    q = [1 + int(spare * x / sum(w)) for x in w]
    q[-1] += case["tokens"] - sum(q)
    return q, [n + case["history"] for n in q]


def _beam_lens(case):
    """Per group: tokens of the shared prompt, tokens that each beam holds behind it."""
    r = random.Random(case["lens_seed"])
    lo = lambda n: max(1, n // 2)
    return [(r.randint(lo(case["shared"]), case["shared"]),
             r.randint(lo(case["grown"]), case["grown"])) for _ in range(case["groups"])]


def _kept(case, lens):
    """Start of the compacted tail of each sequence and how many of its rows stay."""
    r = random.Random(case["lens_seed"] + 1)
    starts = [max(0, n - case["tail"]) if case["tail"] else 0 for n in lens]
    return starts, [r.randint(0, min(case["kept"], n - s)) if case["tail"]
                    else min(case["kept"], n - s) for n, s in zip(lens, starts)]


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _ints(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def _pool(case, pages, g):
    """A cache [pages, page, kv_heads, dim] that already holds values."""
    t = _randn(g, pages, case["page"], case["kv_heads"], case["dim"])
    if case.get("cache") == "e4m3":
        t = (t.float() * 100).clamp(-448, 448).to(FP8)
    return t


def _kv_scales(case, g):
    """Per-head scales of an FP8 cache: what a unit-variance head needs, about 1/100."""
    if case.get("cache") != "e4m3":
        return None, None
    h = case["kv_heads"]
    return tuple(0.008 + 0.004 * torch.rand(h, generator=g, device="cuda") for _ in range(2))


def _paged(s, case, lens, g):
    """The caches and the page table of sequences of these lengths, pages in any order."""
    need = [-(-n // case["page"]) for n in lens]
    width, total = max(need), sum(need)
    s["k_cache"], s["v_cache"] = _pool(case, total, g), _pool(case, total, g)
    s["k_scale"], s["v_scale"] = _kv_scales(case, g)
    where = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    at = (torch.cumsum(n, 0) - n)[:, None] + torch.arange(width, device="cuda")
    have = torch.arange(width, device="cuda") < n[:, None]
    s["page_table"] = torch.where(have, where[at.clamp(max=total - 1)], 0)
    s["seq_lens"] = _ints(lens)


def _cumulated(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return _ints(c)


def prepare(case, seed):
    g = _gen(seed)
    KV, D = case["kv_heads"], case["dim"]
    s = {"case": case}
    if case["op"] == "beams":
        return _prepare_beams(s, case, g)
    if case["op"] == "compact":
        lens = _lens(case)
        _paged(s, case, lens, g)
        starts, counts = _kept(case, lens)
        s["starts"], s["counts"] = _ints(starts), _ints(counts)
        most = max(1, max(counts))
        s["kept"] = torch.zeros(len(lens), most, dtype=torch.int32, device="cuda")
        for b, (n, a, c) in enumerate(zip(lens, starts, counts)):
            s["kept"][b, :c] = torch.randperm(n - a, generator=g, device="cuda")[:c].sort()[0]
        return s
    H = case["heads"]
    if case["op"] == "tree":
        lens = _lens(case)
        counts, parents = _drafts(case, lens)
        _paged(s, case, lens, g)
        s["q"] = _randn(g, sum(counts), H, D)
        s["cu_q"] = _cumulated(counts)
        s["parents"] = _ints([p for t in parents for p in t]) if case["tree"] else None
    elif case["op"] == "decode":
        lens = _lens(case)
        _paged(s, case, lens, g)
        s["q"] = _randn(g, len(lens), H, D)
    else:
        nq, nk = _prompt_lens(case)
        Tq, Tk = sum(nq), sum(nk)
        if Tq == Tk:
            qkv = _randn(g, Tq, (H + 2 * KV) * D)       # the QKV linear's output
            s["q"] = qkv[:, :H * D].view(Tq, H, D)
            s["k"] = qkv[:, H * D:(H + KV) * D].view(Tq, KV, D)
            s["v"] = qkv[:, (H + KV) * D:].view(Tq, KV, D)
        else:
            s["q"] = _randn(g, Tq, H, D)
            s["k"], s["v"] = _randn(g, Tk, KV, D), _randn(g, Tk, KV, D)
        s["cu_q"], s["cu_k"] = _cumulated(nq), _cumulated(nk)
    s["sinks"] = torch.randn(H, generator=g, device="cuda") if case["sinks"] else None
    # the scratch that a serving loop keeps for its calls
    s["workspace"] = torch.empty(96 << 20, dtype=torch.uint8, device="cuda")
    return s


def _prepare_beams(s, case, g):
    P, beams = case["page"], case["beams"]
    groups = _beam_lens(case)
    rows, lens, used = [], [], 0
    for shared, grown in groups:
        # full pages of the prompt are shared, the rest is each beam's own
        full = shared // P
        own_pages = -(-(shared + grown) // P) - full
        for b in range(beams):
            rows.append(list(range(used, used + full)) +
                        list(range(used + full + b * own_pages, used + full + (b + 1) * own_pages)))
            lens.append(shared + grown)
        used += full + beams * own_pages
    width = max(len(r) for r in rows) + 1
    pages = used + 2 * len(rows) + 5                     # some are free
    s["k_cache"], s["v_cache"] = _pool(case, pages, g), _pool(case, pages, g)
    where = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = _ints([r + [-1] * (width - len(r)) for r in rows])
    table = torch.where(table < 0, -1, where[table.clamp(min=0).long()])
    if case["window"]:
        # earlier steps freed what the window had left behind
        i = torch.arange(width, device="cuda")
        n = _ints(lens)[:, None]
        table[((i + 1) * P <= n - case["window"]) & (i * P >= case["first"])] = -1
    s["table"], s["lens"] = table, _ints(lens)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    held = table[table >= 0].long()
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    s["refs_before"], s["refs"] = refs, refs.clone()
    pick = torch.randint(0, beams, (len(groups), beams), generator=g, device="cuda")
    base = torch.arange(len(groups), device="cuda")[:, None] * beams
    s["parents"] = (base + pick).flatten().to(torch.int32)
    return s


# ------------------------------------------------------------- the plain forms

def _softmax_v(x, mask, sinks, v, lse):
    """x [..., queries, keys] scores, mask the visible ones (None: x is masked), v [..., keys, dim],
    sinks [..., 1, 1] or None: softmax over the keys (a row that sees none gives 0) times v."""
    if mask is not None:
        x = x.masked_fill_(~mask, -math.inf)
    m = x.amax(-1, keepdim=True)
    if sinks is not None:
        m = torch.maximum(m, sinks)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    n = p.sum(-1, keepdim=True)
    if sinks is not None:
        n = n + (sinks - m).exp()
    out = torch.matmul(p, v) / torch.where(n == 0, 1.0, n)
    return out, (m + n.log()).squeeze(-1) if lse else None


def _gathered(s):
    """Keys and values of the page table's rows [B, KV, keys, D] in 32 bits."""
    pages = s["page_table"].long()
    k, v = (t[pages].flatten(1, 2).permute(0, 2, 1, 3).float()
            for t in (s["k_cache"], s["v_cache"]))
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    return k, v


def _plain_tree(s):
    c, q = s["case"], s["q"]
    T, H, D = q.shape
    KV, dev = c["kv_heads"], q.device
    G = H // KV
    cu = s["cu_q"].long()
    counts = cu[1:] - cu[:-1]
    B, N = counts.shape[0], c["drafts"]
    i = torch.arange(T, device=dev)
    b = (i[:, None] >= cu[1:]).sum(1)
    at = i - cu[b]                                        # the row within its sequence
    parents = at - 1 if s["parents"] is None else s["parents"].long()
    # the path of every row: its drafts, and how many steps up each is
    path = torch.full((T, N + 1), -1, device=dev)         # a column more for "past the root"
    up, steps = at.clone(), torch.zeros_like(at)
    for _ in range(N):
        path.scatter_(1, torch.where(up >= 0, up, N)[:, None], steps[:, None])
        steps = steps + (up >= 0)
        up = torch.where(up >= 0, parents[(cu[b] + up).clamp(max=T - 1)], -1)
    path, depth = path[:, :N], steps[:, None] - 1
    k, v = _gathered(s)
    keys = k.shape[2]
    before = (s["seq_lens"].long() - counts)[b][:, None]  # keys of the context
    j = torch.arange(keys, device=dev)
    d = j - before                                        # the draft at a key
    on = torch.where((d >= 0) & (d < counts[b][:, None]),
                     path.gather(1, d.clamp(0, N - 1)), -1)
    if c["window"]:
        old = (j < before) & ((j > before + depth - c["window"]) | (j < c["first"]))
        new = (on >= 0) & ((on < c["window"]) | (before + depth - on < c["first"]))
    else:
        old, new = j < before, on >= 0
    mask = torch.zeros(B, N, keys, dtype=torch.bool, device=dev)
    mask[b, at] = old | new
    qf = torch.zeros(B, N, H, D, device=dev)
    qf[b, at] = q.float() * D ** -0.5
    qf = qf.view(B, N, KV, G, D).permute(0, 2, 3, 1, 4).reshape(B, KV, G * N, D)
    x = torch.matmul(qf, k.transpose(-1, -2))
    x.view(B, KV, G, N, keys).masked_fill_(~mask[:, None, None], -math.inf)
    sinks = None if s["sinks"] is None else \
        s["sinks"].view(KV, G, 1).expand(KV, G, N).reshape(KV, G * N, 1)
    out, lse = _softmax_v(x, None, sinks, v, c["lse"])
    out = out.view(B, KV, G, N, D).permute(0, 3, 1, 2, 4).reshape(B, N, H, D)
    out = out[b, at].to(torch.bfloat16)
    if not c["lse"]:
        return {"out": out}
    lse = lse.view(B, KV, G, N).permute(0, 3, 1, 2).reshape(B, N, H)
    return {"out": out, "lse": lse[b, at]}


def _plain_decode(s):
    c, q = s["case"], s["q"]
    B, H, D = q.shape
    KV = c["kv_heads"]
    k, v = _gathered(s)
    x = torch.matmul(q.float().view(B, KV, H // KV, D) * D ** -0.5, k.transpose(-1, -2))
    j = torch.arange(k.shape[2], device=q.device)
    n = s["seq_lens"][:, None]
    mask = (j < n) & ((j >= n - c["window"]) | (j < c["first"]))
    sinks = None if s["sinks"] is None else s["sinks"].view(KV, H // KV, 1)
    out, lse = _softmax_v(x, mask[:, None, None], sinks, v, c["lse"])
    out = out.reshape(B, H, D).to(torch.bfloat16)
    return {"out": out, "lse": lse.reshape(B, H)} if c["lse"] else {"out": out}


def _plain_prompt(s):
    c, q = s["case"], s["q"]
    Tq, H, D = q.shape
    KV, Tk = c["kv_heads"], s["k"].shape[0]
    i, j = torch.arange(Tq, device=q.device), torch.arange(Tk, device=q.device)
    qs = (i[:, None] >= s["cu_q"][1:]).sum(1)             # the sequence of each row and key
    ks = (j[:, None] >= s["cu_k"][1:]).sum(1)
    # positions counted in the packed keys; the last query stands at its last key
    at = (i - s["cu_q"][1:][qs] + s["cu_k"][1:][qs])[:, None]
    mask = (qs[:, None] == ks) & (j <= at)
    mask &= (j > at - c["window"]) | (j - s["cu_k"][ks] < c["first"])
    qf = q.float().view(Tq, KV, H // KV, D).permute(1, 2, 0, 3) * D ** -0.5
    k, v = (t.float().transpose(0, 1)[:, None] for t in (s["k"], s["v"]))   # [KV, 1, Tk, D]
    sinks = None if s["sinks"] is None else s["sinks"].view(KV, H // KV, 1, 1)
    out, lse = _softmax_v(torch.matmul(qf, k.transpose(-1, -2)), mask, sinks, v, c["lse"])
    out = out.permute(2, 0, 1, 3).reshape(Tq, H, D).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(2, 0, 1).reshape(Tq, H)} if c["lse"] else {"out": out}


def _plain_fork(table, lens, refs, parents, P):
    """A row of `table` for every parent: full pages shared, an open last page kept by the
    first child if nothing else holds it, and else given a fresh page to be copied into."""
    free = (refs == 0).nonzero().flatten()
    p = parents.long()
    B, width = table.shape
    new, n = table[p], lens[p].long()
    i = torch.arange(width, device=table.device)
    used = -(-n // P)
    new = torch.where(i < used[:, None], new, -1)
    open_rows = n % P                                     # tokens in the open page
    last = (used - 1).clamp(min=0)
    page = new.gather(1, last[:, None])[:, 0]
    has_open = (open_rows > 0) & (page >= 0)
    child = torch.arange(len(p), device=table.device)
    first = torch.full((B,), len(p), device=table.device).scatter_reduce_(0, p, child, "amin")
    keeps = has_open & (first[p] == child) & (refs[page.clamp(min=0).long()] == 1)
    wants = has_open & ~keeps
    fresh = free[(torch.cumsum(wants, 0) - 1).clamp(min=0)].to(torch.int32)
    new.scatter_(1, last[:, None], torch.where(wants, fresh, page)[:, None])
    new = torch.where(i < used[:, None], new, -1)
    copies = torch.where(wants[:, None], torch.stack([page, fresh, open_rows.int()], 1),
                         _ints([-1, -1, 0]))
    # what the old rows held goes, what the new ones hold comes
    held = -(-lens.long() // P)[:, None]
    gone = table[(i < held) & (table >= 0)].long()
    come = new[new >= 0].long()
    one = torch.ones((), dtype=torch.int32, device=table.device)
    refs.index_add_(0, gone, -one.expand(len(gone)))
    refs.index_add_(0, come, one.expand(len(come)))
    return new, lens[p], copies


def _plain_copy(k_cache, v_cache, copies):
    t = torch.arange(k_cache.shape[1], device=k_cache.device)
    move = (copies[:, :1] >= 0) & (t < copies[:, 2:])     # [pairs, tokens]
    pair, row = move.nonzero(as_tuple=True)
    src, dst = copies[pair, 0].long(), copies[pair, 1].long()
    for cache in (k_cache, v_cache):
        cache[dst, row] = cache[src, row]


def _plain_resize(table, lens, new_lens, refs, P, window, first):
    free = (refs == 0).nonzero().flatten()
    i = torch.arange(table.shape[1], device=table.device)
    n0, n1 = (-(-n.long() // P)[:, None] for n in (lens, new_lens))
    take = (i >= n0) & (i < n1)
    drop = (i >= n1) & (i < n0)
    if window:
        drop |= (i < torch.minimum(n0, n1)) & ((i + 1) * P <= new_lens[:, None] - window) & (
            i * P >= first)
    gone = table[drop & (table >= 0)].long()
    fresh = free[:int(take.sum())]
    table[drop] = -1
    table[take] = fresh.to(torch.int32)
    one = torch.ones((), dtype=torch.int32, device=table.device)
    refs.index_add_(0, gone, -one.expand(len(gone)))
    refs[fresh] = 1


def _plain_beams(s):
    c = s["case"]
    s["refs"].copy_(s["refs_before"])
    table, lens, copies = _plain_fork(s["table"], s["lens"], s["refs"], s["parents"], c["page"])
    _plain_copy(s["k_cache"], s["v_cache"], copies)
    _plain_resize(table, lens, lens + 1, s["refs"], c["page"], c["window"], c["first"])
    return {"table": table, "lens": lens, "copies": copies, "refs": s["refs"],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_compact(s):
    P, kept = s["case"]["page"], s["kept"].long()
    to = torch.arange(kept.shape[1], device=kept.device)
    b, i = (to < s["counts"][:, None]).nonzero(as_tuple=True)
    start = s["starts"].long()[b]
    src, dst = start + kept[b, i], start + i
    sp, dp = s["page_table"][b, src // P].long(), s["page_table"][b, dst // P].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[dp, dst % P] = cache[sp, src % P]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ----------------------------------------------------------- the package's calls

def _own(s):
    import mxfp4_quantized_gemm_token_gb300 as mxq
    c = s["case"]
    if c["op"] == "beams":
        s["refs"].copy_(s["refs_before"])
        table, lens, copies = mxq.cache_fork(s["table"], s["lens"], s["refs"], s["parents"],
                                             c["page"])
        mxq.cache_copy_pages(s["k_cache"], s["v_cache"], copies)
        mxq.cache_resize(table, lens, lens + 1, s["refs"], c["page"], window=c["window"],
                         first=c["first"])
        return {"table": table, "lens": lens, "copies": copies, "refs": s["refs"],
                "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "compact":
        mxq.cache_compact(s["k_cache"], s["v_cache"], s["page_table"], s["starts"], s["kept"],
                          s["counts"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "tree":
        r = mxq.paged_attention_tree(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                     s["seq_lens"], s["cu_q"], s["parents"], window=c["window"],
                                     first=c["first"], sinks=s["sinks"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"], return_lse=c["lse"],
                                     workspace=s["workspace"])
    elif c["op"] == "decode":
        r = mxq.paged_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                       s["seq_lens"], window=c["window"], sinks=s["sinks"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"],
                                       return_lse=c["lse"], workspace=s["workspace"],
                                       first=c["first"])
    else:
        r = mxq.attention_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                 window=c["window"], sinks=s["sinks"], return_lse=c["lse"],
                                 workspace=s["workspace"], first=c["first"])
    return {"out": r[0], "lse": r[1]} if c["lse"] else {"out": r}


def run(state):
    if own:
        return _own(state)
    return {"tree": _plain_tree, "decode": _plain_decode, "prompt": _plain_prompt,
            "beams": _plain_beams, "compact": _plain_compact}[state["case"]["op"]](state)


# ---------------------------------------------------------------------- the work

def _seen(n, window, first):
    """Keys that the row at position n - 1 sees."""
    return n if not window else min(n, window + min(first, max(0, n - window)))


def work(case):
    KV, D = case["kv_heads"], case["dim"]
    if case["op"] == "beams":
        P, rows = case["page"], case["groups"] * case["beams"]
        # in the mean (1 - 1/e) of the beams go on, the others' open pages are copied
        moved = sum(case["beams"] * ((a + n) % P) for a, n in _beam_lens(case)) / math.e
        table = sum(case["beams"] * -(-(a + n) // P) for a, n in _beam_lens(case))
        return {"bytes": int(2 * 2 * moved * KV * D * 2 + 4 * (2 * table + 6 * rows)), "flops": 0}
    if case["op"] == "compact":
        lens = _lens(case)
        _, counts = _kept(case, lens)
        return {"bytes": max(1, sum(counts)) * (2 * 2 * KV * D * 2 + 4), "flops": 0}
    H, one = case["heads"], 1 if case.get("cache") == "e4m3" else 2
    w, f = case["window"], case["first"]
    if case["op"] == "decode":
        seen = sum(_seen(n, w, f) for n in _lens(case))
        return {"bytes": 2 * seen * KV * D * one + case["batch"] * H * D * 4,
                "flops": 4 * seen * H * D}
    if case["op"] == "tree":
        lens = _lens(case)
        counts, parents = _drafts(case, lens)
        pairs = keys = 0
        for n, m, tree in zip(lens, counts, parents):
            d = _depths(tree)
            pairs += sum(_seen(n - m + x + 1, w, f) for x in d)
            keys += _seen(n - m, max(0, w - 1) if w else 0, f) + m if w else n
        return {"bytes": 2 * keys * KV * D * one + sum(counts) * H * D * 4,
                "flops": 4 * pairs * H * D}
    nq, nk = _prompt_lens(case)
    seen = sum(_seen(b - a + i + 1, w, f) for a, b in zip(nq, nk) for i in range(a))
    return {"bytes": 2 * D * (2 * H * sum(nq) + 2 * KV * sum(nk)), "flops": 4 * seen * H * D}


# --------------------------------------------------------------- the definition

def _rows64(q, k, v, visible, sinks, scale):
    """q [n, H, D], k, v [m, KV, D] in 64 bits, visible [n, m]: out [n, H, D], lse [n, H]."""
    H, KV = q.shape[1], k.shape[1]
    out, lse = torch.empty_like(q), q.new_empty(q.shape[:2])
    for h in range(H):
        x = (q[:, h] @ k[:, h // (H // KV)].T * scale).masked_fill(~visible, -math.inf)
        if sinks is not None:
            x = torch.cat([x, sinks[h].double().expand(len(x), 1)], 1)
        lse[:, h] = torch.logsumexp(x, 1)
        w = (x[:, :k.shape[0]] - lse[:, h:h + 1]).exp()
        out[:, h] = w @ v[:, h // (H // KV)]
    return out, lse


def _context(s, b, n):
    """The n keys and values of sequence b in 64 bits."""
    at = torch.arange(n, device="cuda")
    page, off = s["page_table"][b].long()[at // s["case"]["page"]], at % s["case"]["page"]
    k, v = s["k_cache"][page, off].double(), s["v_cache"][page, off].double()
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
    return k, v


def _exact_beams(s, case):
    """The step as loops over plain lists."""
    P, w, f = case["page"], case["window"], case["first"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    refs, parents = s["refs_before"].tolist(), s["parents"].tolist()
    before = list(refs)
    fresh = iter([p for p, n in enumerate(refs) if n == 0])
    for row, n in zip(table, lens):
        for p in row[:-(-n // P)]:
            if p >= 0:
                refs[p] -= 1
    new, copies, served = [], [], set()
    for r in parents:
        n = lens[r]
        row = table[r][:-(-n // P)]
        copy = [-1, -1, 0]
        if n % P and row[-1] >= 0:
            if before[row[-1]] > 1 or r in served:
                copy = [row[-1], next(fresh), n % P]
                row[-1] = copy[1]
        served.add(r)
        for p in row:
            if p >= 0:
                refs[p] += 1
        new.append(row)
        copies.append(copy)
    k, v = s["k_cache"].clone(), s["v_cache"].clone()
    for src, dst, n in copies:
        if src >= 0:
            k[dst, :n], v[dst, :n] = k[src, :n], v[src, :n]
    fresh = iter([p for p, n in enumerate(refs) if n == 0])
    grown = [lens[r] + 1 for r in parents]
    freed = []
    for row, n in zip(new, grown):
        held = len(row)
        if -(-n // P) > held:
            row.append(next(fresh))
            refs[row[-1]] += 1
        for i in range(held):
            if w and (i + 1) * P <= n - w and i * P >= f and row[i] >= 0:
                freed.append(row[i])
                row[i] = -1
    for p in freed:
        refs[p] -= 1
    width = s["table"].shape[1]
    return {"table": _ints([r + [-1] * (width - len(r)) for r in new]),
            "lens": _ints([lens[r] for r in parents]), "copies": _ints(copies),
            "refs": _ints(refs), "k_cache": k, "v_cache": v}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "beams":
        return _exact_beams(s, case)
    if case["op"] == "compact":
        k, v = s["k_cache"].clone(), s["v_cache"].clone()
        P = case["page"]
        for b, n in enumerate(_lens(case)):
            start, count = int(s["starts"][b]), int(s["counts"][b])
            at = torch.arange(n, device="cuda")
            slot = s["page_table"][b].long()[at // P] * P + at % P
            src = slot[start + s["kept"][b, :count].long()]
            for to, of in ((k, s["k_cache"]), (v, s["v_cache"])):
                to.view(-1, *to.shape[2:])[slot[start:start + count]] = \
                    of.view(-1, *of.shape[2:])[src]
        return {"k_cache": k, "v_cache": v}
    D, w, f = case["dim"], case["window"], case["first"]
    parts = []
    if case["op"] == "decode":
        for b, n in enumerate(_lens(case)):
            j = torch.arange(n, device="cuda")
            seen = ((j >= n - w) | (j < f)).nonzero()[:, 0]
            k, v = _context(s, b, n)
            parts.append(_rows64(s["q"][b:b + 1].double(), k[seen], v[seen],
                                 torch.ones(1, len(seen), dtype=torch.bool, device="cuda"),
                                 s["sinks"], D ** -0.5))
    elif case["op"] == "tree":
        lens = _lens(case)
        counts, parents = _drafts(case, lens)
        a = 0
        for b, (n, m) in enumerate(zip(lens, counts)):
            visible = torch.zeros(m, n, dtype=torch.bool)
            for i, d in enumerate(_depths(parents[b])):
                at = n - m + d
                visible[i, :n - m] = True
                if w:
                    visible[i, min(f, n - m):max(min(f, n - m), min(n - m, at - w + 1))] = False
                up, pos = i, at
                while up >= 0:
                    visible[i, n - m + up] = not w or pos > at - w or pos < f
                    up, pos = parents[b][up], pos - 1
            k, v = _context(s, b, n)
            parts.append(_rows64(s["q"][a:a + m].double(), k, v, visible.cuda(), s["sinks"],
                                 D ** -0.5))
            a += m
    else:
        a = b = 0
        for n, m in zip(*_prompt_lens(case)):
            at = (torch.arange(n, device="cuda") + m - n)[:, None]
            j = torch.arange(m, device="cuda")
            visible = (j <= at) & ((j > at - w) | (j < f))
            parts.append(_rows64(s["q"][a:a + n].double(), s["k"][b:b + m].double(),
                                 s["v"][b:b + m].double(), visible, s["sinks"], D ** -0.5))
            a, b = a + n, b + m
    out = torch.cat([p[0] for p in parts])
    return {"out": out, "lse": torch.cat([p[1] for p in parts])} if case["lse"] else {"out": out}

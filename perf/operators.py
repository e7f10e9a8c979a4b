"""Workloads of the attention operators: the paged cache's append, the decode
step's attention over it, and the attention of whole packed prompts.

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

def _append(name, tokens, heads, kv_heads, dim, rot, page, cache="bf16", interleaved=False,
            head_major=False):
    return {"name": name, "op": "append", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "rot": rot, "page": page, "cache": cache, "interleaved": interleaved,
            "head_major": head_major}


def _decode(name, batch, shortest, longest, heads, kv_heads, dim, page, cache="bf16", window=0,
            sinks=False, lse=False, lens_seed=1):
    return {"name": name, "op": "decode", "batch": batch, "shortest": shortest,
            "longest": longest, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "cache": cache, "window": window, "sinks": sinks, "lse": lse, "lens_seed": lens_seed}


def _prompt(name, batch, tokens, heads, kv_heads, dim, history=0, causal=True, window=0,
            sinks=False, lse=False, lens_seed=1):
    return {"name": name, "op": "prompt", "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "history": history, "causal": causal,
            "window": window, "sinks": sinks, "lse": lse, "lens_seed": lens_seed}


def listed():
    return [
        # one decode step's new tokens of 64 sequences, q rotated too: latency counts
        _append("append_step_64", 64, 32, 8, 128, 128, 16),
        # a long prompt's keys and values into an FP8 cache
        _append("append_prompt_8192_fp8", 8192, 32, 8, 128, 128, 64, cache="e4m3"),
        # odd token count and page size, half of the head rotated in adjacent pairs, a cache
        # stored head-major
        _append("append_odd_1777", 1777, 24, 3, 64, 32, 24, interleaved=True, head_major=True),
        # one user, a short conversation: latency counts
        _decode("decode_one_1500", 1, 1500, 1500, 32, 8, 128, 16),
        # a full server: 64 conversations from a few tokens to 8192
        _decode("decode_64_ragged_8192", 64, 5, 8192, 32, 8, 128, 64),
        # long documents in an FP8 cache, the log-sum-exp kept for joining with another part
        _decode("decode_16_long_fp8", 16, 9000, 32768, 64, 8, 128, 128, cache="e4m3", lse=True),
        # a sliding-window layer with sinks, many conversations
        _decode("decode_128_window", 128, 1, 4096, 64, 8, 64, 16, window=128, sinks=True),
        # a one-line prompt: latency counts
        _prompt("prompt_one_37", 1, 37, 32, 8, 128),
        # a batch of prompts of very different lengths, packed
        _prompt("prompt_packed_8192", 11, 8192, 32, 8, 128),
        # one long prompt
        _prompt("prompt_one_8192", 1, 8192, 32, 8, 128),
        # chunks of two long prompts against the keys so far, with the log-sum-exp
        _prompt("prompt_chunk_600_of_8192", 2, 600, 32, 8, 128, history=7592, lse=True),
        # a sliding-window layer with sinks over packed prompts
        _prompt("prompt_window_4096", 5, 4096, 64, 8, 64, window=128, sinks=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        c = _append("", _log(rng, 1, 8192), min(heads, 32 * 128 // dim), kv, dim,
                    rng.choice([32, 64, dim]), rng.choice([1, 16, 24, 64, 128]),
                    rng.choice(["bf16", "e4m3"]), rng.random() < 0.3, rng.random() < 0.5)
    elif op == "decode":
        longest = _log(rng, 1, 32768)
        batch = _log(rng, 1, max(1, min(256, (1 << 18) // longest)))
        window = rng.choice([0, 0, 128, _log(rng, 1, 4096)])
        c = _decode("", batch, max(1, int(longest * rng.random())), longest, heads, kv, dim,
                    rng.choice([1, 16, 24, 64, 128]), rng.choice(["bf16", "e4m3"]), window,
                    rng.random() < 0.3, rng.random() < 0.3, rng.randrange(1 << 20))
    else:
        causal = rng.random() < 0.8
        tokens = _log(rng, 1, 8192 if heads <= 32 and causal else 4096)
        batch = _log(rng, 1, max(1, min(64, tokens)))
        history = rng.choice([0, 0, _log(rng, 1, 8192)])
        if (tokens + batch * history) * tokens * heads * (1 if causal else 2) > 8192 * 8192 * 16:
            history = 0
        window = rng.choice([0, 0, _log(rng, 1, 2048)]) if causal else 0
        c = _prompt("", batch, tokens, heads, kv, dim, history, causal, window,
                    rng.random() < 0.3, rng.random() < 0.3, rng.randrange(1 << 20))
    del c["name"]
    return c


def _decode_lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["shortest"], case["longest"]) for _ in range(case["batch"])]


def _prompt_lens(case):
    """Query lengths (their sum is `tokens`) and key lengths of the packed sequences."""
    r = random.Random(case["lens_seed"])
    w = [r.random() ** 2 + 0.02 for _ in range(case["batch"])]
    spare = case["tokens"] - case["batch"]
    q = [1 + int(spare * x / sum(w)) for x in w]
    q[-1] += case["tokens"] - sum(q)
    return q, [n + case["history"] for n in q]


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _pool(case, pages, g):
    """A cache [pages, page, kv_heads, dim] that already holds values."""
    P, H, D = case["page"], case["kv_heads"], case["dim"]
    t = _randn(g, pages, H, P, D) if case.get("head_major") else _randn(g, pages, P, H, D)
    if case["cache"] == "e4m3":
        t = (t.float() * 100).clamp(-448, 448).to(FP8)
    return t.transpose(1, 2) if case.get("head_major") else t


def _kv_scales(case, g):
    """Per-head scales of an FP8 cache: what a unit-variance head needs, about 1/100."""
    if case["cache"] != "e4m3":
        return None, None
    h = case["kv_heads"]
    return tuple(0.008 + 0.004 * torch.rand(h, generator=g, device="cuda") for _ in range(2))


def prepare(case, seed):
    g = _gen(seed)
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case}
    if case["op"] == "append":
        T, P = case["tokens"], case["page"]
        qkv = _randn(g, T, (H + 2 * KV) * D)        # the QKV linear's output
        s["q"] = qkv[:, :H * D].view(T, H, D)
        s["k"] = qkv[:, H * D:(H + KV) * D].view(T, KV, D)
        s["v"] = qkv[:, (H + KV) * D:].view(T, KV, D)
        pages = -(-T // P) + 3
        s["k_cache"], s["v_cache"] = _pool(case, pages, g), _pool(case, pages, g)
        s["k_scale"], s["v_scale"] = _kv_scales(case, g)
        where = torch.randperm(pages, generator=g, device="cuda")     # pages come in any order
        i = torch.arange(T, device="cuda")
        s["slots"] = where[i // P] * P + i % P
        s["positions"] = torch.randint(0, 8192, (T,), generator=g, device="cuda",
                                       dtype=torch.int32)
        inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])
        a = torch.arange(8192, device="cuda").double()[:, None] * inv
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], dim=1).float()
    elif case["op"] == "decode":
        lens, P = _decode_lens(case), case["page"]
        need = [-(-n // P) for n in lens]
        width, total = max(need), sum(need)
        s["q"] = _randn(g, len(lens), H, D)
        s["k_cache"], s["v_cache"] = _pool(case, total, g), _pool(case, total, g)
        s["k_scale"], s["v_scale"] = _kv_scales(case, g)
        where = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        n = torch.tensor(need, device="cuda")
        at = (torch.cumsum(n, 0) - n)[:, None] + torch.arange(width, device="cuda")
        have = torch.arange(width, device="cuda") < n[:, None]
        s["page_table"] = torch.where(have, where[at.clamp(max=total - 1)], 0)
        s["seq_lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
    else:
        nq, nk = _prompt_lens(case)
        Tq, Tk = sum(nq), sum(nk)
        if Tq == Tk:
            qkv = _randn(g, Tq, (H + 2 * KV) * D)
            s["q"] = qkv[:, :H * D].view(Tq, H, D)
            s["k"] = qkv[:, H * D:(H + KV) * D].view(Tq, KV, D)
            s["v"] = qkv[:, (H + KV) * D:].view(Tq, KV, D)
        else:
            s["q"] = _randn(g, Tq, H, D)
            s["k"], s["v"] = _randn(g, Tk, KV, D), _randn(g, Tk, KV, D)
        for name, n in (("cu_q", nq), ("cu_k", nk)):
            c = [0]
            for x in n:
                c.append(c[-1] + x)
            s[name] = torch.tensor(c, device="cuda", dtype=torch.int32)
    if case.get("sinks"):
        s["sinks"] = torch.randn(H, generator=g, device="cuda")
    else:
        s["sinks"] = None
    # the scratch that a serving loop keeps for its calls
    s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, rot, interleaved):
    """Rotation of the first `rot` elements, in 32 bits."""
    x = x.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _store(cache, slots, x, scale):
    if scale is None:
        cache[slots // cache.shape[1], slots % cache.shape[1]] = x.to(torch.bfloat16)
    else:
        x = (x / scale[:, None]).clamp(-448, 448).to(FP8)
        cache.view(torch.uint8)[slots // cache.shape[1], slots % cache.shape[1]] = \
            x.view(torch.uint8)


def _plain_append(s):
    rot, pairs = s["case"]["rot"], s["case"]["interleaved"]
    t = s["cos_sin"][s["positions"]]
    cos, sin = t[:, None, :rot // 2], t[:, None, rot // 2:]
    _store(s["k_cache"], s["slots"], _rotate(s["k"], cos, sin, rot, pairs), s["k_scale"])
    _store(s["v_cache"], s["slots"], s["v"].float(), s["v_scale"])
    return {"q": _rotate(s["q"], cos, sin, rot, pairs).to(torch.bfloat16),
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _softmax_v(x, mask, sinks, v, lse):
    """x [..., queries, keys] scores, mask the visible ones, v [..., keys, dim], sinks [..., 1, 1]
    or None: softmax over the keys (a row that sees none gives 0) times v."""
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


def _plain_decode(s):
    c, q = s["case"], s["q"]
    B, H, D = q.shape
    KV = c["kv_heads"]
    pages = s["page_table"].long()
    k, v = (t[pages].flatten(1, 2).permute(0, 2, 1, 3).float()
            for t in (s["k_cache"], s["v_cache"]))        # [B, KV, keys, D]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    x = torch.matmul(q.float().view(B, KV, H // KV, D) * D ** -0.5, k.transpose(-1, -2))
    j = torch.arange(k.shape[2], device=q.device)
    n = s["seq_lens"][:, None]
    mask = j < n
    if c["window"]:
        mask = mask & (j >= n - c["window"])
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
    mask = qs[:, None] == ks
    if c["causal"]:
        mask &= j <= at
    if c["window"]:
        mask &= j > at - c["window"]
    qf = q.float().view(Tq, KV, H // KV, D).permute(1, 2, 0, 3) * D ** -0.5
    k, v = (t.float().transpose(0, 1)[:, None] for t in (s["k"], s["v"]))   # [KV, 1, Tk, D]
    sinks = None if s["sinks"] is None else s["sinks"].view(KV, H // KV, 1, 1)
    out, lse = _softmax_v(torch.matmul(qf, k.transpose(-1, -2)), mask, sinks, v, c["lse"])
    out = out.permute(2, 0, 1, 3).reshape(Tq, H, D).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(2, 0, 1).reshape(Tq, H)} if c["lse"] else {"out": out}


# ----------------------------------------------------------- the package's calls

def _own(s):
    import mxfp4_quantized_gemm_token_gb300 as mxq
    c = s["case"]
    if c["op"] == "append":
        q = mxq.rope_append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"],
                               s["cos_sin"], s["positions"], q=s["q"], k_scale=s["k_scale"],
                               v_scale=s["v_scale"], interleaved=c["interleaved"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "decode":
        r = mxq.paged_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"],
                                       s["seq_lens"], window=c["window"], sinks=s["sinks"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"],
                                       return_lse=c["lse"], workspace=s["workspace"])
    else:
        r = mxq.attention_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                 causal=c["causal"], window=c["window"], sinks=s["sinks"],
                                 return_lse=c["lse"], workspace=s["workspace"])
    return {"out": r[0], "lse": r[1]} if c["lse"] else {"out": r}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode,
            "prompt": _plain_prompt}[state["case"]["op"]](state)


# ---------------------------------------------------------------------- the work

def _pairs(nq, nk, causal, window):
    """Visible (query, key) pairs of one sequence."""
    ends = [(i + nk - nq, min(i + nk - nq, nk - 1) if causal else nk - 1) for i in range(nq)]
    return sum(max(0, hi - (max(0, at - window + 1) if window else 0) + 1) for at, hi in ends)


def work(case):
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        T, one = case["tokens"], 1 if case["cache"] == "e4m3" else 2
        b = T * (2 * H * D * 2 + 2 * KV * D * (2 + one) + 4 * case["rot"] + 12)
        return {"bytes": b, "flops": 3 * T * (H + KV) * case["rot"]}
    if case["op"] == "decode":
        lens, one = _decode_lens(case), 1 if case["cache"] == "e4m3" else 2
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        b = 2 * seen * KV * D * one + len(lens) * H * D * 4
        return {"bytes": b, "flops": 4 * seen * H * D}
    nq, nk = _prompt_lens(case)
    seen = sum(_pairs(a, b, case["causal"], case["window"]) for a, b in zip(nq, nk))
    return {"bytes": 2 * D * (2 * H * sum(nq) + 2 * KV * sum(nk)), "flops": 4 * seen * H * D}


# --------------------------------------------------------------- the definition

def _one_head(q, k, v, lo, hi, sink):
    """One head in 64 bits: q [n, D] (scaled), k, v [m, D]; row i sees keys lo[i] <= j < hi[i]."""
    x = q @ k.T
    j = torch.arange(k.shape[0], device=q.device)
    x[(j < lo[:, None]) | (j >= hi[:, None])] = -math.inf
    if sink is not None:
        x = torch.cat([x, sink.double().expand(len(q), 1)], 1)
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x[:, :k.shape[0]] - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return w @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        T, P, R = case["tokens"], case["page"], case["rot"]
        cs = s["cos_sin"].double()[s["positions"].long()].view(T, 1, 2, R // 2)
        i = torch.arange(R // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)

        def turn(x):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * torch.complex(cs[:, :, 0],
                                                                             cs[:, :, 1])
            y[..., first], y[..., second] = z.real, z.imag
            return y

        def placed(cache, x, scale):
            full = cache.double()
            if scale is not None:
                x = (x / scale.double()[:, None]).clamp(-448, 448)
            full[s["slots"] // P, s["slots"] % P] = x
            return full

        return {"q": turn(s["q"]), "k_cache": placed(s["k_cache"], turn(s["k"]), s["k_scale"]),
                "v_cache": placed(s["v_cache"], s["v"].double(), s["v_scale"])}
    G = H // KV
    if case["op"] == "decode":
        lens = _decode_lens(case)
        out = torch.zeros(len(lens), H, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(len(lens), H, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            first = max(0, n - case["window"]) if case["window"] else 0
            at = torch.arange(first, n, device="cuda")
            page, off = s["page_table"][b].long()[at // case["page"]], at % case["page"]
            k, v = s["k_cache"][page, off].double(), s["v_cache"][page, off].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
            x = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(KV, G, D), k) * D ** -0.5
            x = x.reshape(H, -1)
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"].double()[:, None]], 1)
            lse[b] = torch.logsumexp(x, 1)
            w = torch.exp(x[:, :n - first] - lse[b][:, None]).view(KV, G, -1)
            out[b] = torch.einsum("hgn,nhd->hgd", w, v).reshape(H, D)
    else:
        nq, nk = _prompt_lens(case)
        out = torch.zeros(sum(nq), H, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(sum(nq), H, dtype=torch.float64, device="cuda")
        a = b = 0
        for n, m in zip(nq, nk):
            at = torch.arange(n, device="cuda") + m - n
            hi = at + 1 if case["causal"] else torch.full_like(at, m)
            lo = at - case["window"] + 1 if case["window"] else torch.zeros_like(at)
            for h in range(H):
                k, v = (t[b:b + m, h // G].double() for t in (s["k"], s["v"]))
                q = s["q"][a:a + n, h].double() * D ** -0.5
                out[a:a + n, h], lse[a:a + n, h] = _one_head(
                    q, k, v, lo, hi, None if s["sinks"] is None else s["sinks"][h])
            a, b = a + n, b + m
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}

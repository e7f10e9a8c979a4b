"""Plain 64-bit forms of the paged cache and attention operators, with the
error bounds their tests use.

Attention output, per element, with w the exact softmax weights and
A = sum_j w_j |v_j|.  bf16 keeps 8 significant bits, so rounding to it moves a
value by up to 2^-8 of it (half of 2^-7, the step above 1); f16 keeps 11, so
2^-11.  The weights enter the value product rounded to u = 2^-8 (bf16 cache)
or u = 2^-11 (e4m3 cache, f16 weights, whose smallest step below 2^-14 adds 2^-25
of the largest weight for every key), the result rounds to bf16 (2^-8 of it, or half
of the smallest step, 2^-134); score, exponential and sum errors in fp32 are
below 2^-11 of A for the scores drawn here (score error <= D 2^-24 sum |q k|
scale, under 2^-12).
    |got - ref| <= 2^-8 |ref| + (u + 2^-11) A + 2^-134 (+ 2^-25 max w sum |v|)
Log-sum-exp: the largest score error, plus 2^-18 for exponential, sum and
logarithm, plus 2^-22 relative for its own rounding and that of the maximum.
"""
import math

import torch


def attend(q, k, v, visible, scale, sink=None, f16=False):
    """q [n, D], k, v [m, D], visible [n, m], all on one device: (out, lse,
    bound of out, bound of lse) in float64."""
    q, k, v = q.double(), k.double(), v.double()
    n, D = q.shape
    # invisible keys take no part, whatever they hold
    seen = visible.any(0)
    k = torch.where(seen[:, None], k, 0.0)
    v = torch.where(seen[:, None], v, 0.0)
    x = (q @ k.T) * scale
    x = torch.where(visible, x, -math.inf)
    size = torch.where(visible, (q.abs() @ k.abs().T) * scale, 0.0)
    size = size.amax(1) if k.shape[0] else torch.zeros(n, device=q.device).double()
    if sink is not None:
        x = torch.cat([x, torch.full((n, 1), float(sink), device=q.device).double()], 1)
    lse = torch.logsumexp(x, 1) if x.shape[1] else torch.full((n,), -math.inf,
                                                            device=q.device).double()
    w = torch.exp(x[:, :k.shape[0]] - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    out = w @ v
    u = 2.0 ** -11 if f16 else 2.0 ** -8
    bound = 2.0 ** -8 * out.abs() + (u + 2.0 ** -11) * (w @ v.abs()) + 2.0 ** -134
    if f16 and k.shape[0]:
        bound = bound + 2.0 ** -25 * w.amax(1)[:, None] * (visible.double() @ v.abs())
    lse_bound = D * 2.0 ** -24 * size + 2.0 ** -18 + 2.0 ** -22 * torch.where(
        lse == -math.inf, 0.0, lse.abs())
    return out, lse, bound, lse_bound


def assert_within(got, ref, bound, what):
    got = got.double()
    same = (got == ref) | ((got - ref).abs() <= bound)
    assert bool(same.all()), "%s: %d of %d outside the bound, worst %g x" % (
        what, int((~same).sum()), same.numel(),
        float(((got - ref).abs() / bound.clamp(min=1e-30))[~same].max()))


def decode_ref(q, k_cache, v_cache, page_table, lens, scale, window=0, sinks=None, k_scale=None,
               v_scale=None):
    B, H, D = q.shape
    KV, P = k_cache.shape[2], k_cache.shape[1]
    res = []
    for b in range(B):
        n = lens[b]
        j = torch.arange(n, device=q.device)
        page = page_table[b].long()[j // P] if n else j
        rows = []
        for h in range(H):
            g = h // (H // KV)
            k, v = k_cache[page, j % P, g].double(), v_cache[page, j % P, g].double()
            if k_scale is not None:
                k = k * k_scale[g].double()
            if v_scale is not None:
                v = v * v_scale[g].double()
            vis = (j >= (n - window if window else 0))[None]
            rows.append(attend(q[b, h:h + 1], k, v, vis, scale,
                               None if sinks is None else sinks[h],
                               k_cache.dtype == torch.float8_e4m3fn))
        res.append([torch.cat([r[i] for r in rows]) for i in range(4)])
    return [torch.stack([r[i] for r in res]) for i in range(4)]


def prompt_ref(q, k, v, lens_q, lens_k, scale, causal=True, window=0, sinks=None):
    T, H, D = q.shape
    KV = k.shape[1]
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.zeros(T, H, dtype=torch.float64, device=q.device)
    lb = torch.zeros_like(lse)
    a = b = 0
    for n, m in zip(lens_q, lens_k):
        i = torch.arange(n, device=q.device)[:, None] + m - n
        j = torch.arange(m, device=q.device)[None]
        vis = (j <= i) if causal else torch.ones(n, m, dtype=torch.bool, device=q.device)
        if window:
            vis = vis & (j > i - window)
        for h in range(H):
            g = h // (H // KV)
            r = attend(q[a:a + n, h], k[b:b + m, g], v[b:b + m, g], vis, scale,
                       None if sinks is None else sinks[h])
            out[a:a + n, h], lse[a:a + n, h], bound[a:a + n, h], lb[a:a + n, h] = r
        a, b = a + n, b + m
    return out, lse, bound, lb

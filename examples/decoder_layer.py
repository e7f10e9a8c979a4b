"""A decoder layer of a quantized mixture-of-experts model, from a packed batch of
prompts to generated tokens, on this package's operators alone:

    rms norm -> block-FP8 QKV linear -> rope_append_kv -> attention -> block-FP8
    output linear -> rms norm -> MXFP4 routed experts

Prompts run through attention_varlen and leave their keys and values in a
paged cache; each decode step appends one token per sequence and attends with
paged_attention_decode.  Weights are random.  The run checks that the last
prompt position, computed again as a decode step over the cache, gives the
same layer output.

    python examples/decoder_layer.py [--cache e4m3] [--steps 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_quantized_gemm_token_gb300 as mxq  # noqa: E402
from mxfp4_quantized_gemm_token_gb300 import synth  # noqa: E402

FP8 = torch.float8_e4m3fn


class DecoderLayer:
    def __init__(self, hidden=1024, heads=16, kv_heads=4, dim=64, experts=8, topk=2, ffn=512,
                 window=0, pages=64, page=16, cache="bf16", max_pos=4096, device="cuda"):
        self.hidden, self.heads, self.kv, self.dim = hidden, heads, kv_heads, dim
        self.topk, self.window, self.page = topk, window, page
        rows = (heads + 2 * kv_heads) * dim
        self.qkv_w, self.qkv_s = synth.block_fp8_weight(rows, hidden, 128, seed=1, device=device)
        self.out_w, self.out_s = synth.block_fp8_weight(hidden, heads * dim, 128, seed=2,
                                                        device=device)
        w1, s1, w2, s2 = synth.moe_mxfp4_weights(experts, ffn, hidden, seed=3)
        self.experts = tuple(t.to(device) for t in (w1, s1, w2, s2))
        self.router = synth.randn((experts, hidden), seed=4, device=device) * 0.05
        self.sinks = synth.randn((heads,), seed=5, device=device)
        a = torch.arange(max_pos)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2) / dim)
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).to(device)
        shape = (pages, page, kv_heads, dim)
        dtype = FP8 if cache == "e4m3" else torch.bfloat16
        self.k_cache = torch.zeros(shape, device=device).to(dtype)
        self.v_cache = torch.zeros(shape, device=device).to(dtype)
        # what a unit-variance key or value needs to use the e4m3 range
        one = torch.full((kv_heads,), 0.02, device=device) if cache == "e4m3" else None
        self.k_scale = self.v_scale = one

    def _norm(self, x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def _qkv(self, x, positions, slots, keep_k):
        """Rotated q (and k, if kept) and v; k and v also go to the cache."""
        T, H = x.shape[0], self.heads
        y = mxq.w8a8_block_fp8_linear(self._norm(x), self.qkv_w, [128, 128], self.qkv_s)
        y = y.view(T, H + 2 * self.kv, self.dim)
        k, v = y[:, H:H + self.kv], y[:, H + self.kv:]             # views: no copies
        # k's heads ride along with q's where the caller needs them rotated too
        q = mxq.rope_append_kv(k, v, self.k_cache, self.v_cache, slots, self.cos_sin, positions,
                               q=y[:, :H + self.kv if keep_k else H], k_scale=self.k_scale,
                               v_scale=self.v_scale)
        return q[:, :H], q[:, H:], v

    def _rest(self, x, attention):
        T = x.shape[0]
        x = x + mxq.w8a8_block_fp8_linear(attention.view(T, -1), self.out_w, [128, 128],
                                          self.out_s)
        y = self._norm(x)
        p = torch.softmax(y.float() @ self.router.T, -1)
        weights, ids = p.topk(self.topk, -1)
        return x + mxq.fused_experts(y, *self.experts, weights, ids.int(), wtype=mxq.W_MXFP4)

    def prompts(self, x, cu_seqlens, positions, slots):
        """x [tokens, hidden] of all prompts packed; fills the cache."""
        q, k, v = self._qkv(x, positions, slots, True)
        return self._rest(x, mxq.attention_varlen(q, k, v, cu_seqlens, window=self.window,
                                                  sinks=self.sinks))

    def step(self, x, positions, slots, page_table, lens):
        """x [sequences, hidden], one new token each, at the end of `lens` keys."""
        q, _, _ = self._qkv(x, positions, slots, False)
        return self._rest(x, mxq.paged_attention_decode(
            q, self.k_cache, self.v_cache, page_table, lens, window=self.window,
            sinks=self.sinks, k_scale=self.k_scale, v_scale=self.v_scale))


def run(cache="bf16", steps=16, lens=(37, 5, 100), window=0, device="cuda"):
    layer = DecoderLayer(cache=cache, window=window, device=device)
    B, page = len(lens), layer.page
    most = -(-(max(lens) + steps) // page)
    # pages in any order, one row of the table per sequence
    table = torch.randperm(layer.k_cache.shape[0], generator=torch.Generator().manual_seed(0))
    table = table[:B * most].view(B, most).int().to(device)

    def slot(seq, pos):
        return table[seq, pos // page].long() * page + pos % page

    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(lens)]).to(device)
    pos = torch.cat([torch.arange(n) for n in lens]).to(device)
    cu = torch.tensor([0, *lens]).cumsum(0).int().to(device)
    x = synth.randn((sum(lens), layer.hidden), seed=9, device=device).bfloat16()
    out = layer.prompts(x, cu, pos.int(), slot(seq, pos))

    # the last prompt token again, as a decode step over the filled cache
    n = torch.tensor(lens, device=device)
    last = cu[1:].long() - 1
    everyone = torch.arange(B, device=device)
    again = layer.step(x[last], (n - 1).int(), slot(everyone, n - 1), table, n.int())
    difference = float((again.float() - out[last].float()).norm() / out[last].float().norm())

    # generation: the layer's output stands for the next token's embedding
    tokens = out[last]
    for _ in range(steps):
        n = n + 1
        tokens = layer.step(tokens, (n - 1).int(), slot(everyone, n - 1), table, n.int())
    mxq.sync_status()
    return difference, tokens


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--window", type=int, default=0)
    a = p.parse_args()
    d, t = run(a.cache, a.steps, window=a.window)
    print("prompt against decode step: relative difference %.2g" % d)
    print("after %d steps: %s, norm %.3f" % (a.steps, list(t.shape), float(t.float().norm())))

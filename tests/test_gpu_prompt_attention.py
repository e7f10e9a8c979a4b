"""attention_varlen against a plain 64-bit form within the bounds of
attention_util: lengths, groups, masks that leave rows empty, chunks, windows,
sinks, strides, and what other sequences hold."""
import ctypes

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib
from attention_util import assert_within, prompt_ref

pytestmark = pytest.mark.gpu
NAN = float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def offsets(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, device="cuda", dtype=torch.int32)


def check(nq, nk, H, KV, D, causal=True, window=0, sinks=False, seed=0, fused=False):
    g = gen(seed + sum(nq) * 7 + H)
    if fused and nq == nk:
        T = sum(nq)
        qkv = randn(g, T, (H + 2 * KV) * D)
        q, k, v = (qkv[:, a * D:b * D].view(T, b - a, D)
                   for a, b in ((0, H), (H, H + KV), (H + KV, H + 2 * KV)))
    else:
        q, k, v = randn(g, sum(nq), H, D), randn(g, sum(nk), KV, D), randn(g, sum(nk), KV, D)
    s = torch.randn(H, generator=g, device="cuda") * 2 if sinks else None
    out, lse = mxq.attention_varlen(q, k, v, offsets(nq), None if nq == nk else offsets(nk),
                                    causal=causal, window=window, sinks=s, return_lse=True)
    mxq.sync_status()
    ref, rl, b, bl = prompt_ref(q, k, v, nq, nk, D ** -0.5, causal, window, s)
    assert_within(out, ref, b, "out")
    assert_within(lse, rl, bl, "lse")


LENGTHS = [[1], [2], [31], [64], [127], [128], [129], [255], [257], [385], [700],
           [1, 1, 1], [5, 0, 300, 1, 0], [0, 0, 3], [128, 128], [130, 1, 260, 77, 64]]


@pytest.mark.parametrize("lens", LENGTHS)
@pytest.mark.parametrize("H,KV,D", [(4, 2, 128), (8, 1, 64)])
def test_lengths(lens, H, KV, D):
    check(lens, lens, H, KV, D)


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 3), (6, 2), (8, 2), (5, 1), (7, 1), (16, 1), (20, 1),
                                  (32, 1), (48, 1), (128, 1), (100, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_groups(H, KV, D):
    check([70, 3, 150], [70, 3, 150], H, KV, D, seed=1, fused=True)


@pytest.mark.parametrize("nq,nk", [([1], [500]), ([100], [400]), ([3, 200], [900, 200]),
                                   ([130], [1024]), ([10, 20, 30], [10, 300, 31])])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(nq, nk, causal):
    check(nq, nk, 8, 2, 128, causal, seed=2)
    check(nq, nk, 4, 4, 64, causal, seed=3, sinks=True)


@pytest.mark.parametrize("nq,nk", [([10], [0]), ([200], [50]), ([3, 150, 7], [0, 20, 7])])
def test_rows_without_keys(nq, nk):
    """More queries than keys: the first rows see nothing and are 0 (lse -inf,
    or the sink)."""
    for sinks in (False, True):
        check(nq, nk, 4, 2, 64, sinks=sinks, seed=4)
    check(nq, nk, 4, 2, 128, causal=False, seed=5)


@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 300])
@pytest.mark.parametrize("sinks", [False, True])
def test_window(window, sinks):
    check([400, 1, 90], [400, 1, 90], 8, 2, 64, window=window, sinks=sinks, seed=6)
    check([50, 140], [700, 140], 4, 1, 128, window=window, sinks=sinks, seed=7)


def test_not_causal_packed():
    check([300, 17, 128], [300, 17, 128], 6, 2, 128, causal=False, seed=8)


def test_long():
    check([3000], [3000], 4, 1, 128, seed=9)
    check([2100, 40], [2100, 40], 2, 2, 64, causal=False, seed=10)
    check([40], [20000], 8, 2, 128, seed=11)


@pytest.mark.parametrize("nq,nk,H,KV,D,window", [
    ([5], [1025], 2, 1, 128, 0), ([64], [1153], 8, 8, 64, 0),
    ([300, 9], [5000, 2111], 8, 2, 128, 0),
    ([1, 1, 0, 7], [3000, 129, 50, 4001], 6, 2, 64, 0), ([30], [6000], 4, 1, 64, 3000),
    ([700], [3500], 3, 1, 128, 0), ([16, 16], [0, 9000], 128, 1, 64, 0)])
@pytest.mark.parametrize("sinks", [False, True])
def test_few_rows_many_keys(nq, nk, H, KV, D, window, sinks):
    """The keys of one item go to several CTAs and are joined."""
    check(nq, nk, H, KV, D, window=window, sinks=sinks, seed=20)
    check(nq, nk, H, KV, D, causal=False, sinks=sinks, seed=21)


def test_many_sequences():
    lens = [(i * 37) % 90 for i in range(150)]
    check(lens, lens, 4, 2, 64, seed=12)


@pytest.mark.parametrize("B", [128, 129, 256, 257, 505, 600])
def test_any_number_of_items(B):
    """The list's order, with each number of threads an item and by both ways."""
    nq = [1 + (i * 7) % 3 for i in range(B)]
    nk = [n + (i * 131) % 300 for i, n in enumerate(nq)]
    check(nq, nk, 4, 2, 64, seed=13)


def test_pieces_repeat_bit_for_bit():
    """Items of equal length, cut and joined, in the same places each time."""
    g = gen(23)
    nq, nk = [90] * 5, [3000] * 5
    q, k, v = randn(g, 450, 8, 128), randn(g, 15000, 2, 128), randn(g, 15000, 2, 128)
    runs = [mxq.attention_varlen(q, k, v, offsets(nq), offsets(nk)) for _ in range(8)]
    mxq.sync_status()
    assert all(torch.equal(runs[0], r) for r in runs[1:])


def test_offsets_that_run_backwards_are_reported():
    """Sequences that overlap, in more items than there is room for."""
    g = gen(24)
    q, k, v = randn(g, 50, 32, 64), randn(g, 50, 1, 64), randn(g, 50, 1, 64)
    cu = torch.tensor([0, 50] * 40, device="cuda", dtype=torch.int32)
    mxq.sync_status()
    mxq.attention_varlen(q, k, v, cu)
    with pytest.raises(mxq.MxqError) as e:
        mxq.sync_status()
    assert e.value.status == _lib.ERR_DEVICE
    check([50], [50], 32, 1, 64)


def test_other_sequences_do_not_reach_in():
    """Neighbours and rows outside every sequence hold NaN and infinities."""
    g = gen(13)
    H, KV, D = 8, 2, 128
    lens = [70, 100, 90]
    T = 300                                      # 40 rows past the last sequence
    q, k, v = randn(g, T, H, D), randn(g, T, KV, D), randn(g, T, KV, D)
    ref, _, b, _ = prompt_ref(q[70:170], k[70:170], v[70:170], [100], [100], D ** -0.5)
    for t in (q, k, v):
        t[:70] = NAN
        t[170:260] = float("inf")
        t[260:] = NAN
    out = torch.full((T, H, D), 7.0, device="cuda", dtype=torch.bfloat16)
    mxq.attention_varlen(q, k, v, offsets(lens), out=out)
    assert_within(out[70:170], ref, b, "out")
    assert bool((out[260:] == 7).all())          # not written


def test_large_scores():
    """Scores of several hundred: rounding moves the weights, nothing overflows."""
    g = gen(14)
    q, k, v = randn(g, 300, 4, 128) * 30, randn(g, 300, 2, 128), randn(g, 300, 2, 128)
    out = mxq.attention_varlen(q, k, v, offsets([300]))
    ref = prompt_ref(q, k, v, [300], [300], 128 ** -0.5)[0]
    assert torch.isfinite(out.float()).all()
    assert float((out.double() - ref).norm() / ref.norm()) < 2.0 ** -7
    # rising scores: the running maximum moves at every tile
    k = torch.linspace(-60, 60, 900, device="cuda")[:, None, None] * torch.ones(900, 1, 64,
                                                                              device="cuda")
    k, v = k.bfloat16(), randn(g, 900, 1, 64)
    q = torch.full((900, 2, 64), 0.25, device="cuda", dtype=torch.bfloat16)
    out = mxq.attention_varlen(q, k, v, offsets([900]))
    ref = prompt_ref(q, k, v, [900], [900], 0.125)[0]
    assert float((out.double() - ref).norm() / ref.norm()) < 2.0 ** -7


def test_strides_streams_and_given_buffers():
    g = gen(15)
    H, KV, D, T = 6, 3, 64, 150
    qs = randn(g, H, T, D).transpose(0, 1)                       # head-major storage
    ks, vs = randn(g, KV, T, D).transpose(0, 1), randn(g, T, KV, 2 * D)[:, :, D:]
    big = torch.full((T, H, 3 * D), 5.0, device="cuda", dtype=torch.bfloat16)
    ws = torch.full((max(256, mxq.attention_varlen_workspace_size(T, 2, H, KV, D)),), 255,
                    dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = mxq.attention_varlen(qs, ks, vs, offsets([100, 50]), out=big[:, :, D:2 * D],
                                   workspace=ws)
    s.synchronize()
    ref, _, b, _ = prompt_ref(qs, ks, vs, [100, 50], [100, 50], 0.125)
    assert_within(out, ref, b, "out")
    assert bool((big[:, :, :D] == 5).all()) and bool((big[:, :, 2 * D:] == 5).all())
    # an odd inner offset and a broadcast head are copied, not refused
    odd = randn(g, T, H * D + 3)[:, 3:].view(T, H, D)
    wide = randn(g, T, 1, D).expand(T, KV, D)
    out = mxq.attention_varlen(odd, wide, vs, offsets([T]))
    ref, _, b, _ = prompt_ref(odd, wide, vs, [T], [T], 0.125)
    assert_within(out, ref, b, "out")


def test_repeats_bit_for_bit():
    g = gen(16)
    q, k, v = randn(g, 60, 8, 128), randn(g, 9000, 1, 128), randn(g, 9000, 1, 128)
    args = (q, k, v, offsets([60]), offsets([9000]))
    first = mxq.attention_varlen(*args)
    for _ in range(3):
        assert torch.equal(mxq.attention_varlen(*args), first)


def test_bad_offsets_are_reported():
    g = gen(17)
    q, k, v = randn(g, 50, 4, 64), randn(g, 50, 2, 64), randn(g, 50, 2, 64)
    mxq.sync_status()
    out = torch.full_like(q, 7.0)
    cu = torch.tensor([0, 20, 10, 51], device="cuda", dtype=torch.int32)
    mxq.attention_varlen(q, k, v, cu, out=out)
    with pytest.raises(mxq.MxqError) as e:
        mxq.sync_status()
    assert e.value.status == _lib.ERR_DEVICE
    ref, _, b, _ = prompt_ref(q[:20], k[:20], v[:20], [20], [20], 0.125)
    assert_within(out[:20], ref, b, "out")
    assert bool((out[20:] == 7).all())


def test_refusals():
    g = gen(18)
    q, k, v, cu = randn(g, 5, 4, 64), randn(g, 5, 2, 64), randn(g, 5, 2, 64), offsets([5])
    for args, kw in [((q.float(), k, v, cu), {}), ((q, k, v[:4], cu), {}),
                     ((q, k[..., :32], v[..., :32], cu), {}), ((q, k, v, cu.long()), {}),
                     ((q, k, v, cu, offsets([2, 3])), {}), ((q.cpu(), k, v, cu), {}),
                     ((q, k.cpu(), v, cu), {}), ((q[0], k, v, cu), {}),
                     ((q, k, v, cu), {"sinks": torch.ones(3, device="cuda")}),
                     ((q, k, v, cu), {"out": q[:4]})]:
        with pytest.raises((ValueError, TypeError)):
            mxq.attention_varlen(*args, **kw)
    for args, kw, st in [((q[:, :3], k, v, cu), {}, _lib.ERR_INVALID_ARG),
                         ((q, k, v, cu), {"scale": 0.0}, _lib.ERR_INVALID_ARG),
                         ((q, k, v, cu), {"window": -2}, _lib.ERR_INVALID_ARG),
                         ((q, k, v, cu), {"window": 4, "causal": False}, _lib.ERR_INVALID_ARG),
                         ((q[..., :32], k[..., :32], v[..., :32], cu), {}, _lib.ERR_UNSUPPORTED)]:
        with pytest.raises(mxq.MxqError) as e:
            mxq.attention_varlen(*args, **kw)
        assert e.value.status == st
    empty = mxq.attention_varlen(q[:0], k[:0], v[:0], offsets([0]))
    assert empty.shape == (0, 4, 64)
    lib = _lib.load()
    base = [q.data_ptr(), 256, 64, k.data_ptr(), 128, 64, v.data_ptr(), 128, 64, cu.data_ptr(),
            cu.data_ptr(), 1, 5, 5, 4, 2, 64, 0.125, 1, 0, None, q.data_ptr(), 256, 64, None, None,
            0, None]
    for i, val, st in [(0, None, _lib.ERR_INVALID_ARG), (3, k.data_ptr() + 8, _lib.ERR_UNSUPPORTED),
                       (4, 132, _lib.ERR_UNSUPPORTED), (5, 60, _lib.ERR_INVALID_ARG),
                       (9, None, _lib.ERR_INVALID_ARG), (15, 3, _lib.ERR_INVALID_ARG),
                       (12, -1, _lib.ERR_INVALID_ARG), (21, None, _lib.ERR_INVALID_ARG)]:
        args = list(base)
        args[i] = val
        assert lib.mxq_attention_varlen(*args) == st, i
    size = ctypes.c_size_t(0)
    assert lib.mxq_attention_varlen_workspace_size(5, 1, 4, 2, 32, ctypes.byref(size)) == \
        _lib.ERR_UNSUPPORTED


@pytest.mark.parametrize("nq,nk", [([300], [300]), ([70, 20], [70, 3000])])
def test_stalled_loads_time_out_and_recover(nq, nk):
    """With the test-only switch no tile is loaded: every wait runs out, the status
    says so, and the next call is right."""
    g = gen(22)
    q, k, v = randn(g, sum(nq), 8, 128), randn(g, sum(nk), 2, 128), randn(g, sum(nk), 2, 128)
    mxq.sync_status()
    old = mxq.get_option(_lib.OPT_WAIT_BUDGET_NS)
    try:
        mxq.set_option(_lib.OPT_WAIT_BUDGET_NS, 20_000_000)
        mxq.set_option(_lib.OPT_INJECT_STALL, 1)
        mxq.attention_varlen(q, k, v, offsets(nq), offsets(nk))
        with pytest.raises(mxq.MxqError) as e:
            mxq.sync_status()
        assert e.value.status == _lib.ERR_TIMEOUT
    finally:
        mxq.set_option(_lib.OPT_INJECT_STALL, 0)
        mxq.set_option(_lib.OPT_WAIT_BUDGET_NS, old)
    check(nq, nk, 8, 2, 128, seed=23)

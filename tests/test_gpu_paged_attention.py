"""rope_append_kv and paged_attention_decode against plain forms: the append
bit for bit against elementary fp32 operations, the attention against 64 bits
within the bounds of attention_util."""
import ctypes

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib
from attention_util import assert_within, decode_ref

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
NAN = float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def pool(g, pages, page, kv, D, fp8, head_major=False):
    t = randn(g, pages, kv, page, D) if head_major else randn(g, pages, page, kv, D)
    if fp8:
        t = (t.float() * 60).clamp(-448, 448).to(FP8)
    return t.transpose(1, 2) if head_major else t


def bits(t):
    return t.contiguous().view(torch.uint8 if t.dtype == FP8 else torch.int16)


# ------------------------------------------------------------------- append

def rotate_ref(x, cs, rot, interleaved):
    x = x.float()
    if rot == 0:
        return x
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


@pytest.mark.parametrize("T,H,KV,D,rot,page,fp8,inter,major", [
    (1, 1, 1, 16, 16, 1, False, False, False),
    (3, 8, 2, 64, 32, 5, False, True, True),
    (65, 32, 8, 128, 128, 16, True, False, False),
    (17, 0, 3, 128, 64, 24, True, True, True),       # no q
    (40, 5, 5, 96, 96, 7, False, False, True),
    (9, 20, 4, 192, 0, 16, True, False, False),      # no rotation
    (300, 12, 1, 512, 64, 64, False, False, False),
    (11, 7, 7, 48, 16, 3, True, False, False),       # threads per head not a power of two
    (2000, 12, 2, 64, 64, 16, False, True, True),    # more tokens than blocks: few heads,
    (1600, 16, 4, 128, 64, 16, True, False, False),  # more,
    (1000, 32, 8, 128, 128, 32, False, False, False),    # many
])
def test_append_bit_exact(T, H, KV, D, rot, page, fp8, inter, major):
    g = gen(T)
    qkv = randn(g, T, (H + 2 * KV) * D)
    q = qkv[:, :H * D].view(T, H, D) if H else None
    k = qkv[:, H * D:(H + KV) * D].view(T, KV, D)
    v = qkv[:, (H + KV) * D:].view(T, KV, D)
    pages = -(-T // page) + 2
    kc, vc = pool(g, pages, page, KV, D, fp8, major), pool(g, pages, page, KV, D, fp8)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    if T > 2:
        slots[1] = -1                                  # a token that is not cached
    pos = torch.randint(0, 500, (T,), generator=g, device="cuda", dtype=torch.int32)
    cs = torch.randn(500, max(rot, 1), generator=g, device="cuda")
    ks = vs = None
    if fp8:
        ks = torch.rand(KV, generator=g, device="cuda") * 0.01 + 0.002
        vs = torch.rand(KV, generator=g, device="cuda") * 0.01 + 0.002
    rows = cs[pos.long()]
    want = []
    for cache, x, sc in ((kc, rotate_ref(k, rows, rot, inter), ks), (vc, v.float(), vs)):
        x = (x / sc[:, None]).clamp(-448, 448).to(FP8) if fp8 else x.to(torch.bfloat16)
        w = bits(cache.clone(memory_format=torch.contiguous_format)).view(pages * page, KV, D)
        keep = slots >= 0
        w[slots[keep]] = bits(x)[keep]
        want.append(w)
    got = mxq.rope_append_kv(k, v, kc, vc, slots, cs if rot else None, pos if rot else None, q=q,
                             k_scale=ks, v_scale=vs, interleaved=inter)
    for cache, w in ((kc, want[0]), (vc, want[1])):
        assert torch.equal(bits(cache).view(pages * page, KV, D), w)
    if H:
        assert torch.equal(bits(got), bits(rotate_ref(q, rows, rot, inter).to(torch.bfloat16)))
    else:
        assert got is None


def test_append_in_place_and_special_values():
    """q rotated in place; NaN, infinities and values past the e4m3 range."""
    g = gen(5)
    T, H, KV, D, page = 6, 4, 2, 64, 4
    q, k, v = randn(g, T, H, D), randn(g, T, KV, D), randn(g, T, KV, D)
    v[0, 0, :4] = torch.tensor([NAN, float("inf"), -float("inf"), 1e30])
    cs = torch.randn(10, D, generator=g, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    kc, vc = pool(g, 2, page, KV, D, True), pool(g, 2, page, KV, D, True)
    want = rotate_ref(q, cs[:T], D, False).to(torch.bfloat16)
    got = mxq.rope_append_kv(k, v, kc, vc, slots, cs, pos, q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(bits(q), bits(want))
    first = vc[0, 0, 0].float()
    assert torch.isnan(first[0]) and first[1:4].tolist() == [448.0, -448.0, 448.0]
    assert torch.equal(bits(vc.reshape(-1, KV, D)[1:T]),
                       bits(v[1:].float().clamp(-448, 448).to(FP8)))


def test_append_bad_slot_and_position_are_skipped_and_reported():
    g = gen(6)
    T, KV, D, page = 4, 2, 64, 4
    k, v = randn(g, T, KV, D), randn(g, T, KV, D)
    kc, vc = pool(g, 2, page, KV, D, False), pool(g, 2, page, KV, D, False)
    before = kc.clone()
    cs = torch.randn(10, D, generator=g, device="cuda")
    slots = torch.tensor([8, 1, 2, 3], device="cuda")            # 8 slots: 0..7
    pos = torch.tensor([0, 10, -1, 9], device="cuda", dtype=torch.int32)
    mxq.sync_status()
    mxq.rope_append_kv(k, v, kc, vc, slots, cs, pos)
    with pytest.raises(mxq.MxqError) as e:
        mxq.sync_status()
    assert e.value.status == _lib.ERR_DEVICE
    before.view(-1, KV, D)[3] = rotate_ref(k[3:], cs[9:10], D, False)[0].to(torch.bfloat16)
    assert torch.equal(bits(kc), bits(before))


# ------------------------------------------------------------------- decode

def decode_case(seed, lens, H, KV, D, page, fp8=False, major=False, poison=True, pages=None,
                q_scale=1.0):
    """Inputs whose unused pages, rows past each length and table entries hold
    what must never be read."""
    g = gen(seed)
    B = len(lens)
    need = [-(-n // page) for n in lens]
    total = sum(need) + 2
    kc, vc = pool(g, total, page, KV, D, fp8, major), pool(g, total, page, KV, D, fp8, major)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1) + 1
    table = torch.full((B, width), -7, device="cuda", dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        if poison and lens[b] % page:
            for c in (kc, vc):
                c[order[at - 1].long(), lens[b] % page:] = torch.full(
                    (1,), NAN, device="cuda").to(c.dtype)
    if poison:
        for c in (kc, vc):
            c[order[at:].long()] = torch.full((1,), NAN, device="cuda").to(c.dtype)
    q = (randn(g, B, H, D).float() * q_scale).bfloat16()
    n = torch.tensor(lens, device="cuda", dtype=torch.int32)
    return q, kc, vc, table, n, g


def run_decode(c, lens, window=0, sinks=None, ks=None, vs=None, scale=None):
    q, kc, vc, table, n, _ = c
    out, lse = mxq.paged_attention_decode(q, kc, vc, table, n, scale=scale, window=window,
                                          sinks=sinks, k_scale=ks, v_scale=vs, return_lse=True)
    mxq.sync_status()
    ref, rl, b, bl = decode_ref(q, kc, vc, table, lens, scale or q.shape[2] ** -0.5, window, sinks,
                                ks, vs)
    assert_within(out, ref, b, "out")
    assert_within(lse, rl, bl, "lse")
    return out, lse


@pytest.mark.parametrize("lens,H,KV,D,page,fp8,major", [
    ([1], 1, 1, 64, 1, False, False),
    ([0, 1, 2, 15, 16, 17], 8, 2, 128, 16, False, False),
    ([0, 0], 4, 4, 64, 16, False, True),
    ([33, 0, 64, 500, 7], 6, 2, 128, 24, False, True),          # groups of 3
    ([1000, 3], 20, 4, 64, 1, False, False),                    # groups of 5, one-row pages
    ([129, 777, 64], 32, 8, 128, 64, True, False),
    ([5, 300], 16, 1, 128, 128, True, True),                    # one kv head, 16 queries
    ([70, 1, 130], 21, 1, 64, 7, True, False),                  # 21 queries a head
    ([257, 31], 128, 1, 128, 16, False, False),                 # 128 queries a head
    ([6000], 32, 8, 128, 16, False, False),                     # one long sequence
    ([20000, 1, 9], 8, 1, 64, 64, True, False),
    ([40 * i for i in range(70)], 4, 2, 64, 32, False, False),  # many sequences
])
def test_decode(lens, H, KV, D, page, fp8, major):
    run_decode(decode_case(sum(lens) + H, lens, H, KV, D, page, fp8, major), lens)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 4000])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_window_and_sinks(window, fp8):
    lens = [0, 1, 99, 100, 101, 3000]
    c = decode_case(window, lens, 16, 2, 64, 16, fp8)
    g = c[-1]
    sinks = torch.randn(16, generator=g, device="cuda") * 3
    out, lse = run_decode(c, lens, window, sinks)
    assert torch.equal(out[0], torch.zeros_like(out[0]))
    assert torch.equal(lse[0], sinks)                            # only the sink is left
    run_decode(c, lens, window, None)


@pytest.mark.parametrize("D,fp8,limit", [(64, False, 288), (64, True, 288), (128, False, 144),
                                         (128, True, 288)])
def test_decode_where_sequences_stay_whole(D, fp8, limit):
    """Calls whose longest possible sequence is just short enough to be one
    warp's, and calls just past that: bounded by the page table, by the window."""
    for n in (limit - 17, limit - 1, limit, limit + 1, limit + 16):
        q, kc, vc, table, lens, g = decode_case(n, [n, 3, n], 8, 2, D, 16, fp8)
        table = table[:, :-(-n // 16)]
        run_decode((q, kc, vc, table, lens, g), [n, 3, n])
    lens = [1000, limit, 1007]
    c = decode_case(D, lens, 8, 2, D, 16, fp8)
    for window in (limit - 16, limit - 15, limit - 14, limit):
        run_decode(c, lens, window)


@pytest.mark.parametrize("D,fp8", [(64, False), (64, True), (128, False), (128, True)])
def test_decode_many_short_among_long(D, fp8):
    """Parts of one step and more, with sequences around a part's length."""
    for B, longest in [(3, 400), (24, 250), (40, 90), (150, 333)]:
        lens = [1 + (i * 97) % longest for i in range(B)]
        run_decode(decode_case(B, lens, 8, 2, D, 16, fp8), lens)


def test_decode_scales_and_large_scores():
    """Per-head scales of an e4m3 cache; scores of several hundred."""
    lens = [1, 200, 3333]
    c = decode_case(3, lens, 24, 8, 128, 64, True)
    g = c[-1]
    ks, vs = (torch.rand(8, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2))
    run_decode(c, lens, 0, None, ks, vs)
    c = decode_case(4, lens, 24, 8, 128, 64, False, q_scale=40.0)
    q = c[0]
    out = mxq.paged_attention_decode(*c[:5])
    # scores this large round by more than the bounds above: the largest score's
    # key must still carry the weight, and nothing may overflow
    assert torch.isfinite(out.float()).all()
    ref = decode_ref(q, c[1], c[2], c[3], lens, 128 ** -0.5)[0]
    assert float((out.double() - ref).norm() / ref.norm()) < 2.0 ** -7


def test_decode_empty_rows_without_sinks():
    c = decode_case(8, [0, 0, 0], 8, 2, 128, 16)
    out, lse = mxq.paged_attention_decode(*c[:5], return_lse=True)
    assert not out.any() and bool((lse == -float("inf")).all())


def test_decode_strided_q_and_out_and_other_stream():
    lens = [100, 37]
    q, kc, vc, table, n, g = decode_case(9, lens, 8, 2, 64, 16)
    wide = randn(g, 2, 3 * 8 * 64)
    q = wide[:, 8 * 64:16 * 64].view(2, 8, 64)
    big = torch.full((2, 8, 192), 5.0, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = mxq.paged_attention_decode(q, kc, vc, table, n, out=big[:, :, 64:128])
    s.synchronize()
    ref, _, b, _ = decode_ref(q, kc, vc, table, lens, 0.125)
    assert_within(out, ref, b, "out")
    assert bool((big[:, :, :64] == 5).all()) and bool((big[:, :, 128:] == 5).all())


def test_decode_offsets_past_32_bits():
    """Pages 2^30 elements apart: the third starts at 2^31 bytes and elements."""
    big = torch.empty((1 << 31) + (1 << 20), dtype=torch.uint8, device="cuda").view(FP8)
    page, KV, D = 16, 2, 64
    kc = big.as_strided((3, page, KV, D), (1 << 30, KV * D, D, 1))
    vc = big[1 << 18:].as_strided((3, page, KV, D), (1 << 30, KV * D, D, 1))
    g = gen(11)
    for c in (kc, vc):
        c.copy_((torch.randn(3, page, KV, D, generator=g, device="cuda") * 30).to(FP8))
    table = torch.tensor([[2, 1, 0]], device="cuda", dtype=torch.int32)
    n = torch.tensor([40], device="cuda", dtype=torch.int32)
    q = randn(g, 1, 4, D)
    run_decode((q, kc, vc, table, n, g), [40], ks=torch.full((2,), 0.02, device="cuda"))
    k, v = randn(g, 1, KV, D), randn(g, 1, KV, D)
    mxq.rope_append_kv(k, v, kc, vc, torch.tensor([2 * page + 3], device="cuda"))
    assert torch.equal(bits(kc[2, 3]), bits(k[0].to(FP8)))
    assert torch.equal(bits(vc[2, 3]), bits(v[0].to(FP8)))


def test_decode_bad_page_and_length_are_reported():
    lens = [40, 33]
    q, kc, vc, table, n, g = decode_case(12, lens, 4, 2, 64, 16, poison=False)
    table[0, 1] = kc.shape[0]                                    # one past the last page
    mxq.sync_status()
    out = mxq.paged_attention_decode(q, kc, vc, table, n)
    with pytest.raises(mxq.MxqError) as e:
        mxq.sync_status()
    assert e.value.status == _lib.ERR_DEVICE
    # the page's keys are left out; the other sequence is unharmed
    keep = torch.cat([torch.arange(16), torch.arange(32, 40)]).cuda()
    t2 = table.clone()
    t2[0, 1] = 0
    page, off = t2[0].long()[keep // 16], keep % 16
    from attention_util import attend
    for h in range(4):
        r, _, b, _ = attend(q[0, h:h + 1], kc[page, off, h // 2], vc[page, off, h // 2],
                            torch.ones(1, 24, dtype=torch.bool, device="cuda"), 0.125)
        assert_within(out[0, h:h + 1], r, b, "out")
    ref, _, b, _ = decode_ref(q[1:], kc, vc, table[1:], lens[1:], 0.125)
    assert_within(out[1:], ref, b, "out")
    n2 = torch.tensor([-3, 10 ** 6], device="cuda", dtype=torch.int32)
    table.fill_(1)
    out = mxq.paged_attention_decode(q, kc, vc, table, n2)
    with pytest.raises(mxq.MxqError):
        mxq.sync_status()
    assert not out[0].any() and torch.isfinite(out[1].float()).all()


def test_decode_repeats_bit_for_bit():
    c = decode_case(13, [5000, 17, 900], 32, 8, 128, 16)
    first = mxq.paged_attention_decode(*c[:5])
    for _ in range(3):
        assert torch.equal(mxq.paged_attention_decode(*c[:5]), first)


def test_append_then_decode_sees_the_new_token():
    lens = [33, 80]
    q, kc, vc, table, n, g = decode_case(14, lens, 8, 2, 64, 16, poison=False)
    k, v = randn(g, 2, 2, 64), randn(g, 2, 2, 64)
    slots = torch.stack([table[b, (lens[b] - 1) // 16].long() * 16 + (lens[b] - 1) % 16
                         for b in range(2)])
    cs = torch.randn(100, 64, generator=g, device="cuda")
    pos = n - 1
    qr = mxq.rope_append_kv(k, v, kc, vc, slots, cs, pos, q=q)
    run_decode((qr, kc, vc, table, n, g), lens)


def test_refusals():
    c = decode_case(15, [16], 4, 2, 64, 16)
    q, kc, vc, table, n, g = c
    ones = torch.ones(2, device="cuda")
    cpu = q.cpu()
    for bad, kw in [
        ((cpu, kc, vc, table, n), {}),
        ((q, kc.float(), vc, table, n), {}),
        ((q, kc, vc[:, :8], table, n), {}),
        ((q, kc, vc, table.long(), n), {}),
        ((q, kc, vc, table, n.long()), {}),
        ((q, kc, vc, table[0], n), {}),
        ((q.float(), kc, vc, table, n), {}),
        ((q[:, 0], kc, vc, table, n), {}),
        ((q, kc, vc, table, n), {"sinks": ones}),
        ((q, kc, vc, table, n), {"k_scale": torch.ones(3, device="cuda")}),
        ((q, kc, vc, table, n), {"out": torch.empty(1, 4, 32, device="cuda").bfloat16()}),
    ]:
        with pytest.raises((ValueError, TypeError)):
            mxq.paged_attention_decode(*bad, **kw)
    for bad, kw, st in [
        ((q[:, :3], kc, vc, table, n), {}, _lib.ERR_INVALID_ARG),          # 3 over 2 heads
        ((q, kc, vc, table, n), {"k_scale": ones}, _lib.ERR_INVALID_ARG),  # bf16 cache
        ((q, kc, vc, table, n), {"scale": -1.0}, _lib.ERR_INVALID_ARG),
        ((q, kc, vc, table, n), {"scale": NAN}, _lib.ERR_INVALID_ARG),
        ((q, kc, vc, table, n), {"window": -1}, _lib.ERR_INVALID_ARG),
        ((q[..., :32], kc[..., :32], vc[..., :32], table, n), {}, _lib.ERR_UNSUPPORTED),
    ]:
        with pytest.raises(mxq.MxqError) as e:
            mxq.paged_attention_decode(*bad, **kw)
        assert e.value.status == st
    k = v = randn(g, 3, 2, 64)
    slots = torch.arange(3, device="cuda")
    cs, pos = torch.ones(4, 64, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.int32)
    for args, kw in [((k, v, kc, vc, slots.int()), {}), ((k, v, kc, vc, slots, cs), {}),
                     ((k, v, kc, vc, slots, cs.double(), pos), {}),
                     ((k, v[:2], kc, vc, slots), {}), ((k, v, kc, vc.to(FP8), slots), {}),
                     ((k, v, kc, vc, slots), {"q_out": k}),
                     ((k, v, kc, vc, slots), {"q": randn(g, 2, 2, 64)})]:
        with pytest.raises((ValueError, TypeError)):
            mxq.rope_append_kv(*args, **kw)
    with pytest.raises(mxq.MxqError):
        mxq.rope_append_kv(k, v, kc, vc, slots, cs[:, :24].contiguous(), pos)   # rot % 16
    with pytest.raises(mxq.MxqError):
        mxq.rope_append_kv(k, v, kc, vc, slots, k_scale=ones, v_scale=ones)


def test_empty_calls():
    g = gen(16)
    kc = pool(g, 2, 16, 2, 64, False)
    e = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    slots = torch.empty(0, device="cuda", dtype=torch.int64)
    assert mxq.rope_append_kv(e, e, kc, kc.clone(), slots) is None
    out = mxq.paged_attention_decode(torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16),
                                     kc, kc, torch.empty(0, 3, device="cuda", dtype=torch.int32),
                                     torch.empty(0, device="cuda", dtype=torch.int32))
    assert out.shape == (0, 4, 64)


def test_workspace_given_by_the_caller():
    c = decode_case(17, [4000, 9], 8, 2, 128, 16)
    n = mxq.paged_attention_decode_workspace_size(2, 8, 2, 128)
    want = mxq.paged_attention_decode(*c[:5])
    ws = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")    # NaN bytes
    assert torch.equal(mxq.paged_attention_decode(*c[:5], workspace=ws), want)
    if n:
        with pytest.raises(mxq.MxqError) as e:
            mxq.paged_attention_decode(*c[:5], workspace=ws[:n // 2])
        assert e.value.status == _lib.ERR_INVALID_ARG


def test_c_refusals_without_touching_outputs():
    lib = _lib.load()
    c = decode_case(18, [16], 4, 2, 64, 16)
    q, kc, vc, table, n, _ = c
    out = torch.full_like(q, 3.0)
    base = [q.data_ptr(), 256, 64, 1, 4, 2, 64, kc.data_ptr(), vc.data_ptr(), _lib.BF16,
            kc.shape[0], 16, 2048, 128, 64, 2048, 128, 64, table.data_ptr(), table.shape[1],
            table.shape[1], n.data_ptr(), 0.125, 0, None, None, None, out.data_ptr(), 256, 64,
            None, None, 0, None]
    for i, val, st in [(0, None, _lib.ERR_INVALID_ARG), (0, q.data_ptr() + 2, _lib.ERR_UNSUPPORTED),
                       (2, 60, _lib.ERR_INVALID_ARG), (2, 68, _lib.ERR_UNSUPPORTED),
                       (9, _lib.F32, _lib.ERR_UNSUPPORTED), (11, 0, _lib.ERR_INVALID_ARG),
                       (13, 132, _lib.ERR_UNSUPPORTED), (19, 0, _lib.ERR_INVALID_ARG),
                       (21, None, _lib.ERR_INVALID_ARG), (27, None, _lib.ERR_INVALID_ARG),
                       (11, 1 << 30, _lib.ERR_UNSUPPORTED)]:
        args = list(base)
        args[i] = val
        assert lib.mxq_paged_attention_decode(*args) == st, i
        assert lib.mxq_last_error()
    size = ctypes.c_size_t(0)
    assert lib.mxq_paged_attention_decode_workspace_size(1, 3, 2, 64, ctypes.byref(size)) == \
        _lib.ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((out == 3).all())

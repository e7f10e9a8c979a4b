"""The attention operators at the edges of what they accept: offsets, scales, queries and
values far from the usual, and what a call must refuse."""
import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib
from attention_util import assert_within, decode_ref, prompt_ref
from test_gpu_paged_attention import bits, decode_case, gen, randn, rotate_ref, run_decode

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")


def test_prompts_that_overlap_in_many_items_are_reported():
    """More than 512 items' room, and three times as many as there is room for."""
    g = gen(40)
    T = 5000
    q, k, v = randn(g, T, 32, 64), randn(g, T, 1, 64), randn(g, T, 1, 64)
    out = torch.full_like(q, 7.0)
    mxq.sync_status()
    mxq.attention_varlen(q, k, v, torch.tensor([0, T] * 3 + [0], device="cuda").int(), out=out)
    with pytest.raises(mxq.MxqError) as e:
        mxq.sync_status()
    assert e.value.status == _lib.ERR_DEVICE
    assert bool((out == 7).all())
    lens = [700, 1, 4299]
    got = mxq.attention_varlen(q, k, v, torch.tensor([0, 700, 701, T], device="cuda").int())
    ref, _, b, _ = prompt_ref(q, k, v, lens, lens, 0.125)
    assert_within(got, ref, b, "out")


def test_a_workspace_that_is_not_one_piece_is_refused():
    """An expanded tensor has the bytes of one row, a strided one somebody else's between."""
    g = gen(41)
    q, k, v = randn(g, 40, 8, 64), randn(g, 40, 2, 64), randn(g, 40, 2, 64)
    cu = torch.tensor([0, 10, 40], device="cuda").int()
    cache = randn(g, 3, 16, 2, 64)
    table, lens = (torch.ones(n, device="cuda").int() for n in ((40, 2), (40,)))
    need = max(mxq.attention_varlen_workspace_size(40, 2, 8, 2, 64),
               mxq.paged_attention_decode_workspace_size(40, 8, 2, 64))
    for ws in (torch.zeros(1, 256, dtype=torch.uint8, device="cuda").expand(need // 256 + 1, 256),
               torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]):
        assert ws.nbytes >= need
        with pytest.raises(ValueError, match="contiguous"):
            mxq.attention_varlen(q, k, v, cu, workspace=ws)
        with pytest.raises(ValueError, match="contiguous"):
            mxq.paged_attention_decode(q, cache, cache, table, lens, workspace=ws)
    whole = torch.zeros(need // 64 + 1, 64, dtype=torch.uint8, device="cuda")
    assert torch.equal(mxq.attention_varlen(q, k, v, cu, workspace=whole),
                       mxq.attention_varlen(q, k, v, cu))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[6000, 40], [300] * 30 + [9000]])
def test_a_query_that_is_not_a_number_shows(lens, fp8):
    """Every score of the head's row is NaN, in whole sequences and in those that several
    parts share."""
    c = decode_case(44, lens, 8, 2, 128, 16, fp8)
    q, kc, vc, table, n, g = c
    ref, rl, b, bl = decode_ref(q, kc, vc, table, lens, 128 ** -0.5)
    q = q.clone()
    q[:, 5, 77] = NAN
    out, lse = mxq.paged_attention_decode(q, kc, vc, table, n, return_lse=True)
    assert bool(torch.isnan(out[:, 5]).all()) and bool(torch.isnan(lse[:, 5]).all())
    rest = [0, 1, 2, 3, 4, 6, 7]
    assert_within(out[:, rest], ref[:, rest], b[:, rest], "out")
    assert_within(lse[:, rest], rl[:, rest], bl[:, rest], "lse")


@pytest.mark.parametrize("nq,nk", [([300], [300]), ([40, 9], [20000, 9])])
def test_a_prompt_row_that_is_not_a_number_shows(nq, nk):
    """The same in whole items and in pieces."""
    g = gen(45)
    q, k, v = randn(g, sum(nq), 8, 128), randn(g, sum(nk), 2, 128), randn(g, sum(nk), 2, 128)
    ref, rl, b, bl = prompt_ref(q, k, v, nq, nk, 128 ** -0.5)
    q[7, 5, 77] = NAN
    cu = [torch.tensor([0, *n], device="cuda").cumsum(0).int() for n in (nq, nk)]
    out, lse = mxq.attention_varlen(q, k, v, *cu, return_lse=True)
    assert bool(torch.isnan(out[7, 5]).all()) and bool(torch.isnan(lse[7, 5]))
    rest = torch.ones(sum(nq), 8, dtype=torch.bool, device="cuda")
    rest[7, 5] = False
    assert_within(out[rest], ref[rest], b[rest], "out")
    assert_within(lse[rest], rl[rest], bl[rest], "lse")


LENS = [0, 1, 40, 300, 5000]


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_a_key_scale_that_is_not_finite_shows(bad, with_sinks):
    """Rows that see a key are NaN, those without keys stay what they are, and the other
    key/value head is not touched."""
    c = decode_case(41, LENS, 8, 2, 128, 16, True)
    q, kc, vc, table, n, g = c
    sinks = torch.randn(8, generator=g, device="cuda") if with_sinks else None
    ks = torch.tensor([0.02, bad], device="cuda")
    out, lse = mxq.paged_attention_decode(q, kc, vc, table, n, sinks=sinks, k_scale=ks,
                                          return_lse=True)
    assert bool(torch.isnan(out[1:, 4:]).all())
    if bad != bad:
        assert bool(torch.isnan(lse[1:, 4:]).all())
    assert not out[0].any()
    assert torch.equal(lse[0], sinks if with_sinks else torch.full_like(lse[0], -INF))
    ref, rl, b, bl = decode_ref(q, kc, vc, table, LENS, 128 ** -0.5, 0, sinks,
                                torch.full((2,), 0.02, device="cuda"))
    assert_within(out[:, :4], ref[:, :4], b[:, :4], "out")
    assert_within(lse[:, :4], rl[:, :4], bl[:, :4], "lse")


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("scales", [(0.0, 0.02), (-0.02, 0.01), (-0.0, -0.02)])
def test_zero_and_negative_key_scales(scales, window):
    """A scale of zero weighs every visible key alike."""
    c = decode_case(42, LENS, 8, 2, 64, 16, True)
    run_decode(c, LENS, window, None, torch.tensor(scales, device="cuda"),
               torch.tensor([0.02, -0.01], device="cuda"))


def test_a_small_scale_of_large_scores():
    """bf16 keys whose products with q come near 1e37, and the scale that brings them
    back to a few units."""
    lens = [1, 200, 3000]
    q, kc, vc, table, n, g = decode_case(43, lens, 8, 2, 64, 16, poison=False)
    q, kc = (q.float() * 2.0 ** 60).bfloat16(), (kc.float() * 2.0 ** 60).bfloat16()
    run_decode((q, kc, vc, table, n, g), lens, scale=2.0 ** -123)


@pytest.mark.parametrize("power", [100, 118])
def test_large_queries_over_an_e4m3_cache(power):
    """q is scaled into the range of f16 whatever its size."""
    lens = [1, 200, 3000]
    q, kc, vc, table, n, g = decode_case(45, lens, 8, 2, 64, 16, True)
    q = (q.float() * 2.0 ** power).bfloat16()
    run_decode((q, kc, vc, table, n, g), lens, scale=2.0 ** -(power + 7))


@pytest.mark.parametrize("scale", [None, 0.02, -0.02, 1.0])
@pytest.mark.parametrize("rot", [0, 64])
def test_append_keeps_the_sign_of_zero(scale, rot):
    """A quotient of zero has the sign that the division gives it."""
    g = gen(46)
    T, KV, D, page = 5, 3, 64, 4
    k, v = randn(g, T, KV, D), randn(g, T, KV, D)
    for x in (k, v):
        x[:, :, ::3] = -0.0
        x[:, :, 1::3] = 0.0
    x = torch.tensor([1e-38, -1e-38, 1e-30, -1e-30], device="cuda").bfloat16()
    v[0, 0, :4], k[0, 0, 60:] = x, x
    cs = torch.randn(9, 64, generator=g, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    kc, vc = (torch.zeros(2, page, KV, D, device="cuda").to(FP8) for _ in range(2))
    s = None if scale is None else torch.full((KV,), scale, device="cuda")
    mxq.rope_append_kv(k, v, kc, vc, torch.arange(T, device="cuda"), cs if rot else None,
                       pos if rot else None, k_scale=s, v_scale=s)
    turned = rotate_ref(k, cs[:T], rot, False)
    for cache, want in ((kc, turned), (vc, v.float())):
        want = (want / (1.0 if scale is None else scale)).clamp(-448, 448).to(FP8)
        assert torch.equal(bits(cache).view(-1, KV, D)[:T], bits(want))


@pytest.mark.parametrize("seed", range(4))
def test_append_quotients_around_midpoints(seed):
    """Scales that put quotients on and next to the middle between two codes, where a
    quotient off by one unit changes the code: 8 x 786432 of them."""
    g = gen(47 + seed)
    KV, D = 49152, 16
    # an odd multiple of half a code's step, times powers of two: a midpoint of each binade
    mid = (torch.randint(8, 16, (KV,), generator=g, device="cuda") + 0.5) / 16
    v = torch.randint(128, 256, (KV,), generator=g, device="cuda") / 256.0
    s = ((v / mid).view(torch.int32) + torch.randint(-3, 4, (KV,), generator=g, device="cuda",
                                                     dtype=torch.int32)).view(torch.float32)
    power = torch.arange(D, device="cuda") - 7
    sign = torch.randint(0, 2, (1, KV, D), generator=g, device="cuda") * 2 - 1
    v = (v[None, :, None] * 2.0 ** power * sign).bfloat16()
    kc, vc = (torch.zeros(1, 1, KV, D, device="cuda").to(FP8) for _ in range(2))
    mxq.rope_append_kv(v, v, kc, vc, torch.zeros(1, device="cuda", dtype=torch.int64), k_scale=s,
                       v_scale=s * 4)
    for cache, scale in ((kc, s), (vc, s * 4)):
        want = (v.float() / scale[None, :, None]).clamp(-448, 448).to(FP8)
        assert torch.equal(bits(cache).view(1, KV, D), bits(want))

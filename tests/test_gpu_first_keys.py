"""Windows that leave the first keys visible, in paged_attention_decode and attention_varlen,
against a plain 64-bit form within the bounds of attention_util."""
import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
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


def decode_case(lens, H, KV, D, page, window, first, fp8=False, sinks=False, seed=0):
    g = gen(seed + sum(lens) * 7 + H)
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + 1, max(1, max(need))
    kc, vc = randn(g, pages, page, KV, D), randn(g, pages, page, KV, D)
    ks = vs = None
    if fp8:
        kc, vc = ((t.float() * 100).clamp(-448, 448).to(FP8) for t in (kc, vc))
        ks, vs = (0.01 + 0.01 * torch.rand(KV, generator=g, device="cuda") for _ in range(2))
    order = torch.randperm(pages, generator=g, device="cuda").int().tolist()
    table = [[order.pop() for _ in range(n)] for n in need]
    q = randn(g, len(lens), H, D)
    s = torch.randn(H, generator=g, device="cuda") * 2 if sinks else None
    ref = []
    # the keys in between are nobody's: their pages are freed, what they hold is NaN
    kq, vq = kc.clone(), vc.clone()
    freed = [list(r) for r in table]
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        at = ints(table[b]).long()[j // page] if n else j
        seen = (j >= n - window) | (j < first)
        for t in (kq, vq):
            raw = t.view(torch.uint8) if fp8 else t
            raw[at[~seen], j[~seen] % page] = 0x7f if fp8 else NAN
        for i in range(need[b]):
            if i * page >= first and (i + 1) * page <= n - window:
                freed[b][i] = -1
        rows = []
        for h in range(H):
            kv = h // (H // KV)
            k, v = kc[at, j % page, kv].double(), vc[at, j % page, kv].double()
            if fp8:
                k, v = k * ks[kv].double(), v * vs[kv].double()
            rows.append(attend(q[b, h:h + 1], k, v, seen[None], D ** -0.5,
                               None if s is None else s[h], fp8))
        ref.append([torch.cat([r[i] for r in rows]) for i in range(4)])
    ref = [torch.stack([r[i] for r in ref]) for i in range(4)]
    t = ints([r + [-1] * (width - len(r)) for r in freed])
    out, lse = mxq.paged_attention_decode(q, kq, vq, t, ints(lens), window=window, first=first,
                                          sinks=s, k_scale=ks, v_scale=vs, return_lse=True)
    mxq.sync_status()
    assert_within(out, ref[0], ref[2], "out")
    assert_within(lse, ref[1], ref[3], "lse")


@pytest.mark.parametrize("lens", [[0, 1, 5], [15, 16, 17, 33], [100, 300, 40, 2], [3000],
                                  [700, 1, 2500, 64, 65]])
@pytest.mark.parametrize("window,first", [(1, 1), (16, 4), (17, 16), (20, 33), (128, 100),
                                          (100, 1000), (2000, 5)])
@pytest.mark.parametrize("D,fp8", [(64, False), (128, False), (64, True), (128, True)])
def test_decode(lens, window, first, D, fp8):
    decode_case(lens, 4, 2, D, 16, window, first, fp8, sinks=window == 16)


@pytest.mark.parametrize("page", [1, 3, 24, 128])
@pytest.mark.parametrize("H,KV", [(1, 1), (20, 1), (6, 3)])
def test_decode_pages_and_groups(page, H, KV):
    decode_case([333, 90, 0, 4], H, KV, 128, page, 50, 21, seed=3)


def test_decode_long_and_many():
    decode_case([20000], 8, 2, 64, 64, 3000, 2000, seed=4)
    decode_case([(i * 37) % 400 for i in range(300)], 2, 1, 64, 16, 33, 18, seed=5)


def test_first_without_a_window_changes_nothing():
    g = gen(6)
    kc, vc, q = randn(g, 9, 16, 2, 64), randn(g, 9, 16, 2, 64), randn(g, 1, 4, 64)
    t, n = torch.arange(9, device="cuda").int()[None], ints([140])
    a = mxq.paged_attention_decode(q, kc, vc, t, n)
    assert torch.equal(a, mxq.paged_attention_decode(q, kc, vc, t, n, first=7))
    x, cu = randn(g, 50, 8, 64), ints([0, 20, 50])
    a = mxq.attention_varlen(x[:, :4], x[:, 4:6], x[:, 6:], cu)
    assert torch.equal(a, mxq.attention_varlen(x[:, :4], x[:, 4:6], x[:, 6:], cu, first=7))


def prompt_case(nq, nk, H, KV, D, window, first, sinks=False, seed=0):
    g = gen(seed + sum(nq) * 7 + H)
    q, k, v = randn(g, sum(nq), H, D), randn(g, sum(nk), KV, D), randn(g, sum(nk), KV, D)
    s = torch.randn(H, generator=g, device="cuda") * 2 if sinks else None
    cu = lambda x: ints([sum(x[:i]) for i in range(len(x) + 1)])
    out, lse = mxq.attention_varlen(q, k, v, cu(nq), cu(nk), window=window, first=first, sinks=s,
                                    return_lse=True)
    mxq.sync_status()
    a = b = 0
    for n, m in zip(nq, nk):
        at = torch.arange(n, device="cuda")[:, None] + m - n
        j = torch.arange(m, device="cuda")[None]
        seen = (j <= at) & ((j > at - window) | (j < first))
        for h in range(H):
            r = attend(q[a:a + n, h], k[b:b + m, h // (H // KV)], v[b:b + m, h // (H // KV)], seen,
                       D ** -0.5, None if s is None else s[h])
            assert_within(out[a:a + n, h], r[0], r[2], "out")
            assert_within(lse[a:a + n, h], r[1], r[3], "lse")
        a, b = a + n, b + m


@pytest.mark.parametrize("window,first", [(1, 1), (16, 4), (128, 128), (100, 129), (300, 5),
                                          (64, 700), (2000, 3)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq", [[1], [300], [129, 1, 640, 0, 77], [1500]])
def test_prompt(nq, window, first, D):
    prompt_case(nq, nq, 4, 2, D, window, first, sinks=first == 4)


@pytest.mark.parametrize("nq,nk", [([1], [900]), ([100], [2000]), ([3, 200], [1900, 200]),
                                   ([200], [50]), ([20, 600], [4000, 3000])])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_chunks(nq, nk, D):
    """Chunks behind a history, cut into pieces where few rows see many keys."""
    prompt_case(nq, nk, 8, 2, D, 1024, 300, seed=1)
    prompt_case(nq, nk, 8, 2, D, 40, 140, seed=2, sinks=True)


def test_prompt_many_items():
    prompt_case([3] * 700, [3] * 700, 1, 1, 64, 1, 1, seed=7)
    prompt_case([700] * 4 + [2] * 600, [700] * 4 + [2] * 600, 2, 1, 64, 50, 40, seed=8)


def test_prompt_keys_between_are_not_loaded():
    """Blocks of 128 keys that no row sees may hold anything."""
    g = gen(9)
    n, m = 40, 3000
    q, k, v = randn(g, n, 4, 64), randn(g, m, 2, 64), randn(g, m, 2, 64)
    cu = [ints([0, n]), ints([0, m])]
    want = mxq.attention_varlen(q, k, v, *cu, window=200, first=10)
    k[128:2688], v[128:2688] = NAN, NAN
    assert torch.equal(want, mxq.attention_varlen(q, k, v, *cu, window=200, first=10))

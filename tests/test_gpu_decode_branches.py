"""paged_attention_decode where its work is laid out in other ways: more sequences than
entries of the prefix table or threads, more key/value heads than warps, caches
with strides of their own.  References in 64 bits over padded sequences, bounds as in
attention_util."""
import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from attention_util import assert_within
from test_gpu_paged_attention import decode_case, run_decode

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
NAN = float("nan")


def reference(q, kc, vc, table, n, window):
    """(out, lse, their bounds), for few keys a sequence or few sequences."""
    B, H, D = q.shape
    KV, page, L = kc.shape[2], kc.shape[1], max(1, int(n.max()))
    j = torch.arange(L, device="cuda")
    visible = (j < n[:, None]) & (j >= (n[:, None] - window if window else 0))    # [B, L]
    at = torch.where(visible, table.gather(1, (j // page).expand(B, L)).long(), 0)
    k, v = (torch.where(visible[..., None, None], c.view(torch.uint8 if c.dtype == FP8 else
                                                         torch.int16)[at, j % page], 0)
            .view(c.dtype).double() for c in (kc, vc))                            # [B, L, KV, D]
    x = q.double().view(B, KV, H // KV, D)
    scale, f16 = D ** -0.5, kc.dtype == FP8
    s = torch.einsum("bghd,blgd->bghl", x, k) * scale
    size = (torch.einsum("bghd,blgd->bghl", x.abs(), k.abs()) * scale).amax(-1)
    s = torch.where(visible[:, None, None], s, -float("inf"))
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse == -float("inf"), 0.0, lse)[..., None])
    out, A = (torch.einsum("bghl,blgd->bghd", w, t) for t in (v, v.abs()))
    u = 2.0 ** -11 if f16 else 2.0 ** -8
    bound = 2.0 ** -8 * out.abs() + (u + 2.0 ** -11) * A + 2.0 ** -134
    if f16:
        bound += 2.0 ** -25 * w.amax(-1)[..., None] * v.abs().sum(1)[:, :, None]
    lb = D * 2.0 ** -24 * size + 2.0 ** -18 + 2.0 ** -22 * torch.where(
        lse == -float("inf"), 0.0, lse.abs())
    return (out.reshape(B, H, D), lse.reshape(B, H), bound.reshape(B, H, D), lb.reshape(B, H))


def check(seed, lens, H, KV, D, fp8, window=0, longest=64):
    """lens: up to `longest` each, but for a few."""
    q, kc, vc, table, n, _ = decode_case(seed, lens, H, KV, D, 16, fp8)
    out, lse = mxq.paged_attention_decode(q, kc, vc, table, n, window=window, return_lse=True)
    mxq.sync_status()
    long = n > longest
    for rows in (torch.where(~long)[0], *torch.where(long)[0][:, None]):
        ref, rl, b, bl = reference(q[rows], kc, vc, table[rows], n[rows], window)
        assert_within(out[rows], ref, b, "out")
        assert_within(lse[rows], rl, bl, "lse")


@pytest.mark.parametrize("B", [256, 257, 2047, 2048, 2049, 4097, 5000])
@pytest.mark.parametrize("D,fp8", [(64, False), (128, True)])
@pytest.mark.parametrize("window", [0, 24])
def test_many_sequences(B, D, fp8, window):
    """Several entries of the prefix table a thread, several sequences an entry; long
    sequences among them are cut and joined."""
    lens = [(i * 29) % 41 for i in range(B)]
    check(B, lens, 4, 2, D, fp8, window)
    for at, n in ((0, 3000), (B // 3, 700), (B // 2, 2000), (B // 2 + 1, 2500), (B - 1, 5000)):
        lens[at] = n
    check(B + 1, lens, 4, 2, D, fp8, window)


@pytest.mark.parametrize("KV,G", [(1217, 1), (1300, 3), (650, 20)])
@pytest.mark.parametrize("fp8", [False, True])
def test_more_heads_than_warps(KV, G, fp8):
    """A warp takes several heads' tasks in turn, and no sequence is cut."""
    check(KV, [0, 5, 200, 33, 64], KV * G, KV, 64, fp8, 0, 300)
    check(KV, [150, 7], KV * G, KV, 64, fp8, 40, 300)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_caches_with_strides_of_their_own(D, fp8):
    """A head-major cache beside a token-major one, either way, and rows with gaps."""
    lens = [0, 1, 40, 555, 3000]
    q, kc, vc, table, n, g = decode_case(7, lens, 8, 2, D, 16, fp8)

    def head_major(c):
        return c.transpose(1, 2).contiguous().transpose(1, 2)

    def gaps(c):
        wide = torch.full((*c.shape[:2], 3, 2 * D), NAN, device="cuda").to(c.dtype)
        wide[:, :, :2, D:] = c
        return wide[:, :, :2, D:]

    first = None
    for k, v in ((kc, vc), (head_major(kc), vc), (kc, head_major(vc)), (gaps(kc), vc),
                 (head_major(kc), gaps(vc))):
        out, lse = run_decode((q, k, v, table, n, g), lens)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
        run_decode((q, k, v, table, n, g), lens, 70)

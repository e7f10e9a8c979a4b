"""The attention operators at the edges of what they accept: offsets, scales, queries and
values far from the usual, and what a call must refuse."""
import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib
from attention_util import assert_within, prompt_ref
from test_gpu_prompt_attention import gen, randn

pytestmark = pytest.mark.gpu


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

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

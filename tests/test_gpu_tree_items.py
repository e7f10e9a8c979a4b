"""CTAs of paged_attention_tree that take items of different sizes one after the other: a full one of
two tiles, then one of few rows, whose queries are there at once."""
import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from attention_util import assert_within
from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


# 2 * 128 / G rows and 1 by turns: within a few blocks of keys, whose items stay whole, and over
# longer ones, whose pieces leave partial results
@pytest.mark.parametrize("lens", [(60, 7), (700, 90), (1500, 300)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_full_items_and_short_ones_by_turns(lens, D, fp8):
    n = 240
    c = Case([32, 1] * (n // 2), [lens[i & 1] + i % 5 for i in range(n)], 16, 2, D, 64, fp8=fp8,
             seed=31)
    want, wl = c.call()
    for _ in range(60):
        out, lse = c.call()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    mxq.sync_status()
    # some of the heads, one of each key/value head
    heads = [3, 12]
    c.q, c.H = c.q[:, heads].contiguous(), 2
    ref = c.reference()
    assert_within(want[:, heads], ref[0], ref[2], "out")
    assert_within(wl[:, heads], ref[1], ref[3], "lse")

"""What the attention operators' Python calls refuse before any entry point or
device is reached (no GPU needed)."""
import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq

BF = torch.bfloat16
Q = torch.zeros(2, 4, 64, dtype=BF)
CACHE = torch.zeros(3, 16, 2, 64, dtype=BF)
TABLE = torch.zeros(2, 3, dtype=torch.int32)
LENS = torch.zeros(2, dtype=torch.int32)
KV = torch.zeros(2, 2, 64, dtype=BF)


@pytest.mark.parametrize("call", [
    lambda: mxq.rope_append_kv(KV, KV, CACHE, CACHE, torch.zeros(2, dtype=torch.int64)),
    lambda: mxq.paged_attention_decode(Q, CACHE, CACHE, TABLE, LENS),
    lambda: mxq.attention_varlen(Q, KV, KV, torch.zeros(3, dtype=torch.int32))])
def test_cpu_tensors_are_refused(call):
    with pytest.raises(ValueError, match="CUDA tensors"):
        call()


@pytest.mark.parametrize("call", [
    lambda: mxq.rope_append_kv(None, KV, CACHE, CACHE, None),
    lambda: mxq.rope_append_kv(KV, [1], CACHE, CACHE, LENS),
    lambda: mxq.paged_attention_decode(Q, CACHE, CACHE, TABLE, 5),
    lambda: mxq.attention_varlen(Q, KV, KV, LENS, "x")])
def test_what_is_no_tensor_is_refused(call):
    with pytest.raises(TypeError, match="must be a tensor"):
        call()

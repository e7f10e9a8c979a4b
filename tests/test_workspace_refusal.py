"""A caller's workspace is taken by its address and bytes, so it has to be one piece on the
GPU: refused on the host otherwise (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq


def on_gpu(t):
    return SimpleNamespace(is_cuda=True, get_device=lambda: 0, is_contiguous=t.is_contiguous)


def test_workspaces(monkeypatch):
    monkeypatch.setattr(mxq, "_current_device", lambda: 0)
    one = torch.zeros(1, 256, dtype=torch.uint8)
    mxq._need_whole(None)
    mxq._need_whole(on_gpu(one))
    mxq._need_whole(on_gpu(one[:, :0]))
    for bad in (on_gpu(one.expand(9, 256)), on_gpu(one[:, ::2]), one):
        with pytest.raises(ValueError):
            mxq._need_whole(bad)


@pytest.mark.gpu
def test_calls_look_at_it():
    d = "cuda"
    a, w = torch.zeros(4, 256, device=d).bfloat16(), torch.zeros(128, 256, device=d).to(
        torch.float8_e4m3fn)
    ws = torch.zeros(1, 256, dtype=torch.uint8, device=d).expand(1 << 16, 256)
    with pytest.raises(ValueError, match="contiguous"):
        mxq.fp8_scaled_mm(a, w, torch.ones(1, device=d), workspace=ws)
    with pytest.raises(ValueError, match="contiguous"):
        mxq.fused_experts(a, *[a] * 6, workspace=ws)

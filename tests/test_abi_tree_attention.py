"""Host-side refusals of the tree attention entry point and of its Python call."""
import ctypes

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib

P = 1 << 20                        # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED = _lib.OK, _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED

TREE = dict(q=P, sq_t=512, sq_h=64, T=7, Hq=8, Hkv=2, D=64, k_cache=P, v_cache=P,
            dtype=_lib.BF16, pages=3, page_size=16, ckp=2048, ckt=128, ckh=64, cvp=2048, cvt=128,
            cvh=64, table=P, ld_table=3, max_pages=3, lens=P, cu=P, parents=P, B=2, scale=0.125,
            window=0, first=0, sinks=None, k_scale=None, v_scale=None, out=P, so_t=512, so_h=64,
            lse=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("changed,status", [
    (dict(B=0), OK), (dict(T=0), OK), (dict(B=-1), INVALID), (dict(T=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(Hq=7), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=258), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(window=-1), INVALID), (dict(first=-1), INVALID),
    (dict(pages=0), INVALID), (dict(page_size=0), INVALID), (dict(B=65536), UNSUPPORTED),
    (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(ld_table=2), INVALID), (dict(table=None), INVALID),
    (dict(max_pages=1 << 28, ld_table=1 << 28), UNSUPPORTED), (dict(lens=None), INVALID),
    (dict(cu=None), INVALID), (dict(cu=P + 2), INVALID), (dict(parents=P + 1), INVALID),
    (dict(sinks=P + 1), INVALID), (dict(lse=P + 2), INVALID), (dict(q=None), INVALID),
    (dict(q=P + 8), UNSUPPORTED), (dict(out=None), INVALID), (dict(so_h=60), INVALID),
    (dict(dtype=7), UNSUPPORTED), (dict(k_scale=P), INVALID), (dict(ckh=68), UNSUPPORTED),
    (dict(dtype=_lib.E4M3, ckh=72), UNSUPPORTED), (dict(v_cache=None), INVALID),
    (dict(k_cache=P + 8), UNSUPPORTED), (dict(ckp=1 << 35), UNSUPPORTED),
    (dict(cvt=1 << 36), UNSUPPORTED)])
def test_tree(changed, status):
    lib = _lib.load()
    args = dict(TREE)
    assert set(changed) <= set(args)
    args.update(changed)
    assert lib.mxq_paged_attention_tree(*args.values()) == status
    assert status == OK or lib.mxq_last_error()


def test_workspace_query():
    f, n = _lib.load().mxq_paged_attention_tree_workspace_size, ctypes.c_size_t(9)
    assert f(0, 4, 8, 2, 64, ctypes.byref(n)) == OK and n.value == 0
    assert f(4, 0, 8, 2, 64, ctypes.byref(n)) == OK and n.value == 0
    for args in ((1, 1, 8, 3, 64), (-1, 1, 8, 2, 64), (1, -1, 8, 2, 64), (1, 1, 8, 0, 64)):
        assert f(*args, ctypes.byref(n)) == INVALID
    assert f(1, 1, 8, 2, 80, ctypes.byref(n)) == UNSUPPORTED
    assert f(1, 1, 8, 2, 64, None) == INVALID


def test_python_call_refuses():
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 64,
                                                                     dtype=torch.bfloat16)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors"):
        mxq.paged_attention_tree(q, kv, kv, t, n, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="must be a tensor"):
        mxq.paged_attention_tree(q, kv, kv, t, n, [0, 1, 2])

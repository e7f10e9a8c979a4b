"""Host-side refusals of the paged cache and attention entry points: each
argument error returns its documented status before any device is touched
(these calls need no GPU), and empty problems are accepted."""
import ctypes

import pytest

from mxfp4_quantized_gemm_token_gb300 import _lib

P = 1 << 20                        # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED = _lib.OK, _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def call(fn, defaults, **changed):
    args = dict(defaults)
    for k, v in changed.items():
        assert k in args, k
        args[k] = v
    return fn(*args.values())


APPEND = dict(q=P, sq_t=512, sq_h=64, Hq=8, q_out=P, so_t=512, so_h=64, k=P, sk_t=128, sk_h=64,
              v=P, sv_t=128, sv_h=64, T=4, Hkv=2, D=64, cos_sin=P, max_pos=100, rot=64,
              positions=P, interleaved=0, slots=P, k_cache=P, v_cache=P, dtype=_lib.BF16, pages=3,
              page_size=16, ckp=2048, ckt=128, ckh=64, cvp=2048, cvt=128, cvh=64, k_scale=None,
              v_scale=None, stream=None)

DECODE = dict(q=P, sq_b=512, sq_h=64, B=2, Hq=8, Hkv=2, D=64, k_cache=P, v_cache=P,
              dtype=_lib.BF16, pages=3, page_size=16, ckp=2048, ckt=128, ckh=64, cvp=2048, cvt=128,
              cvh=64, table=P, ld_table=3, max_pages=3, lens=P, scale=0.125, window=0, sinks=None,
              k_scale=None, v_scale=None, out=P, so_b=512, so_h=64, lse=None, ws=None, ws_bytes=0,
              stream=None)

PROMPT = dict(q=P, sq_t=512, sq_h=64, k=P, sk_t=128, sk_h=64, v=P, sv_t=128, sv_h=64, cu_q=P,
              cu_k=P, B=2, Tq=9, Tk=9, Hq=8, Hkv=2, D=64, scale=0.125, causal=1, window=0,
              sinks=None, out=P, so_t=512, so_h=64, lse=None, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("changed,status", [
    (dict(T=0), OK), (dict(T=-1), INVALID), (dict(Hkv=0), INVALID), (dict(D=24), UNSUPPORTED),
    (dict(D=528), UNSUPPORTED), (dict(rot=24), INVALID), (dict(rot=80), INVALID),
    (dict(rot=-16), INVALID), (dict(pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(Hq=0), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(slots=None), INVALID), (dict(slots=P + 4), INVALID), (dict(cos_sin=None), INVALID),
    (dict(positions=None), INVALID), (dict(max_pos=0), INVALID), (dict(cos_sin=P + 4), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(k=P + 2), UNSUPPORTED), (dict(sk_t=132), UNSUPPORTED), (dict(sk_h=60), INVALID),
    (dict(sq_h=68), UNSUPPORTED), (dict(so_t=60), INVALID), (dict(so_h=128), INVALID),
    (dict(dtype=_lib.F32), UNSUPPORTED), (dict(k_scale=P), INVALID), (dict(ckp=10), INVALID),
    (dict(cvt=132), UNSUPPORTED), (dict(dtype=_lib.E4M3, ckt=132), UNSUPPORTED),
    (dict(dtype=_lib.E4M3, k_scale=P + 2), INVALID)])
def test_append(lib, changed, status):
    assert call(lib.mxq_rope_append_kv, APPEND, **changed) == status
    if status != OK:
        assert lib.mxq_last_error()


@pytest.mark.parametrize("changed,status", [
    (dict(B=0), OK), (dict(B=-1), INVALID), (dict(Hq=7), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(window=-1), INVALID), (dict(pages=0), INVALID), (dict(page_size=-1), INVALID),
    (dict(B=65536), UNSUPPORTED), (dict(max_pages=1 << 28, ld_table=1 << 28), UNSUPPORTED),
    (dict(max_pages=-1), INVALID), (dict(ld_table=2), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(lens=P + 2), INVALID), (dict(sinks=P + 1), INVALID),
    (dict(lse=P + 2), INVALID), (dict(q=None), INVALID), (dict(q=P + 8), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(so_h=60), INVALID), (dict(dtype=7), UNSUPPORTED),
    (dict(k_scale=P), INVALID), (dict(ckh=68), UNSUPPORTED),
    (dict(dtype=_lib.E4M3, ckh=72), UNSUPPORTED), (dict(v_cache=None), INVALID)])
def test_decode(lib, changed, status):
    assert call(lib.mxq_paged_attention_decode, DECODE, **changed) == status
    if status != OK:
        assert lib.mxq_last_error()


@pytest.mark.parametrize("changed,status", [
    (dict(B=0), OK), (dict(Tq=0), OK), (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID),
    (dict(Hq=3), INVALID), (dict(D=32), UNSUPPORTED), (dict(scale=-1.0), INVALID),
    (dict(window=-1), INVALID), (dict(window=4, causal=0), INVALID), (dict(B=65536), UNSUPPORTED),
    (dict(Tq=(1 << 30) + 1), UNSUPPORTED), (dict(cu_q=None), INVALID), (dict(cu_k=None), INVALID),
    (dict(cu_k=P + 2), INVALID), (dict(sinks=P + 2), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=P + 4), UNSUPPORTED), (dict(sk_h=60), INVALID),
    (dict(sk_t=132), UNSUPPORTED), (dict(out=None), INVALID), (dict(so_t=60), INVALID),
    (dict(so_t=500), UNSUPPORTED)])
def test_prompt(lib, changed, status):
    assert call(lib.mxq_attention_varlen, PROMPT, **changed) == status
    if status != OK:
        assert lib.mxq_last_error()


def test_workspace_queries(lib):
    n = ctypes.c_size_t(9)
    d, v = lib.mxq_paged_attention_decode_workspace_size, lib.mxq_attention_varlen_workspace_size
    assert d(0, 8, 2, 64, ctypes.byref(n)) == OK and n.value == 0
    assert v(0, 0, 8, 2, 64, ctypes.byref(n)) == OK and n.value == 0
    for args in ((1, 8, 3, 64), (1, 8, 0, 64), (-1, 8, 2, 64)):
        assert d(*args, ctypes.byref(n)) == INVALID
        assert v(1, *args, ctypes.byref(n)) == INVALID
    assert d(1, 8, 2, 80, ctypes.byref(n)) == UNSUPPORTED
    assert d(1, 8, 2, 64, None) == INVALID and v(1, 1, 8, 2, 64, None) == INVALID

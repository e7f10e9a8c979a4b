"""Host-side refusals of the page entry points, before any device is touched, and
of their Python calls."""
import ctypes

import pytest
import torch

import mxfp4_quantized_gemm_token_gb300 as mxq
from mxfp4_quantized_gemm_token_gb300 import _lib

P = 1 << 20                        # never dereferenced: validation fails first
FAR = 1 << 24
OK, INVALID, UNSUPPORTED = _lib.OK, _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def call(lib, name, defaults, changed):
    args = dict(defaults)
    for k, v in changed.items():
        assert k in args, k
        args[k] = v
    return getattr(lib, name)(*args.values())


RESIZE = dict(table=P, ld=8, B=3, max_pages=8, lens=P, new=P, refs=P, pages=20, page_size=16,
              window=0, first=0, ws=P, ws_bytes=1 << 20, stream=None)
FORK = dict(table=P, ld=8, B=3, max_pages=8, lens=P, refs=P, pages=20, page_size=16, parents=P, n=4,
            new=FAR, ld_new=8, new_lens=P, copies=P, ws=P, ws_bytes=1 << 20, stream=None)
CACHE = dict(k=P, v=P, dtype=_lib.BF16, pages=3, page_size=16, Hkv=2, D=64, ckp=2048, ckt=128,
             ckh=64, cvp=2048, cvt=128, cvh=64)
COPY = dict(CACHE, copies=P, n=2, stream=None)
COMPACT = dict(CACHE, table=P, ld=8, B=3, max_pages=8, starts=P, kept=P, ld_kept=5, most=5,
               counts=P, stream=None)


@pytest.mark.parametrize("changed,status", [
    (dict(B=0), OK), (dict(B=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(pages=0), INVALID),
    (dict(pages=1 << 31), INVALID), (dict(page_size=0), INVALID), (dict(refs=None), INVALID),
    (dict(refs=P + 4), UNSUPPORTED), (dict(max_pages=1 << 27, ld=1 << 27), UNSUPPORTED),
    (dict(B=1 << 31), UNSUPPORTED), (dict(window=-1), INVALID), (dict(first=-1), INVALID),
    (dict(table=None), INVALID), (dict(table=P + 2), INVALID), (dict(ld=7), INVALID),
    (dict(lens=None), INVALID), (dict(new=None), INVALID), (dict(new=P + 1), INVALID),
    (dict(ws=None), INVALID), (dict(ws_bytes=100), INVALID), (dict(ws=P + 16), INVALID)])
def test_resize(lib, changed, status):
    assert call(lib, "mxq_cache_resize", RESIZE, changed) == status
    assert status == OK or lib.mxq_last_error()


@pytest.mark.parametrize("changed,status", [
    (dict(B=0, n=0), OK), (dict(n=-1), INVALID), (dict(n=1 << 31), UNSUPPORTED),
    (dict(parents=None), INVALID), (dict(new=None), INVALID), (dict(new_lens=None), INVALID),
    (dict(copies=None), INVALID), (dict(copies=P + 2), INVALID), (dict(ld_new=7), INVALID),
    (dict(new=P + 64), INVALID), (dict(new=P), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(refs=None), INVALID), (dict(ws_bytes=0), INVALID)])
def test_fork(lib, changed, status):
    assert call(lib, "mxq_cache_fork", FORK, changed) == status
    assert status == OK or lib.mxq_last_error()


@pytest.mark.parametrize("output", ["new", "new_lens", "copies"])
@pytest.mark.parametrize("read", ["table", "lens", "parents", "refs"])
def test_fork_results_lie_apart_from_what_it_reads(lib, output, read):
    """Side by side with it on either side it is the workspace that is refused."""
    apart = dict(table=1 << 24, lens=2 << 24, parents=3 << 24, refs=4 << 24, new=5 << 24,
                 new_lens=6 << 24, copies=7 << 24, ws=None)
    size = dict(table=(3 - 1) * 8 + 8, lens=3, parents=4, refs=20, new=(4 - 1) * 8 + 8, new_lens=4,
                copies=12)
    for at, meet in ((4 * size[read] - 16, True), (4 * size[read], False),
                     (-4 * size[output] + 16, True), (-4 * size[output], False)):
        args = dict(apart, **{output: apart[read] + at})
        assert call(lib, "mxq_cache_fork", FORK, args) == INVALID
        assert (b"must not overlap" in lib.mxq_last_error()) == meet


BAD_CACHE = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=P + 8), UNSUPPORTED),
    (dict(dtype=_lib.F32), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=0), INVALID),
    (dict(D=528), UNSUPPORTED), (dict(Hkv=0), INVALID), (dict(Hkv=70000), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(page_size=0), INVALID), (dict(ckt=60), INVALID),
    (dict(cvh=68), UNSUPPORTED), (dict(dtype=_lib.E4M3, ckp=2056), UNSUPPORTED),
    (dict(cvp=10), INVALID)]


@pytest.mark.parametrize("changed,status", BAD_CACHE + [
    (dict(n=0), OK), (dict(n=-1), INVALID), (dict(copies=None), INVALID),
    (dict(copies=P + 3), INVALID), (dict(n=1 << 31), UNSUPPORTED)])
def test_copy_pages(lib, changed, status):
    assert call(lib, "mxq_cache_copy_pages", COPY, changed) == status
    assert status == OK or lib.mxq_last_error()


@pytest.mark.parametrize("changed,status", BAD_CACHE + [
    (dict(B=0), OK), (dict(most=0), OK), (dict(B=-1), INVALID), (dict(most=-1), INVALID),
    (dict(B=65536), UNSUPPORTED), (dict(most=1 << 31, ld_kept=1 << 31), UNSUPPORTED),
    (dict(max_pages=1 << 27, ld=1 << 27), UNSUPPORTED), (dict(ld=7), INVALID),
    (dict(table=None), INVALID), (dict(starts=None), INVALID), (dict(kept=None), INVALID),
    (dict(counts=None), INVALID), (dict(kept=P + 2), INVALID), (dict(ld_kept=4), INVALID)])
def test_compact(lib, changed, status):
    assert call(lib, "mxq_cache_compact", COMPACT, changed) == status
    assert status == OK or lib.mxq_last_error()


def test_workspace_query(lib):
    n = ctypes.c_size_t(0)
    f = lib.mxq_cache_pages_workspace_size
    assert f(4, 100, ctypes.byref(n)) == OK and n.value >= 4 * 8 + 100 * 4
    assert f(0, 1, ctypes.byref(n)) == OK
    for rows, pages in ((-1, 4), (4, 0), (1 << 31, 4), (4, 1 << 31)):
        assert f(rows, pages, ctypes.byref(n)) == INVALID
    assert f(4, 4, None) == INVALID


N, T = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
KV = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda x: mxq.cache_resize(x, N, N, N, 16), lambda x: mxq.cache_fork(x, N, N, N, 16),
    lambda x: mxq.cache_copy_pages(KV, KV, x), lambda x: mxq.cache_compact(KV, KV, x, N, T, N)])
def test_python_calls_refuse(call):
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(T)
    with pytest.raises(TypeError, match="must be a tensor"):
        call(None)

"""Sizes and scales at the ends of the attention entry points' ranges are compared without
overflow (no GPU needed: each is refused before a device is looked for)."""
import pytest

from mxfp4_quantized_gemm_token_gb300 import _lib
from test_abi_attention import APPEND, DECODE, INVALID, PROMPT, UNSUPPORTED, call


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.mark.parametrize("max_pages,page_size", [(1 << 40, 1 << 24), (1 << 33, 1 << 30),
                                                 ((1 << 62) + 1, 16), (1 << 30, 1), (2, 1 << 29)])
def test_keys_of_a_sequence(lib, max_pages, page_size):
    assert call(lib.mxq_paged_attention_decode, DECODE, max_pages=max_pages, ld_table=max_pages,
                page_size=page_size) == UNSUPPORTED
    assert b"2^30 keys" in lib.mxq_last_error()


def test_cache_slots(lib):
    assert call(lib.mxq_rope_append_kv, APPEND, pages=1 << 40, page_size=1 << 24) == INVALID
    assert b"2^60 cache slots" in lib.mxq_last_error()


@pytest.mark.parametrize("scale", [2.4e38, 3.3e38])
def test_scales_whose_exponent_would_overflow(lib, scale):
    for fn, args in ((lib.mxq_paged_attention_decode, DECODE), (lib.mxq_attention_varlen, PROMPT)):
        assert call(fn, args, scale=scale) == INVALID
        assert b"log2 e" in lib.mxq_last_error()
        call(fn, args, scale=2.3e38)                     # goes on to the workspace or the device
        assert b"log2 e" not in lib.mxq_last_error()

"""Refusals of the attention entry points whose window leaves first keys visible."""
import pytest

from mxfp4_quantized_gemm_token_gb300 import _lib
from test_abi_attention import DECODE, PROMPT, INVALID, OK, P, UNSUPPORTED


def call(fn, defaults, changed):
    args = {}
    for k, v in defaults.items():
        args[k] = v
        if k == "window":
            args["first"] = 4
    assert set(changed) <= set(args)
    args.update(changed)
    return fn(*args.values())


@pytest.mark.parametrize("changed,status", [
    (dict(B=0), OK), (dict(first=-1), INVALID), (dict(window=-1), INVALID),
    (dict(first=1 << 30, B=0), OK), (dict(Hq=7), INVALID), (dict(lens=None), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(sinks=P + 1), INVALID)])
def test_decode(changed, status):
    assert call(_lib.load().mxq_paged_attention_decode_ex, DECODE, changed) == status


@pytest.mark.parametrize("changed,status", [
    (dict(B=0), OK), (dict(first=-1), INVALID), (dict(window=4, causal=0), INVALID),
    (dict(Tq=0), OK), (dict(cu_q=None), INVALID), (dict(v=P + 4), UNSUPPORTED)])
def test_prompt(changed, status):
    assert call(_lib.load().mxq_attention_varlen_ex, PROMPT, changed) == status

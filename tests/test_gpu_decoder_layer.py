"""The example decoder layer: prompts, the cache they leave, and decode steps.

The last prompt token computed twice, by attention over the packed prompt and
as a decode step over the cache, may differ by the roundings of the two
attentions (2^-8 of the attention output each, bf16 cache) and by the cache's own
rounding (e4m3: 2^-4 of every key and value, which moves the scores as well);
the attention is one of three terms of the layer's output."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.mark.parametrize("cache,window,bound", [("bf16", 0, 2.0 ** -6), ("bf16", 16, 2.0 ** -6),
                                                ("e4m3", 0, 2.0 ** -3)])
def test_prompt_and_decode_agree(cache, window, bound):
    import decoder_layer
    difference, tokens = decoder_layer.run(cache=cache, steps=4, window=window)
    assert difference < bound
    assert tokens.shape == (3, 1024) and bool(torch.isfinite(tokens.float()).all())

"""The example that runs the attention-side operators between the quantized products."""
import os
import runpy

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")


def test_chunks_and_single_tokens_agree_with_whole_sequences():
    """bf16 q|k|v, weights of the softmax and two output roundings (2^-9 rms each at most) on values that
    pass two products: a row differs by well under 2e-2 of its norm."""
    assert runpy.run_path(PATH)["main"]() < 2e-2

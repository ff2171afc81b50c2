"""The example that runs the serving calls together (examples/decoder_layer.py)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decoder_layer():
    """Prompt, single tokens and evictions; the attention is off by its output's rounding (half a step of bf16) and the
    numerators' (2^-12 each), relative to the largest output."""
    import decoder_layer
    error, evictions = decoder_layer.main()
    assert evictions == 1
    assert error <= torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -12 + 2.0 ** -16

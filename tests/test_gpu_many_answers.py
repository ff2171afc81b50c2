"""The example that runs the calls around forked sequences together (examples/many_answers.py)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kw", [{}, dict(prompts=1, prompt=64, answers=2, generate=5, every=2),
                                dict(prompts=5, prompt=700, answers=4, generate=70, every=20)])
def test_many_answers(kw):
    """Forks, copies, shared attention and compaction: the attention is off by its output's rounding (half a step of bf16) and
    the numerators' (2^-12 each), relative to the largest output; no page is owned by anyone in the end."""
    import many_answers
    error, forks, used, owned = many_answers.main(**kw)
    assert forks == 1 + kw.get("generate", 40) // kw.get("every", 12) and used > 0 and owned == 0
    assert error <= torch.finfo(torch.bfloat16).eps / 2 + 2.0 ** -12 + 2.0 ** -16

"""The example layer: prompts and then single tokens give what longer prompts give.

The prompt's form rounds operands of its products and both forms round the outputs, each by at
most 2^-8 of a term; projections of up to 2^9 terms of random sign then differ by a few times 2^-8
of their root mean square, and their largest of some thousands by up to five times that: 2^-8 * 3 *
5 = 0.06 at most, and the residual stream, whose size is that of the block's output, halves it.
"""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("more", [{}, dict(heads=6, value_size=80, groups=3, key_size=72, width=256),
                                  dict(heads=4, value_size=32, groups=4, key_size=16, lengths=(1, 2, 3, 300)),
                                  dict(heads=4, value_size=128, groups=2, key_size=128, lengths=(700, 64))])
def test_tokens_continue_prompts(more):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if ROOT not in sys.path:
        sys.path.insert(0, ROOT)
    spec = importlib.util.spec_from_file_location("gated_delta_layer", os.path.join(ROOT, "examples", "gated_delta_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.run(**more) <= 0.06

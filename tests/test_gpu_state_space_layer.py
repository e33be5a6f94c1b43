"""The example layer: prompts and then single tokens give what longer prompts give.

Both ways round the convolution's and the recurrence's results to BF16 at different
places (the prompt's x, B, C and products; the token's only at the end), each by at most
2^-8 of a term; sums of up to 2^9 terms of random sign then differ by a few times 2^-8 of
their root mean square, and their largest of some thousands by up to five times that:
2^-8 * 3 * 5 = 0.06 at most.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "state_space_layer.py")


@pytest.mark.parametrize("more", [{}, dict(heads=6, head_size=80, groups=1, state_size=72, width=256),
                                  dict(heads=4, head_size=32, groups=4, state_size=16, lengths=(1, 2, 3, 300))])
def test_tokens_continue_prompts(more):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("state_space_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.run(**more) <= 0.06
